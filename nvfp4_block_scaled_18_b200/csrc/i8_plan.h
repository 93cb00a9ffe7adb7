// Choices of the 8-bit linear's launchers and the order of its tiles, in plain
// C++: they compile without CUDA, so that they can be checked without a GPU.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>

#ifdef __CUDACC__
#define NVFP4_HD __host__ __device__ __forceinline__
#else
#define NVFP4_HD inline
#endif

namespace nvfp4 {
namespace i8 {

constexpr int BK = 128;       // bytes (= elements) of K per stage of the tensor-core kernels
constexpr int BN_MAX = 256;   // columns per tile, at most

// Tiles of a pair of CTAs: 256 tokens x bn channels, or (swap) 256 channels x bn
// tokens, by an estimate.  A K-slice takes 84 ns + 1 ns a column, and 222 ns at
// least (measured, 128 to 256 columns); filling, the last epilogue and the launch
// come on top (777 x 11008 x 4096: 160 tokens wide 32.4 us, 224 channels wide 35.6;
// 512 x 4096 x 14336: 128 channels wide 29.4, 224 wide 33.0).
struct Tiles {
  int bn;
  bool swap;
  double ns;                  // the estimate
};
inline Tiles choose_tiles(int64_t M, int64_t N, int64_t K, int num_sms) {
  const int64_t k_tiles = (K + BK - 1) / BK, pairs = std::max(1, num_sms / 2);
  Tiles best{0, false, 0.0};
  for (int side = 0; side < 2; ++side) {
    const int64_t rows = side ? N : M, columns = side ? M : N, mb = (rows + 255) / 256;
    for (int c = 32; c <= BN_MAX; c += 32) {
      const int64_t waves = (mb * ((columns + c - 1) / c) + pairs - 1) / pairs;
      const double ns = 5000.0 + 8.0 * c + (double)(waves * k_tiles) * std::max(222.0, 84.0 + c) + (side ? 500.0 : 0.0);
      if (best.bn == 0 || ns < best.ns || (!side && ns <= best.ns)) best = Tiles{c, side != 0, ns};
    }
  }
  return best;
}

// The tiles' order: groups of token blocks, within a group channel by channel
// block, tokens fastest.  The CTAs in flight then share W's tiles, and the group's
// tokens stay in L2 while all of W passes.  A tile beyond the last one has no place:
// what it is given is not used, only defined.
struct TileOrder {
  int tok_blocks, ch_blocks;   // blocks of tokens and of channels
  int group;                   // token blocks that W passes by at a time
};
NVFP4_HD void tile_blocks(const TileOrder& o, int tile, int* tok, int* ch) {
  const int per = o.group * o.ch_blocks, g = tile / per, r = tile - g * per;
  const int left = o.tok_blocks - g * o.group, wide = left >= o.group ? o.group : left > 1 ? left : 1;
  *ch = r / wide;
  *tok = g * o.group + r - *ch * wide;
}

// Tokens in groups of 32 MB: 8192 x 28672 x 8192, again and again under the power
// cap, takes 1281 us so, 1436 in one group of 67 MB, which W pushes out of L2, and
// 1338 in groups of 17 MB, for each of which W comes once from DRAM (8192 x 4096 x
// 14336: 341, 371 and 350 us; all on one device).  block_bytes: of a block of tokens.
inline int token_group(int tok_blocks, int64_t block_bytes) {
  const int64_t most = std::max<int64_t>(1, (32ll << 20) / block_bytes), groups = (tok_blocks + most - 1) / most;
  return (int)((tok_blocks + groups - 1) / groups);
}

// k_i8_few: a row tile of W, and the barriers' block.
constexpr int W_ROWS = 128, FEW_BAR_BYTES = 256;

// k_i8_few's shared and tensor memory for NP tokens.
template <int NP, int CTAS>     // CTAS: per SM
struct FewCfg {
  static constexpr int W_BYTES = W_ROWS * BK, X_BYTES = NP * BK;
  static constexpr int STAGE = W_BYTES + X_BYTES;         // one 128-byte K-slice
  // Tokens are owned, staged and sent G at a time.  Partial sums that arrive from
  // the ks - 1 others, [source][token of the owner][row], have an area of their
  // own up to 64 tokens; for more they share the ring with those to be sent.
  static constexpr int G = NP <= 32 ? 4 : 16;
  static constexpr int PART = NP <= 16 ? 14 * 1024 : NP <= 32 ? 16 * 1024 : 32 * 1024;
  static constexpr bool OVERLAY = NP > 64 || CTAS == 1;
  // the SM's 228 KB less 1 KB per CTA, and the barriers, the alignment and the static part
  static constexpr int STAGES_FIT = (233472 / CTAS - 1024 - 1024 - FEW_BAR_BYTES - NP * 4 - 64 - (OVERLAY ? 0 : PART)) / STAGE;
  static constexpr int STAGES = STAGES_FIT < 8 ? STAGES_FIT : 8;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int SMEM = RING + (OVERLAY ? 0 : PART) + FEW_BAR_BYTES + 1024;
  static constexpr uint32_t TMEM_COLS = NP < 32 ? 32 : NP;
  // Of k CTAs: tokens per owner, and whether what is sent and what arrives fits.
  static int per_owner(int M, int k) { return (M + G * k - 1) / (G * k) * G; }
  static bool fits(int M, int k) {
    const int t = per_owner(M, k), all = (M + G - 1) / G * G;
    const int sent = (all - std::max(0, all - (k - 1) * t)) * 512, arrives = (k - 1) * t * 512;   // at most, by the last CTA
    return OVERLAY ? sent + arrives <= RING : sent <= RING && arrives <= PART;
  }
  static_assert((2 * STAGES + 2) * 8 + 16 + 8 <= FEW_BAR_BYTES, "barrier block");
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert((int64_t)(SMEM + 1024) * 512 >= (int64_t)233472 * TMEM_COLS,
                "a share of the SM's shared memory as large as that of its tensor memory, so that tcgen05.alloc waits for none");
  static_assert(X_BYTES % 1024 == 0 && STAGE % 1024 == 0, "128-byte swizzle atoms");
};

// k_i8_few: the largest split of K, up to eight CTAs a cluster, that leaves each CTA
// `least` steps of K to pay for joining them, whose partial sums fit (fits(k)) and
// whose clusters, one a tile, all run at once: the device holds held(k) of them.
template <typename Fits, typename Held>
int split_of_k(int64_t tiles, int k_steps, int least, Fits fits, Held held) {
  for (int k = 8; k >= 2; --k)
    if (k * least <= k_steps && fits(k) && tiles <= held(k)) return k;
  return 1;
}

// Estimated time of k_i8_few for 129 to 256 tokens with K in ks parts.
inline double few_ns(int64_t tiles, int k_steps, int ks, int num_sms) {
  const int64_t waves = (tiles * ks + num_sms - 1) / num_sms;
  return 10000.0 + 460.0 * (double)waves * (double)((k_steps + ks - 1) / ks);
}

// An answer of the device that does not change, asked once; ask() gives -1 for none.
template <typename Ask>
int asked_once(std::atomic<int>* slot, int guess, Ask ask) {
  int n = slot != nullptr ? slot->load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  n = ask();
  if (n < 0) return guess;              // not known: for this call alone
  if (slot != nullptr) slot->store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace i8
}  // namespace nvfp4
