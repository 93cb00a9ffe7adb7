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
// cap, takes 1271 us so, 1423 in one group of 67 MB, which W pushes out of L2, and
// 1293 in groups of 17 MB, for each of which W comes once from DRAM (8192 x 4096 x
// 14336: 337, 374 and 342 us).  block_bytes: of a block of tokens.
inline int token_group(int tok_blocks, int64_t block_bytes) {
  const int64_t most = std::max<int64_t>(1, (32ll << 20) / block_bytes), groups = (tok_blocks + most - 1) / most;
  return (int)((tok_blocks + groups - 1) / groups);
}

// k_i8_few: the largest split of K, up to eight CTAs a cluster, that leaves each CTA
// `least` steps of K to pay for joining them, whose partial sums fit (fits(k)) and
// whose clusters, one a tile, all run at once: the device holds held(k) of them.
template <typename Fits, typename Held>
int split_of_k(int64_t tiles, int k_steps, int least, Fits fits, Held held) {
  for (int k = 8; k >= 2; --k)
    if (k * least <= k_steps && fits(k) && tiles <= held(k)) return k;
  return 1;
}

// An answer of the device that does not change, asked once.
template <typename Ask>
int asked_once(std::atomic<int>* slot, int guess, Ask ask) {
  int n = slot != nullptr ? slot->load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  n = ask();
  if (n <= 0) return guess;             // not known: for this call alone
  if (slot != nullptr) slot->store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace i8
}  // namespace nvfp4
