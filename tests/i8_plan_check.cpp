// Questions about csrc/i8_plan.h, one a line on standard input, answers on standard output:
//   order TOK_BLOCKS CH_BLOCKS BLOCK_BYTES GRID   -> group, and every tile visited once by GRID walkers that look one
//                                                    tile ahead ("ok" or what is wrong)
//   tiles M N K SMS                               -> bn, swap, token blocks, their group, tiles
//   split TILES K_STEPS LEAST LARGEST HELD2 .. HELD8 -> split of K where up to LARGEST parts fit and the device holds
//                                                    HELDk clusters of k, and the number of clusters that it holds
//   few M N K SMS HELD2 .. HELD8                  -> for 129 to 256 tokens: whether K is split instead of tiled, and the
//                                                    split
//   held FIRST SECOND                             -> three answers of asked_once (guess 5) where the device gives
//                                                    FIRST, then SECOND, and how often it was asked
#include <cstdio>
#include <cstring>
#include <vector>

#include "i8_plan.h"

using namespace nvfp4::i8;

static void order(int tok_blocks, int ch_blocks, int64_t block_bytes, int grid) {
  TileOrder o{tok_blocks, ch_blocks, token_group(tok_blocks, block_bytes)};
  const int tiles = tok_blocks * ch_blocks;
  std::vector<int> seen((size_t)tiles);
  for (int first = 0; first < std::min(grid, tiles); ++first) {
    int tok, ch;
    tile_blocks(o, first, &tok, &ch);
    for (int tile = first; tile < tiles; tile += grid) {
      if (tok < 0 || tok >= tok_blocks || ch < 0 || ch >= ch_blocks) {
        std::printf("%d tile %d at %d, %d\n", o.group, tile, tok, ch);
        return;
      }
      ++seen[(size_t)(tok * ch_blocks + ch)];
      tile_blocks(o, tile + grid, &tok, &ch);     // ahead, beyond the last one too
    }
  }
  for (int i = 0; i < tiles; ++i)
    if (seen[(size_t)i] != 1) {
      std::printf("%d block %d visited %d times\n", o.group, i, seen[(size_t)i]);
      return;
    }
  std::printf("%d ok\n", o.group);
}

static void tiles(int64_t M, int64_t N, int64_t K, int sms) {
  const Tiles t = choose_tiles(M, N, K, sms);
  const int64_t tok = t.swap ? (M + t.bn - 1) / t.bn : (M + 255) / 256, ch = t.swap ? (N + 255) / 256 : (N + t.bn - 1) / t.bn;
  std::printf("%d %d %lld %d %lld\n", t.bn, t.swap ? 1 : 0, (long long)tok, token_group((int)tok, (t.swap ? t.bn : 256) * K),
              (long long)(tok * ch));
}

static void split(int64_t tiles, int k_steps, int least, int largest) {
  int n[9], used = 0;
  for (int k = 2; k <= 8; ++k)
    if (std::scanf("%d", &n[k]) != 1) return;
  const int ks = split_of_k(tiles, k_steps, least, [&](int k) { return k <= largest; }, [&](int k) { used = n[k]; return n[k]; });
  std::printf("%d %d\n", ks, ks == 1 ? 0 : used);
}

static void few(int64_t M, int64_t N, int64_t K, int sms) {
  int n[9];
  for (int k = 2; k <= 8; ++k)
    if (std::scanf("%d", &n[k]) != 1) return;
  const int64_t row_tiles = (N + W_ROWS - 1) / W_ROWS;
  const int k_steps = (int)((K + BK - 1) / BK);
  const int ks = split_of_k(row_tiles, k_steps, 10, [&](int k) { return FewCfg<256, 1>::fits((int)M, k); }, [&](int k) { return n[k]; });
  std::printf("%d %d\n", few_ns(row_tiles, k_steps, ks, sms) < choose_tiles(M, N, K, sms).ns ? 1 : 0, ks);
}

static void held(int first, int second) {
  std::atomic<int> slot{0};
  int asked = 0;
  auto ask = [&] { return ++asked == 1 ? first : second; };
  for (int i = 0; i < 3; ++i) std::printf("%d ", asked_once(&slot, 5, ask));
  std::printf("%d\n", asked);
}

int main() {
  char what[16];
  while (std::scanf("%15s", what) == 1) {
    long long a, b, c, d;
    if (!std::strcmp(what, "order") && std::scanf("%lld %lld %lld %lld", &a, &b, &c, &d) == 4) order((int)a, (int)b, c, (int)d);
    else if (!std::strcmp(what, "tiles") && std::scanf("%lld %lld %lld %lld", &a, &b, &c, &d) == 4) tiles(a, b, c, (int)d);
    else if (!std::strcmp(what, "held") && std::scanf("%lld %lld", &a, &b) == 2) held((int)a, (int)b);
    else if (!std::strcmp(what, "split") && std::scanf("%lld %lld %lld %lld", &a, &b, &c, &d) == 4) split(a, (int)b, (int)c, (int)d);
    else if (!std::strcmp(what, "few") && std::scanf("%lld %lld %lld %lld", &a, &b, &c, &d) == 4) few(a, b, c, (int)d);
    else return 2;
    std::fflush(stdout);
  }
  return 0;
}
