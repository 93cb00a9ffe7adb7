// 8-bit integer linear on the 5th-generation tensor cores (tcgen05), sm_100a.
//
// Y[m, n] = (sum_k a[m, k] w[n, k]) * a_scale[m] * w_scale[n] (+ bias[n]), a and
// w int8, both K-major.  tcgen05.mma.kind::i8 accumulates in int32 in tensor
// memory; K < 2^17 keeps every sum below 2^31, so the products are exact and
// their order is free.  The epilogue rounds the sum to fp32, multiplies by the
// token's and then the channel's scale, adds the bias and rounds to Y's type.
//
// Structure (persistent; a pair of CTAs shares one 256-row tile, each
// holding 128 rows of A and of the accumulator and half of the W rows; 384
// threads per CTA):
//   warp 0     loads each stage by TMA (128-byte K-slices, 128-byte swizzle)
//              into a ring of 192 KB; both CTAs' copies arrive on the leader's
//              barrier;
//   warp 1     allocates 512 TMEM columns; the leader's issues the stage's MMAs
//              (K = 32 each); its commits free the stage in both CTAs and hand
//              the accumulator to the epilogue;
//   warps 4-11 two per TMEM lane quadrant: 64 bytes of each row of Y at a time
//              from TMEM, scaled, transposed through shared memory and stored
//              in segments of 16 bytes.  Two accumulators alternate, so a tile's
//              epilogue runs under the next tile's MMAs.
// Every mbarrier wait is bounded, as in the other tensor-core kernels.  The epilogue's
// warps meet at a barrier once per tile, so a warp that gave up goes on to the last
// tile's barrier without working.
//
// Bound: the tensor cores, 3.6 POP/s in bursts and 2.9 to 3.15 under the power cap
// (8192 x 28672 x 8192: 1075 and, by the device, 1223 to 1314 us); for a few waves of
// tiles the filling and the last epilogue, some 6 us, and the last wave's idle pairs
// (777 x 11008 x 4096: 31.5 us, 2.2 POP/s).
#include <algorithm>
#include <type_traits>

#include "i8_plan.h"
#include "i8_tc.cuh"
#include "kernels.h"

namespace nvfp4 {
using namespace tc;
namespace {

constexpr int CG = 2;                   // CTAs of a pair
constexpr int BM = 128;                 // rows of A per CTA
using i8::BK;                           // bytes (= elements) of K per stage: one swizzle row
using i8::BN_MAX;                       // columns per tile, at most
constexpr int A_BYTES = BM * BK;
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr uint32_t TMEM_COLS = 512;     // two accumulators of BN_MAX int32 columns
constexpr int RING_BYTES = 192 * 1024, MAX_STAGES = 12;
constexpr int EPI_PITCH = 20;           // words per staged row of 64 bytes: 16-byte aligned, no bank conflicts
constexpr int EPI_BYTES = EPI_WARPS * 32 * EPI_PITCH * 4;
constexpr int COL_BYTES = 2 * 2 * BN_MAX * 4;     // channel scales and bias of two tiles
constexpr int BAR_BYTES = 512;
constexpr int SMEM_BYTES = RING_BYTES + EPI_BYTES + COL_BYTES + BAR_BYTES + 1024;   // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert((2 * MAX_STAGES + 5) * 8 + 16 + 8 <= BAR_BYTES, "barrier block");

// A stage holds 128 rows of A and bn / CG rows of W; the ring takes as many as fit.
__host__ __device__ constexpr int stage_bytes(int bn) { return A_BYTES + bn / CG * BK; }

struct Params {
  const float* a_scales;
  const float* w_scales;
  const float* bias;
  void* y;
  int64_t ldy;
  int y_align;        // bytes that Y's base and row pitch are multiples of: 16, 4 or 2
  int M, N;           // of the tiles: SWAP has the channels as M and the tokens as N
  int bn;             // columns per tile, a multiple of 32
  int stages;         // of the ring
  i8::TileOrder order;
  int num_tiles, k_tiles;
  int* st;
  uint64_t wait_ns;
  int hold;
};

// The copy lands in this CTA, its bytes count on the leader's barrier (the same
// offset in the even-ranked CTA of the pair).
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar & 0xFEFFFFFFu)
      : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t remote_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_bar) : "memory");
}
// A whole warp's bounded wait: the same answer for every lane.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, WaitState* w, int* st) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_inline<true>(bar, parity, w, st)) != 0;
}

// SWAP: the tiles' rows are channels (W is the tensor cores' A) and their columns
// tokens, for token counts that fill tiles better along the columns' finer grid.
template <bool BF16OUT, bool SWAP>
__global__ void __launch_bounds__(THREADS, 1)
    k_i8_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Params p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t* epi = reinterpret_cast<uint32_t*>(smem + RING_BYTES);
  float* cols = reinterpret_cast<float*>(smem + RING_BYTES + EPI_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + RING_BYTES + EPI_BYTES + COL_BYTES);
  uint64_t* full = bars;                      // [stages] tiles landed (the leader's, for both CTAs)
  uint64_t* empty = bars + MAX_STAGES;        // [stages] MMAs done
  uint64_t* acc_full = bars + 2 * MAX_STAGES; // [2]
  uint64_t* acc_empty = acc_full + 2;         // [2] the epilogue has read the accumulator (the leader's counts both CTAs)
  uint64_t* mma_drain = acc_empty + 2;
  WaitState* ws = reinterpret_cast<WaitState*>(mma_drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ws + 1);

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int group = blockIdx.x / CG, groups = gridDim.x / CG;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(saddr(&full[s]), 1);
      mbar_init(saddr(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(saddr(&acc_full[b]), 1);
      mbar_init(saddr(&acc_empty[b]), EPI_WARPS * CG);
    }
    mbar_init(saddr(mma_drain), 1);
    ws->abort = 0;
    ws->limit_ns = p.wait_ns;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmA) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmB) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync();   // the peer's barriers exist
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    const uint32_t bytes = (uint32_t)(CG * A_BYTES + p.bn * BK);   // of both CTAs
    const int stage = stage_bytes(p.bn);
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = p.hold != kHoldLoads;
    int tok, ch;
    i8::tile_blocks(p.order, group, &tok, &ch);
    for (int tile = group; ok && tile < p.num_tiles; tile += groups) {
      const int mb = SWAP ? ch : tok, nb = SWAP ? tok : ch;
      const int a_row = (mb * CG + (int)rank) * BM, w_row = nb * p.bn + (int)rank * (p.bn / CG);
      for (int kt = 0; kt < p.k_tiles; ++kt) {
        ok = wait_all(saddr(&empty[s]), ph ^ 1u, ws, p.st);
        if (!ok) break;
        const uint32_t dst = saddr(smem) + (uint32_t)(s * stage), bar = saddr(&full[s]);
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(bar, bytes);
          load_2d(dst, &tmA, kt * BK, a_row, bar);
          load_2d(dst + A_BYTES, &tmB, kt * BK, w_row, bar);
        }
        __syncwarp();
        if (kt == 0) i8::tile_blocks(p.order, tile + groups, &tok, &ch);    // the next tile's place, off the ring's critical path
        ++issued;
        if (++s == p.stages) { s = 0; ph ^= 1u; }
      }
    }
    // Copies still in flight if a consumer gave up land before the CTA can exit.  The
    // leader's barriers count both CTAs' copies, but only of stages that the leader
    // issued too: the CTA that gave up (either may be first) gives the other's last
    // ones time to land, copies take microseconds, and neither leaves before both
    // have come to the cluster's last barrier.
    if (rank == 0) {
      for (int i = max(0, issued - p.stages); i < issued; ++i)
        (void)mbar_drain<true>(saddr(&full[i % p.stages]), (uint32_t)((i / p.stages) & 1), ws, p.st);
    }
    if (wait_aborted(ws)) {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t idesc = idesc_i8(BM * CG, p.bn);
    const int stage = stage_bytes(p.bn);
    int s = 0, local = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = group; ok && tile < p.num_tiles; tile += groups, ++local) {
      const int b = local & 1;
      ok = wait_all(saddr(&acc_empty[b]), (uint32_t)((local >> 1) & 1) ^ 1u, ws, p.st);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(b * BN_MAX);
      for (int kt = 0; kt < p.k_tiles; ++kt) {
        ok = wait_all(saddr(&full[s]), ph, ws, p.st);
        if (!ok) break;
        tc_fence_after();
        const uint32_t base = saddr(smem) + (uint32_t)(s * stage);
        const uint64_t da = desc_sw128(base), db = desc_sw128(base + A_BYTES);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j)       // bytes past K are zeros
            mma_i8<CG>(acc, da + (uint64_t)(2 * j), db + (uint64_t)(2 * j), idesc, (kt > 0 || j > 0) ? 1u : 0u);
          commit<CG>(saddr(&empty[s]));
          if (kt == p.k_tiles - 1) commit<CG>(saddr(&acc_full[b]));
        }
        __syncwarp();
        if (++s == p.stages) { s = 0; ph ^= 1u; }
      }
    }
    // every MMA issued has completed before TMEM can be released
    if (elect_one()) commit<CG>(saddr(mma_drain));
    __syncwarp();
    (void)mbar_drain<true>(saddr(mma_drain), 0u, ws, p.st);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 4) >> 2, et = threadIdx.x - 128;
    using Out = std::conditional_t<BF16OUT, __nv_bfloat16, float>;
    constexpr int W = BF16OUT ? 32 : 16;                 // columns staged at a time: rows of 64 bytes
    constexpr int PER = BF16OUT ? 8 : 4;                 // elements per 16-byte segment
    uint32_t* buf = epi + (warp - 4) * 32 * EPI_PITCH;
    const uint32_t quad = (uint32_t)(q * 32) << 16;
    int local = 0;
    bool ok = true;            // of this warp: the others may not have given up yet
    for (int tile = group; tile < p.num_tiles; tile += groups, ++local) {
      int tok, ch;
      i8::tile_blocks(p.order, tile, &tok, &ch);
      const int mb = SWAP ? ch : tok, nb = SWAP ? tok : ch, b = local & 1;
      const int row0 = (mb * CG + (int)rank) * BM + q * 32, n0 = nb * p.bn, n_end = min(p.N, n0 + p.bn);
      float* ct = cols + b * 2 * BN_MAX;
      for (int c = et; c < p.bn; c += 32 * EPI_WARPS) {
        const bool in = n0 + c < p.N;
        ct[c] = in ? (SWAP ? p.a_scales : p.w_scales)[n0 + c] : 0.0f;
        ct[BN_MAX + c] = !SWAP && in && p.bias != nullptr ? p.bias[n0 + c] : kNoBias;
      }
      const bool row_in = row0 + lane < p.M;
      const float sr = row_in ? (SWAP ? p.w_scales : p.a_scales)[row0 + lane] : 0.0f;
      const float bias_r = SWAP && row_in && p.bias != nullptr ? p.bias[row0 + lane] : kNoBias;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (p.hold == kHoldOneWarp && warp == 4 && ok) {
        if (lane == 0) {
          wait_raise(ws);
          report_status(p.st, NVFP4_ERR_TIMEOUT);
        }
        ok = false;
      }
      ok = ok && warp_wait<true>(saddr(&acc_full[b]), (uint32_t)((local >> 1) & 1), ws, p.st);
      if (!ok) continue;
      tc_fence_after();
      auto release = [&] {                                // this warp has read its part of the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(mapa_shared(saddr(&acc_empty[b]), 0));
      };
      // the two warps of a TMEM lane quadrant take alternate runs of W columns
      const int c_end = row0 < p.M ? n_end - n0 : 0;      // uniform across the warp
      if (half * W >= c_end) release();
      for (int c0 = half * W; c0 < c_end; c0 += 2 * W) {
        uint32_t r[W];
        if constexpr (BF16OUT) tmem_ld32(tmem + quad + (uint32_t)(b * BN_MAX + c0), r);
        else tmem_ld16(tmem + quad + (uint32_t)(b * BN_MAX + c0), r);
        tmem_ld_wait();
        if (c0 + 2 * W >= c_end) release();
        if constexpr (SWAP) {
          // a lane's row is a column of Y: one token's 32 columns a store
          Out* y = static_cast<Out*>(p.y) + (int64_t)(n0 + c0) * p.ldy + row0 + lane;
          const int left = row_in ? n_end - n0 - c0 : 0;
#pragma unroll
          for (int i = 0; i < W; i += 4) {
            const float4 t = *reinterpret_cast<const float4*>(ct + c0 + i);
            const float s4[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int e = 0; e < 4; ++e, y += p.ldy) {
              const float f = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[i + e]), s4[e]), sr), bias_r);
              if (i + e < left) {
                if constexpr (BF16OUT) *y = __float2bfloat16_rn(f);
                else *y = f;
              }
            }
          }
          continue;
        }
        const float4* sw4 = reinterpret_cast<const float4*>(ct + c0);
        const float4* bi4 = reinterpret_cast<const float4*>(ct + BN_MAX + c0);
        float v[W];
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const float4 s4 = sw4[i], b4 = bi4[i];
          v[4 * i] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * i]), sr), s4.x), b4.x);
          v[4 * i + 1] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * i + 1]), sr), s4.y), b4.y);
          v[4 * i + 2] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * i + 2]), sr), s4.z), b4.z);
          v[4 * i + 3] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * i + 3]), sr), s4.w), b4.w);
        }
        uint4* mine = reinterpret_cast<uint4*>(buf + lane * EPI_PITCH);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if constexpr (BF16OUT)
            mine[g] = make_uint4(pack_bf16x2(v[8 * g], v[8 * g + 1]), pack_bf16x2(v[8 * g + 2], v[8 * g + 3]),
                                 pack_bf16x2(v[8 * g + 4], v[8 * g + 5]), pack_bf16x2(v[8 * g + 6], v[8 * g + 7]));
          else
            mine[g] = make_uint4(__float_as_uint(v[4 * g]), __float_as_uint(v[4 * g + 1]),
                                 __float_as_uint(v[4 * g + 2]), __float_as_uint(v[4 * g + 3]));
        }
        __syncwarp();
        if (p.y_align == 16) {
          // four lanes per row segment of 64 bytes, eight rows a store
          const int col = n0 + c0 + (lane & 3) * PER, left = n_end - col;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int lr = h * 8 + (lane >> 2), row = row0 + lr;
            const uint32_t* src = buf + lr * EPI_PITCH + (lane & 3) * 4;
            if (row < p.M && left > 0) {
              const int64_t off = (int64_t)row * p.ldy + col;
              if (left >= PER) {
                *reinterpret_cast<uint4*>(static_cast<Out*>(p.y) + off) = *reinterpret_cast<const uint4*>(src);
              } else {
                for (int e = 0; e < left; ++e) static_cast<Out*>(p.y)[off + e] = reinterpret_cast<const Out*>(src)[e];
              }
            }
          }
        } else if (!BF16OUT || p.y_align == 4) {
          // sixteen lanes per row segment, a word each (odd row pitches of fp32, even ones of bf16)
          constexpr int EW = BF16OUT ? 2 : 1;
          const int col = n0 + c0 + (lane & 15) * EW, left = n_end - col;
          Out* y = static_cast<Out*>(p.y) + (int64_t)(row0 + (lane >> 4)) * p.ldy + col;
          const uint32_t* src = buf + (lane >> 4) * EPI_PITCH + (lane & 15);
          for (int row = row0 + (lane >> 4), h = 0; h < 16; ++h, row += 2, y += 2 * p.ldy, src += 2 * EPI_PITCH) {
            if (row >= p.M || left <= 0) continue;
            if (left >= EW) *reinterpret_cast<uint32_t*>(y) = *src;
            else *y = *reinterpret_cast<const Out*>(src);
          }
        } else {
          // odd row pitches of bf16: a whole warp per row segment (8 elements a lane took 1014 us for 6978 x 23122 x 3472)
          const int col = n0 + c0 + lane;
          Out* y = static_cast<Out*>(p.y) + (int64_t)row0 * p.ldy + col;
          const Out* src = reinterpret_cast<const Out*>(buf) + lane;
          const int rows = col < n_end ? min(32, p.M - row0) : 0;
#pragma unroll 4
          for (int h = 0; h < rows; ++h, y += p.ldy, src += 2 * EPI_PITCH) *y = *src;
        }
        __syncwarp();
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();   // the pair's MMAs and arrivals are over before either CTA leaves
  if (warp == 1) {
    // the leader's last commit, issued before it came here, arrives in the other CTA too
    if (rank != 0) (void)mbar_drain<true>(saddr(mma_drain), 0u, ws, p.st);
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

template <bool SWAP>
cudaError_t launch_tiles(const I8GemmArgs& g, int bn, int num_sms, cudaStream_t stream) {
  const int64_t rows = SWAP ? g.N : g.M, columns = SWAP ? g.M : g.N;
  const int64_t mb = (rows + BM * CG - 1) / (BM * CG), nb = (columns + bn - 1) / bn;
  if (mb * nb > INT32_MAX - 4096) return cudaErrorNotSupported;    // 32-bit tile numbers, one grid beyond the last
  CUtensorMap tmA, tmW;
  if (!encode_i8_map(&tmA, g.a, g.M, g.K, g.lda, (uint32_t)(SWAP ? bn / CG : BM)) ||
      !encode_i8_map(&tmW, g.w, g.N, g.K, g.ldw, (uint32_t)(SWAP ? BM : bn / CG)))
    return cudaErrorInvalidValue;
  Params p{};
  p.a_scales = g.a_scales; p.w_scales = g.w_scales; p.bias = g.bias;
  p.y = g.y; p.ldy = g.ldy;
  const uint64_t bytes = reinterpret_cast<uintptr_t>(g.y) | ((uint64_t)g.ldy * (g.y_bf16 ? 2 : 4));
  p.y_align = bytes % 16 == 0 ? 16 : bytes % 4 == 0 ? 4 : 2;
  p.M = (int)rows; p.N = (int)columns; p.bn = bn;
  p.stages = std::min(MAX_STAGES, RING_BYTES / stage_bytes(bn));
  p.num_tiles = (int)(mb * nb); p.k_tiles = (int)((g.K + BK - 1) / BK);
  p.order.tok_blocks = (int)(SWAP ? nb : mb); p.order.ch_blocks = (int)(SWAP ? mb : nb);
  p.order.group = i8::token_group(p.order.tok_blocks, (int64_t)(SWAP ? bn : BM * CG) * g.K);
  p.st = g.st;
  const WaitTest wt = wait_test();
  p.wait_ns = wt.limit_ns; p.hold = wt.hold;
  auto kern = g.y_bf16 ? k_i8_gemm<true, SWAP> : k_i8_gemm<false, SWAP>;
  static SmemOnce once[2];
  cudaError_t e = once[g.y_bf16 ? 1 : 0].set(kern, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(CG * std::max(1, std::min(p.num_tiles, num_sms / CG))));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CG; at[1].val.clusterDim.y = 1; at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, SWAP ? tmW : tmA, SWAP ? tmA : tmW, p);
}

}  // namespace

namespace tc {
bool encode_i8_map(CUtensorMap* map, const int8_t* p, int64_t rows, int64_t K, int64_t ld, uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {(cuuint32_t)128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace tc

cudaError_t launch_i8_gemm(const I8GemmArgs& g, int num_sms, cudaStream_t stream) {
  // One to four tokens: the CUDA cores keep up with W's bytes and start and end
  // sooner (1 x 14336 x 4096: 11.1 us, the tensor-core kernel 13.0; 4 tokens: 11.9
  // and 13.1; 8 tokens: 17.8 and 12.9).
  if (g.M <= 4) return launch_i8_gemv(g, num_sms, stream);
  // Up to 128 tokens W's rows fill the tensor cores' M better than the tokens do
  // (128 x 5120 x 5120: 11.6 us, tiles of 256 tokens x 96 columns 13.8).
  if (g.M <= 128) return launch_i8_gemm_few(g, num_sms, stream);
  // Beyond, tiles of a pair of CTAs by an estimate.  Up to 256 tokens splitting K
  // instead can win (256 x 5120 x 27648: 40 us, tiles 52 us; 256 x 4096 x 4096: 13.7
  // and 11.5 us).
  const i8::Tiles t = i8::choose_tiles(g.M, g.N, g.K, num_sms);
  if (g.M <= 256 && i8_gemm_few_ns(g.M, g.N, g.K, num_sms) < t.ns) return launch_i8_gemm_few(g, num_sms, stream);
  return t.swap ? launch_tiles<true>(g, t.bn, num_sms, stream) : launch_tiles<false>(g, t.bn, num_sms, stream);
}

}  // namespace nvfp4
