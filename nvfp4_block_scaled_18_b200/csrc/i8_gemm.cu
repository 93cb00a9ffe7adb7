// 8-bit integer linear on the 5th-generation tensor cores (tcgen05), sm_100a.
//
// Y[m, n] = (sum_k a[m, k] w[n, k]) * a_scale[m] * w_scale[n] (+ bias[n]), a and
// w int8, both K-major.  tcgen05.mma.kind::i8 accumulates in int32 in tensor
// memory; K < 2^17 keeps every sum below 2^31, so the products are exact and
// their order is free.  The epilogue rounds the sum to fp32, multiplies by the
// token's and then the channel's scale, adds the bias and rounds to Y's type.
//
// Structure (persistent; CG = 2: a pair of CTAs shares one 256-row tile, each
// holding 128 rows of A and of the accumulator and half of the W rows; 256
// threads per CTA):
//   warp 0     one lane loads each stage by TMA (128-byte K-slices, 128-byte
//              swizzle) into a ring; both CTAs' copies arrive on the leader's
//              barrier;
//   warp 1     allocates 512 TMEM columns; one lane of the leader issues the
//              stage's MMAs (K = 32 each); its commits free the stage in both
//              CTAs and hand the accumulator to the epilogue;
//   warps 4-7  one per TMEM lane quadrant: 32 columns at a time from TMEM,
//              scaled, transposed through shared memory and stored with 16-byte
//              row segments.  Two accumulators alternate, so a tile's epilogue
//              runs under the next tile's MMAs.
// Every mbarrier wait is bounded, as in the other tensor-core kernels.
#include <algorithm>

#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4 {
using namespace tc;
namespace {

constexpr int BM = 128;                 // rows of A per CTA
constexpr int BK = 128;                 // bytes (= elements) of K per stage: one swizzle row
constexpr int BN_MAX = 256;             // columns per tile
constexpr int A_BYTES = BM * BK;
constexpr int THREADS = 256;
constexpr uint32_t TMEM_COLS = 512;     // two accumulators of BN_MAX int32 columns
constexpr int EPI_PITCH_W = 36;         // words per staged row of 32 fp32 (bf16: 20), 16-byte aligned, no conflicts
constexpr int EPI_BYTES = 4 * 32 * EPI_PITCH_W * 4;
constexpr int COL_BYTES = 2 * 2 * BN_MAX * 4;     // channel scales and bias of two tiles
constexpr int BAR_BYTES = 256;

template <int CG>
struct Cfg {
  static constexpr int B_BYTES = BN_MAX / CG * BK;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = CG == 2 ? 6 : 4;
  static constexpr int SMEM = STAGES * STAGE + EPI_BYTES + COL_BYTES + BAR_BYTES + 1024;   // + alignment slack
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert((2 * STAGES + 5) * 8 + 16 + 8 <= BAR_BYTES, "barrier block");
};

struct Params {
  const float* a_scales;
  const float* w_scales;
  const float* bias;
  void* y;
  int64_t ldy;
  int y_vec;          // Y's base and row pitch allow 16-byte stores
  int M, N, K;
  int bn;             // columns per tile
  int m_blocks, num_tiles, k_tiles;
  int* st;
  uint64_t wait_ns;
  int hold;
};

// kind::i8: int8 A and B (both K-major), int32 accumulator, M rows, N columns.
__device__ __forceinline__ uint32_t idesc_i8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive, once the MMAs issued so far are complete, on this barrier of every CTA of the group.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    tc_commit(bar);
}
// CG = 2: the copy lands in this CTA, its bytes count on the leader's barrier
// (the same offset in the even-ranked CTA of the pair).
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar & 0xFEFFFFFFu)
        : "memory");
  else
    tma_load_2d(dst, map, c0, c1, bar);
}
__device__ __forceinline__ void arrive_cluster(uint32_t remote_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_bar) : "memory");
}

template <int CG, bool BF16OUT>
__global__ void __launch_bounds__(THREADS, 1)
    k_i8_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Params p) {
  using C = Cfg<CG>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t* epi = reinterpret_cast<uint32_t*>(smem + STAGES * C::STAGE);
  float* cols = reinterpret_cast<float*>(smem + STAGES * C::STAGE + EPI_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE + EPI_BYTES + COL_BYTES);
  uint64_t* full = bars;                  // [STAGES] tiles landed (CG = 2: the leader's, for both CTAs)
  uint64_t* empty = bars + STAGES;        // [STAGES] MMAs done
  uint64_t* acc_full = bars + 2 * STAGES; // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2] the epilogue has read the accumulator (the leader's counts both CTAs)
  uint64_t* mma_drain = acc_empty + 2;
  WaitState* ws = reinterpret_cast<WaitState*>(mma_drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ws + 1);

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const int group = blockIdx.x / CG, groups = gridDim.x / CG;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(saddr(&full[s]), 1);
      mbar_init(saddr(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(saddr(&acc_full[b]), 1);
      mbar_init(saddr(&acc_empty[b]), 4 * CG);
    }
    mbar_init(saddr(mma_drain), 1);
    ws->abort = 0;
    ws->limit_ns = p.wait_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();   // the peer's barriers exist
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  if (warp == 0 && lane == 0) {
    // -------------------------------------------------------- TMA producer
    const uint32_t bytes = (uint32_t)(CG * A_BYTES + p.bn * BK);   // of both CTAs
    int g = 0;
    if (!p.hold)
      for (int tile = group; tile < p.num_tiles; tile += groups) {
        const int mb = tile % p.m_blocks, nb = tile / p.m_blocks;
        for (int kt = 0; kt < p.k_tiles; ++kt, ++g) {
          const int s = g % STAGES;
          if (!mbar_wait_inline<CG == 2>(saddr(&empty[s]), (uint32_t)((g / STAGES) & 1) ^ 1u, ws, p.st)) goto producer_done;
          uint8_t* st_base = smem + s * C::STAGE;
          const uint32_t bar = saddr(&full[s]);
          if (rank == 0) mbar_expect_tx(bar, bytes);
          load_2d<CG>(saddr(st_base), &tmA, kt * BK, (mb * CG + (int)rank) * BM, bar);
          load_2d<CG>(saddr(st_base + A_BYTES), &tmB, kt * BK, nb * p.bn + (int)rank * (p.bn / CG), bar);
        }
      }
  producer_done:
    // copies still in flight if a consumer gave up land before the CTA can exit
    if (rank == 0) {
      for (int g2 = max(0, g - STAGES); g2 < g; ++g2)
        (void)mbar_drain<CG == 2>(saddr(&full[g2 % STAGES]), (uint32_t)((g2 / STAGES) & 1), ws, p.st);
    } else if (wait_aborted(ws)) {
      // the leader's barrier counts this CTA's copies: give them time to land (copies take microseconds)
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t idesc = idesc_i8(BM * CG, p.bn);
    int g = 0, local = 0;
    for (int tile = group; tile < p.num_tiles; tile += groups, ++local) {
      const int b = local & 1;
      if (!mbar_wait_inline<CG == 2>(saddr(&acc_empty[b]), (uint32_t)((local >> 1) & 1) ^ 1u, ws, p.st)) goto mma_done;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(b * BN_MAX);
      for (int kt = 0; kt < p.k_tiles; ++kt, ++g) {
        const int s = g % STAGES;
        if (!mbar_wait_inline<CG == 2>(saddr(&full[s]), (uint32_t)((g / STAGES) & 1), ws, p.st)) goto mma_done;
        tc_fence_after();
        const uint8_t* st_base = smem + s * C::STAGE;
        const uint64_t da = desc_sw128(saddr(st_base)), db = desc_sw128(saddr(st_base + A_BYTES));
        const int jmax = min(4, (p.K - kt * BK + 31) / 32);
        for (int j = 0; j < jmax; ++j)
          mma_i8<CG>(acc, da + (uint64_t)(2 * j), db + (uint64_t)(2 * j), idesc, (kt > 0 || j > 0) ? 1u : 0u);
        commit<CG>(saddr(&empty[s]));
      }
      commit<CG>(saddr(&acc_full[b]));
    }
  mma_done:
    // every MMA issued has completed before TMEM can be released
    commit<CG>(saddr(mma_drain));
    (void)mbar_drain<CG == 2>(saddr(mma_drain), 0u, ws, p.st);
  } else if (CG == 2 && warp == 1 && lane == 0) {
    (void)mbar_drain<true>(saddr(mma_drain), 0u, ws, p.st);   // the leader's last commit has arrived here too
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, et = threadIdx.x - 128;
    constexpr int PITCH = BF16OUT ? 20 : EPI_PITCH_W;    // words
    constexpr int SEGS = BF16OUT ? 4 : 8;                // 16-byte segments per staged row
    constexpr int PER = BF16OUT ? 8 : 4;                 // elements per segment
    uint32_t* buf = epi + q * 32 * EPI_PITCH_W;
    int local = 0;
    for (int tile = group; tile < p.num_tiles; tile += groups, ++local) {
      const int mb = tile % p.m_blocks, nb = tile / p.m_blocks, b = local & 1;
      const int row0 = (mb * CG + (int)rank) * BM + q * 32, n0 = nb * p.bn;
      float* ct = cols + b * 2 * BN_MAX;
      for (int c = et; c < p.bn; c += 128) {
        const bool in = n0 + c < p.N;
        ct[c] = in ? p.w_scales[n0 + c] : 0.0f;
        ct[BN_MAX + c] = in && p.bias != nullptr ? p.bias[n0 + c] : 0.0f;
      }
      const float sa = row0 + lane < p.M ? p.a_scales[row0 + lane] : 0.0f;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_inline<CG == 2>(saddr(&acc_full[b]), (uint32_t)((local >> 1) & 1),
                                                                       ws, p.st)) != 0;
      if (!ok) break;
      tc_fence_after();
      for (int c0 = 0; c0 < p.bn; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BN_MAX + c0), r);
        tmem_ld_wait();
        if (c0 + 32 >= p.bn) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2) arrive_cluster(mapa_shared(saddr(&acc_empty[b]), 0));
            else mbar_arrive(saddr(&acc_empty[b]));
          }
        }
        if (n0 + c0 >= p.N || row0 >= p.M) continue;     // uniform across the warp
        const float4* sw4 = reinterpret_cast<const float4*>(ct + c0);
        const float4* bi4 = reinterpret_cast<const float4*>(ct + BN_MAX + c0);
        float v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 s4 = sw4[i], b4 = bi4[i];
          v[4 * i] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * i]), sa), s4.x), b4.x);
          v[4 * i + 1] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * i + 1]), sa), s4.y), b4.y);
          v[4 * i + 2] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * i + 2]), sa), s4.z), b4.z);
          v[4 * i + 3] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)r[4 * i + 3]), sa), s4.w), b4.w);
        }
        uint4* mine = reinterpret_cast<uint4*>(buf + lane * PITCH);
#pragma unroll
        for (int s = 0; s < SEGS; ++s) {
          if constexpr (BF16OUT)
            mine[s] = make_uint4(pack_bf16x2(v[8 * s], v[8 * s + 1]), pack_bf16x2(v[8 * s + 2], v[8 * s + 3]),
                                 pack_bf16x2(v[8 * s + 4], v[8 * s + 5]), pack_bf16x2(v[8 * s + 6], v[8 * s + 7]));
          else
            mine[s] = make_uint4(__float_as_uint(v[4 * s]), __float_as_uint(v[4 * s + 1]),
                                 __float_as_uint(v[4 * s + 2]), __float_as_uint(v[4 * s + 3]));
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < SEGS; ++h) {
          const int lr = h * (32 / SEGS) + lane / SEGS, sg = lane % SEGS;
          const int row = row0 + lr, col = n0 + c0 + sg * PER;
          const uint32_t* src = buf + lr * PITCH + sg * 4;
          // a tile of fewer than 32 trailing columns belongs to the next tile beyond p.bn
          const int left = min(p.N, n0 + p.bn) - col;
          if (row < p.M && left > 0) {
            const int64_t off = (int64_t)row * p.ldy + col;
            if (p.y_vec && left >= PER) {
              const uint4 o = *reinterpret_cast<const uint4*>(src);
              if (BF16OUT) *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.y) + off) = o;
              else *reinterpret_cast<uint4*>(reinterpret_cast<float*>(p.y) + off) = o;
            } else {
              for (int e = 0; e < PER && e < left; ++e) {
                if (BF16OUT)
                  reinterpret_cast<__nv_bfloat16*>(p.y)[off + e] = reinterpret_cast<const __nv_bfloat16*>(src)[e];
                else
                  reinterpret_cast<float*>(p.y)[off + e] = reinterpret_cast<const float*>(src)[e];
              }
            }
          }
        }
        __syncwarp();
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();   // the pair's MMAs and arrivals are over before either CTA leaves
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

// 2-D tensor map over int8 rows (rows x K, row pitch ld bytes): boxes of 128
// bytes x box_rows rows, 128-byte swizzle, zero fill out of range.
bool encode_i8_map(CUtensorMap* map, const int8_t* p, int64_t rows, int64_t K, int64_t ld, uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {(cuuint32_t)BK, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG>
cudaError_t launch_tiles(const I8GemmArgs& g, int bn, int num_sms, cudaStream_t stream) {
  using C = Cfg<CG>;
  const int64_t mb = (g.M + BM * CG - 1) / (BM * CG), nb = (g.N + bn - 1) / bn;
  if (mb * nb > INT32_MAX) return cudaErrorNotSupported;    // 32-bit tile numbers
  CUtensorMap tmA, tmB;
  if (!encode_i8_map(&tmA, g.a, g.M, g.K, g.lda, BM) ||
      !encode_i8_map(&tmB, g.w, g.N, g.K, g.ldw, (uint32_t)(bn / CG)))
    return cudaErrorInvalidValue;
  Params p{};
  p.a_scales = g.a_scales; p.w_scales = g.w_scales; p.bias = g.bias;
  p.y = g.y; p.ldy = g.ldy;
  const size_t esize = g.y_bf16 ? 2 : 4;
  p.y_vec = reinterpret_cast<uintptr_t>(g.y) % 16 == 0 && ((size_t)g.ldy * esize) % 16 == 0;
  p.M = (int)g.M; p.N = (int)g.N; p.K = (int)g.K; p.bn = bn;
  p.m_blocks = (int)mb; p.num_tiles = (int)(mb * nb); p.k_tiles = (int)((g.K + BK - 1) / BK);
  p.st = g.st;
  const WaitTest wt = wait_test();
  p.wait_ns = wt.limit_ns; p.hold = wt.hold;
  auto kern = g.y_bf16 ? k_i8_gemm<CG, true> : k_i8_gemm<CG, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(CG * std::max(1, std::min(p.num_tiles, num_sms / CG))));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CG; at[1].val.clusterDim.y = 1; at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tmA, tmB, p);
}

}  // namespace

cudaError_t launch_i8_gemm(const I8GemmArgs& g, int num_sms, cudaStream_t stream) {
  return g.M > BM ? launch_tiles<2>(g, 256, num_sms, stream) : launch_tiles<1>(g, 128, num_sms, stream);
}

}  // namespace nvfp4
