// 8-bit integer linear for one to four tokens on the CUDA cores, sm_100a.
//
// A warp takes four rows of W (columns of Y) for one token, eight for more: each
// lane reads 16 bytes of each row and of each token at a time and multiplies them
// with dp4a, so W is streamed once with wide loads and the tokens come from L1.
// When there are too few rows to fill the SMs, the S warps of a group split K;
// the int32 sums are joined in shared memory, exactly.  Bound: W's bytes (1 x
// 14336 x 4096: 11.1 us, 5.3 TB/s; 4 x 14336 x 4096: 11.9, with four rows a warp
// 17.4).
//
// Programmatic dependent launch: before griddepcontrol.wait a warp only asks L2
// to prefetch its first W bytes.
#include <algorithm>

#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4 {
using namespace tc;
namespace {

constexpr int WARPS = 8;       // per CTA
// rows of W per warp: with more tokens each of their loads has to serve more rows
template <int MT> constexpr int rows_per_warp() { return MT == 1 ? 4 : 8; }

struct Params {
  const int8_t* a; int64_t lda; const float* a_scales;
  const int8_t* w; int64_t ldw; const float* w_scales;
  const float* bias;
  void* y; int64_t ldy;
  int M, N, K;
  int split;                   // S: warps that share their rows, 1, 2, 4 or 8
};

// W passes once: past L1
__device__ __forceinline__ uint4 load_w(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
  c = __dp4a((int)a.x, (int)b.x, c);
  c = __dp4a((int)a.y, (int)b.y, c);
  c = __dp4a((int)a.z, (int)b.z, c);
  return __dp4a((int)a.w, (int)b.w, c);
}

template <int MT, bool BF16OUT>
__global__ void __launch_bounds__(WARPS * 32) k_i8_gemv(const Params p) {
  constexpr int ROWS = rows_per_warp<MT>();
  constexpr int UNROLL = MT == 1 ? 4 : MT == 2 ? 2 : 1;
  __shared__ int joined[WARPS][ROWS * MT];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = WARPS / p.split, part = warp % p.split;
  const int64_t run = (int64_t)blockIdx.x * groups + warp / p.split;
  const int n0 = (int)(run * ROWS);
  // this warp's share of K in units of 16 bytes, 32 to a step
  const int units = p.K / 16, steps = (units + 31) / 32;
  const int t0 = (int)((int64_t)part * steps / p.split), t1 = (int)((int64_t)(part + 1) * steps / p.split);
  const bool active = n0 < p.N;
  const int8_t* wr[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) wr[r] = p.w + (int64_t)min(n0 + r, p.N - 1) * p.ldw + lane * 16;   // rows past N repeat the last
  if (active) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < UNROLL; ++i)
        if ((t0 + i) * 32 + lane < units) asm volatile("prefetch.global.L2 [%0];" ::"l"(wr[r] + (int64_t)(t0 + i) * 512));
  }
  griddep_wait();
  int acc[ROWS][MT];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0;
  if (active) {
    const int8_t* ar = p.a + lane * 16;
    int t = t0;
    for (; t + UNROLL <= t1 && (t + UNROLL) * 32 <= units; t += UNROLL) {
      uint4 w[UNROLL][ROWS];
#pragma unroll
      for (int i = 0; i < UNROLL; ++i)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) w[i][r] = load_w(wr[r] + (int64_t)(t + i) * 512);
#pragma unroll
      for (int i = 0; i < UNROLL; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 x = *reinterpret_cast<const uint4*>(ar + (int64_t)min(m, p.M - 1) * p.lda + (int64_t)(t + i) * 512);
#pragma unroll
          for (int r = 0; r < ROWS; ++r) acc[r][m] = dot16(w[i][r], x, acc[r][m]);
        }
    }
    for (; t < t1; ++t) {
      if (t * 32 + lane >= units) continue;
      uint4 w[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) w[r] = load_w(wr[r] + (int64_t)t * 512);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint4 x = *reinterpret_cast<const uint4*>(ar + (int64_t)min(m, p.M - 1) * p.lda + (int64_t)t * 512);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) acc[r][m] = dot16(w[r], x, acc[r][m]);
      }
    }
  }
  // lane r * MT + m holds the warp's sum of row r, token m
  constexpr int VALUES = (ROWS * MT + 31) / 32;     // per lane
  int mine[VALUES] = {};
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int s = __reduce_add_sync(0xFFFFFFFFu, acc[r][m]);
      if (lane == (r * MT + m) % 32) mine[(r * MT + m) / 32] = s;
    }
  if (p.split > 1) {
#pragma unroll
    for (int v = 0; v < VALUES; ++v)
      if (v * 32 + lane < ROWS * MT) joined[warp][v * 32 + lane] = mine[v];
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int v = 0; v < VALUES; ++v)
      if (v * 32 + lane < ROWS * MT)
        for (int s = 1; s < p.split; ++s) mine[v] += joined[warp + s][v * 32 + lane];
  }
#pragma unroll
  for (int v = 0; v < VALUES; ++v) {
    const int i = v * 32 + lane, n = n0 + i / MT, m = i % MT;
    if (active && i < ROWS * MT && n < p.N && m < p.M) {
      float o = __fmul_rn(__fmul_rn(__int2float_rn(mine[v]), p.a_scales[m]), p.w_scales[n]);
      if (p.bias != nullptr) o = __fadd_rn(o, p.bias[n]);
      if (BF16OUT) reinterpret_cast<__nv_bfloat16*>(p.y)[(int64_t)m * p.ldy + n] = __float2bfloat16_rn(o);
      else reinterpret_cast<float*>(p.y)[(int64_t)m * p.ldy + n] = o;
    }
  }
}

template <int MT>
cudaError_t launch_mt(const I8GemmArgs& g, int num_sms, cudaStream_t stream) {
  Params p{};
  p.a = g.a; p.lda = g.lda; p.a_scales = g.a_scales; p.w = g.w; p.ldw = g.ldw; p.w_scales = g.w_scales;
  p.bias = g.bias; p.y = g.y; p.ldy = g.ldy; p.M = (int)g.M; p.N = (int)g.N; p.K = (int)g.K;
  constexpr int ROWS = rows_per_warp<MT>();
  const int64_t runs = (g.N + ROWS - 1) / ROWS, steps = (g.K / 16 + 31) / 32;
  // split K until there are this many warps for every SM, each with two steps or more
  constexpr int want = MT == 1 ? 16 : 8;
  p.split = 1;
  while (p.split < WARPS && runs * p.split < (int64_t)want * num_sms && steps >= 4 * p.split) p.split *= 2;
  const int64_t grid = (runs * p.split + WARPS - 1) / WARPS;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, g.y_bf16 ? k_i8_gemv<MT, true> : k_i8_gemv<MT, false>, p);
}

}  // namespace

cudaError_t launch_i8_gemv(const I8GemmArgs& g, int num_sms, cudaStream_t stream) {
  if (g.M > 4) return cudaErrorNotSupported;
  if (g.M == 1) return launch_mt<1>(g, num_sms, stream);
  if (g.M == 2) return launch_mt<2>(g, num_sms, stream);
  return launch_mt<4>(g, num_sms, stream);
}

}  // namespace nvfp4
