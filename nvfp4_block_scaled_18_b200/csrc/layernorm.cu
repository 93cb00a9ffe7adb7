// Layer norm (forward, backward) and the 8-bit quantizer of rows, sm_100a.
//
// Forward, one row x of K elements (every fp32 step rounded once):
//   mean = fl32(sum x / K)                      sum in binary64
//   rstd = fl32(1 / sqrt(sum d^2 / K + eps))    d = fl32(x - mean), sum in binary64
//   y    = ((d * rstd) * gamma) + beta
// 8-bit codes of a row v: amax = max |v|, scale = amax / 127,
//   code = rint(v * (127 / amax)).
// The sums are formed in binary64 so that mean and rstd do not depend on the
// order of summation (but for one in about 2^28 rows), and with them the codes.
#include <algorithm>

#include "kernels.h"
#include "rows.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {
using namespace rows;
namespace {

struct RowArgs {
  const void* x; int64_t ldx;
  const void* gamma; const void* beta;   // either may be null
  float eps;
  void* y; int64_t ldy;                  // !QUANT
  float* mean; float* rstd;              // !QUANT, may be null
  int8_t* codes; int64_t ldc; float* scales;   // QUANT
  int64_t M;
  int units;                             // K / 8
  int warps;                             // warps per row
  int* st;
};

template <typename P>
__device__ __forceinline__ void affine8(float (&v)[8], const P* gamma, const P* beta, int64_t at) {
  float t[8];
  if (gamma != nullptr) {
    fetch8(gamma + at, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], t[i]);
  }
  if (beta != nullptr) {
    fetch8(beta + at, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(v[i], t[i]);
  }
}

// A team of warps per row; the row's units are held in registers, V per thread.
// Rows longer than that go through in several chunks: each pass then reads
// them again, the last chunk first (it is still in registers).
template <typename T, typename P, bool NORM, bool QUANT, int V>
__global__ void __launch_bounds__(1024) k_rows(const RowArgs a) {
  __shared__ double red_sum[2][kMaxWarps];
  __shared__ uint32_t red_max[2][kMaxWarps];
  Team team;
  team.warps = a.warps;
  team.index = (threadIdx.x >> 5) / a.warps;
  team.warp = (threadIdx.x >> 5) - team.index * a.warps;
  team.lane = threadIdx.x & 31;
  const int teams = (blockDim.x >> 5) / a.warps;
  const int base = team.index * a.warps;
  const int t = team.warp * 32 + team.lane, span = a.warps * 32;
  const int chunks = (a.units + span * V - 1) / (span * V);
  const double inv_k = 1.0 / (8.0 * (double)a.units);

  tc::griddep_launch_dependents();
  tc::griddep_wait();
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * teams + team.index; row < a.M; row += (int64_t)gridDim.x * teams, turn ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    float v[V][8];
    auto load = [&](int c) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int u = (c * V + i) * span + t;
        if (u < a.units) {
          fetch8(x + (int64_t)u * 8, v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
      }
    };
    float mean = 0.0f, rstd = 1.0f;
    if constexpr (NORM) {
      double s = 0.0;
      for (int c = 0; c < chunks; ++c) {
        load(c);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) s += (double)v[i][e];
      }
      mean = (float)(team.sum(s, red_sum[0] + base) * inv_k);
      double q = 0.0;
      for (int c = chunks - 1; c >= 0; --c) {
        if (c != chunks - 1) load(c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if ((c * V + i) * span + t >= a.units) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const double d = (double)__fsub_rn(v[i][e], mean);
            q = fma(d, d, q);
          }
        }
      }
      rstd = (float)(1.0 / sqrt(team.sum(q, red_sum[1] + base) * inv_k + (double)a.eps));
      if (t == 0 && !(abs_key(mean) < 0x7F800000u && abs_key(rstd) < 0x7F800000u)) report_status(a.st, NVFP4_ERR_NONFINITE);
    }
    // the row's result before its last rounding: v holds chunk c
    auto finish = [&](int c) {
      if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int u = (c * V + i) * span + t;
          if (u >= a.units) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = __fmul_rn(__fsub_rn(v[i][e], mean), rstd);
          affine8(v[i], static_cast<const P*>(a.gamma), static_cast<const P*>(a.beta), (int64_t)u * 8);
        }
      }
    };
    // after the statistics pass chunk 0 is in registers; without one, nothing is
    if constexpr (!QUANT) {
      T* y = static_cast<T*>(a.y) + row * a.ldy;
      for (int c = 0; c < chunks; ++c) {
        if (c != 0) load(c);
        finish(c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int u = (c * V + i) * span + t;
          if (u < a.units) store8(y + (int64_t)u * 8, v[i]);
        }
      }
      if (t == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
    } else {
      uint32_t m = 0;
      for (int c = 0; c < chunks; ++c) {
        if (!NORM || c != 0) load(c);
        finish(c);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((c * V + i) * span + t < a.units) m = max(m, abs_key(v[i][e]));
      }
      m = team.max(m, red_max[turn] + base);
      const RowScale rs = row_scale(m);
      if (t == 0) {
        a.scales[row] = rs.scale;
        if (m >= 0x7F800000u) report_status(a.st, NVFP4_ERR_NONFINITE);
      }
      int8_t* codes = a.codes + row * a.ldc;
      const bool zero = rs.inv == 0.0f;
      for (int c = chunks - 1; c >= 0; --c) {
        if (c != chunks - 1) {
          load(c);
          finish(c);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int u = (c * V + i) * span + t;
          if (u < a.units)
            *reinterpret_cast<uint2*>(codes + (int64_t)u * 8) = zero ? make_uint2(0u, 0u) : encode8(v[i], rs.inv);
        }
      }
    }
  }
}

template <typename T, typename P, bool NORM, bool QUANT, int V>
cudaError_t run_rows(const RowArgs& a, int threads, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_rows<T, P, NORM, QUANT, V>, a);
}

template <typename T, typename P, bool NORM, bool QUANT>
cudaError_t launch_rows(RowArgs a, int num_sms, cudaStream_t stream) {
  // few rows: one unit per thread, for latency; many: up to four, for bytes in flight per instruction
  const int v = a.M <= num_sms ? 1 : (a.units > 1024 ? 4 : 2);
  a.warps = std::min(kMaxWarps, (a.units + 32 * v - 1) / (32 * v));
  const int teams = std::max(1, std::min({kMaxTeams, 8 / a.warps, kMaxWarps / a.warps}));
  const int64_t groups = (a.M + teams - 1) / teams;
  const int grid = (int)std::min<int64_t>(groups, (int64_t)1 << 30);
  const int threads = 32 * a.warps * teams;
  if (v == 1) return run_rows<T, P, NORM, QUANT, 1>(a, threads, grid, stream);
  if (v == 2) return run_rows<T, P, NORM, QUANT, 2>(a, threads, grid, stream);
  return run_rows<T, P, NORM, QUANT, 4>(a, threads, grid, stream);
}

template <bool NORM, bool QUANT>
cudaError_t launch_rows_typed(const RowArgs& a, nvfp4_dtype dt, nvfp4_dtype pdt, int num_sms, cudaStream_t stream) {
  if (!NORM || pdt == dt)   // without a norm there are no parameters
    return dt == NVFP4_BF16 ? launch_rows<__nv_bfloat16, __nv_bfloat16, NORM, QUANT>(a, num_sms, stream)
                            : launch_rows<float, float, NORM, QUANT>(a, num_sms, stream);
  if constexpr (NORM)
    return dt == NVFP4_BF16 ? launch_rows<__nv_bfloat16, float, NORM, QUANT>(a, num_sms, stream)
                            : launch_rows<float, __nv_bfloat16, NORM, QUANT>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------- backward
// One row, with xh = (x - mean) * rstd and g = dy * gamma:
//   dx = rstd * (g - mean(g) - xh * mean(g * xh))
// and, over all rows, dgamma = sum dy * xh, dbeta = sum dy.
// A CTA takes the rows blockIdx.x, blockIdx.x + grid, ...; its threads keep the
// running dgamma and dbeta of their own columns in registers and write them once,
// as one row of the workspace.  k_ln_params then sums the grid's rows in a fixed
// order, so results do not change from run to run.
struct BwdArgs {
  const void* dy; int64_t lddy;
  const void* x; int64_t ldx;
  const void* gamma;                 // may be null
  const float* mean; const float* rstd;
  void* dx; int64_t lddx;            // may be null
  float* part;                       // grid x 2 x K partial sums, or null
  int64_t M;
  int units;
};

__device__ __forceinline__ float2 cta_sum2(float2 v, float2* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
  }
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (l == 0) slot[w] = v;
  __syncthreads();
  v = l < nw ? slot[l] : make_float2(0.0f, 0.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
  }
  return v;
}

// The rows' units beyond blockDim.x * V are taken in further column chunks
// (blockIdx.y), each of which forms the row sums over the whole row again.
template <typename T, typename P, int V>
__global__ void __launch_bounds__(512) k_ln_backward(const BwdArgs a) {
  __shared__ float2 red[2][kMaxWarps];
  const int nt = blockDim.x, t = threadIdx.x;
  const int first = blockIdx.y * nt * V;       // this CTA's own columns
  const float inv_k = 1.0f / (8.0f * (float)a.units);
  float dg[V][8], db[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = db[i][e] = 0.0f;
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float xh[V][8], g[V][8];
    float2 s = make_float2(0.0f, 0.0f);
    auto unit = [&](int u, float (&xv)[8], float (&gv)[8], float (&dyv)[8]) {
      fetch8(x + (int64_t)u * 8, xv);
      fetch8(dy + (int64_t)u * 8, dyv);
      float gm[8];
      if (a.gamma != nullptr) fetch8(static_cast<const P*>(a.gamma) + (int64_t)u * 8, gm);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xv[e] = (xv[e] - mean) * rstd;
        gv[e] = a.gamma != nullptr ? dyv[e] * gm[e] : dyv[e];
        s.x += gv[e];
        s.y = fmaf(gv[e], xv[e], s.y);
      }
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = first + i * nt + t;
      if (u < a.units) {
        float dyv[8];
        unit(u, xh[i], g[i], dyv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dg[i][e] = fmaf(dyv[e], xh[i][e], dg[i][e]);
          db[i][e] += dyv[e];
        }
      }
    }
    if (a.dx == nullptr) continue;
    for (int u = t; u < a.units; u += nt) {       // the other chunks' share of the row sums
      if (u >= first && u < first + nt * V) continue;
      float xv[8], gv[8], dyv[8];
      unit(u, xv, gv, dyv);
    }
    s = cta_sum2(s, red[turn]);
    const float c1 = s.x * inv_k, c2 = s.y * inv_k;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = first + i * nt + t;
      if (u < a.units) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rstd * (g[i][e] - fmaf(xh[i][e], c2, c1));
        store8(dx + (int64_t)u * 8, o);
      }
    }
  }
  if (a.part == nullptr) return;
  float* pg = a.part + (int64_t)blockIdx.x * 16 * a.units;
  float* pb = pg + (int64_t)8 * a.units;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int u = first + i * nt + t;
    if (u < a.units) {
      store8(pg + (int64_t)u * 8, dg[i]);
      store8(pb + (int64_t)u * 8, db[i]);
    }
  }
}

// dgamma / dbeta = sum over the workspace's rows: 32 columns per CTA, one warp
// per group of rows, joined in shared memory in the order of the warps.
__global__ void __launch_bounds__(256) k_ln_params(const float* part, int parts, int64_t K, float* dgamma,
                                                   float* dbeta) {
  __shared__ float red[8][33];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + l;   // column of [dgamma | dbeta]
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  float s = 0.0f;
  if (c < 2 * K)
    for (int r = w; r < parts; r += 8) s += part[(int64_t)r * 2 * K + c];
  red[w][l] = s;
  __syncthreads();
  if (w == 0 && c < 2 * K) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][l];
    float* out = c < K ? dgamma : dbeta;
    if (out != nullptr) out[c < K ? c : c - K] = s;
  }
}

template <typename T, typename P>
cudaError_t run_backward(const BwdArgs& a, dim3 grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ln_backward<T, P, 2>, a);
}

}  // namespace

cudaError_t launch_i8_quant(const void* x, nvfp4_dtype dt, int64_t M, int64_t K, int64_t ldx, int8_t* codes,
                            int64_t ldc, float* scales, int* st, int num_sms, cudaStream_t stream) {
  RowArgs a{};
  a.x = x; a.ldx = ldx; a.codes = codes; a.ldc = ldc; a.scales = scales;
  a.M = M; a.units = (int)(K / 8); a.st = st;
  return launch_rows_typed<false, true>(a, dt, dt, num_sms, stream);
}

cudaError_t launch_layernorm(const LayerNormArgs& n, int num_sms, cudaStream_t stream) {
  RowArgs a{};
  a.x = n.x; a.ldx = n.ldx; a.gamma = n.gamma; a.beta = n.beta; a.eps = n.eps;
  a.y = n.y; a.ldy = n.ldy; a.mean = n.mean; a.rstd = n.rstd;
  a.codes = n.codes; a.ldc = n.ldc; a.scales = n.scales;
  a.M = n.M; a.units = (int)(n.K / 8); a.st = n.st;
  return n.codes != nullptr ? launch_rows_typed<true, true>(a, n.dt, n.pdt, num_sms, stream)
                            : launch_rows_typed<true, false>(a, n.dt, n.pdt, num_sms, stream);
}

int layernorm_parts(int64_t M) { return (int)std::min<int64_t>(M, kLnMaxParts); }

cudaError_t launch_layernorm_backward(const LayerNormBwdArgs& n, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  BwdArgs a{};
  a.dy = n.dy; a.lddy = n.lddy; a.x = n.x; a.ldx = n.ldx; a.gamma = n.gamma;
  a.mean = n.mean; a.rstd = n.rstd; a.dx = n.dx; a.lddx = n.lddx;
  const bool params = n.dgamma != nullptr || n.dbeta != nullptr;
  a.part = params ? n.part : nullptr;
  a.M = n.M; a.units = (int)(n.K / 8);
  const int parts = layernorm_parts(n.M);
  const int threads = std::min(512, (a.units + 63) / 64 * 32);
  const dim3 grid((unsigned)parts, (unsigned)((a.units + 2 * threads - 1) / (2 * threads)));
  cudaError_t e;
  if (n.dt == NVFP4_BF16)
    e = n.pdt == NVFP4_BF16 ? run_backward<__nv_bfloat16, __nv_bfloat16>(a, grid, threads, stream)
                            : run_backward<__nv_bfloat16, float>(a, grid, threads, stream);
  else
    e = n.pdt == NVFP4_BF16 ? run_backward<float, __nv_bfloat16>(a, grid, threads, stream)
                            : run_backward<float, float>(a, grid, threads, stream);
  if (e != cudaSuccess || !params) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((2 * n.K + 31) / 32));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ln_params, (const float*)a.part, parts, n.K, n.dgamma, n.dbeta);
}

}  // namespace nvfp4
