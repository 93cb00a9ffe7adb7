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
#include "i8_plan.h"
#include "i8_tc.cuh"

namespace nvfp4 {
using namespace rows;
namespace {

// Threads of a CTA at most, by the registers that v units per thread take.
constexpr int max_threads(int v) { return v <= 2 ? 1024 : v == 4 ? 640 : 512; }

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

// A team of W warps per row; the row's units are held in registers, V per thread.
// FULL: every thread has V units.
// ONE: a row fits (units <= W * 32 * V).  The team then takes row after row, and
// loads the next one before it works on the present one.  Otherwise rows go
// through in several chunks, and each pass reads them again, the last chunk
// first (it is still in registers).
//
// Bound: the quantizer alone by its bytes (8192 x 14336 bf16: 54 us, 6.6 TB/s).
// With the norm, by instruction issue, 19 instructions per element: of 37 us for
// 8192 x 4096 bf16 with fp32 parameters the row's two reductions take 9, the gain
// and the bias 10 and binary64 3 (2048 x 4096 into 8 bits: 12 us).  Tried and not
// kept: two rows per team (41 us), and sums in fp32, whose codes would depend on
// the order.
template <typename T, typename P, bool NORM, bool QUANT, int V, bool ONE, bool FULL>
__global__ void __launch_bounds__(ONE ? max_threads(V) : 1024) k_rows(const RowArgs a) {
  using Raw = Unit<T>;
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
  const int chunks = ONE ? 1 : (a.units + span * V - 1) / (span * V);
  const double inv_k = 1.0 / (8.0 * (double)a.units);
  const int64_t stride = (int64_t)gridDim.x * teams;

  tc::griddep_launch_dependents();
  tc::griddep_wait();
  int turn = 0;
  Raw next[ONE ? V : 1];
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (FULL || i * span + t < a.units) next[i].load(x, i * span + t, a.units);
      else next[i].zero();
    }
  };
  int64_t row = (int64_t)blockIdx.x * teams + team.index;
  if constexpr (ONE) {
    if (row < a.M) fetch(row);
  }
  for (; row < a.M; row += stride, turn ^= 1) {
    float v[V][8];
    auto load = [&](int c) {
      const T* x = static_cast<const T*>(a.x) + row * a.ldx;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int u = (c * V + i) * span + t;
        Raw w;
        if (FULL || u < a.units) w.load(x, u, a.units);
        else w.zero();
        w.unpack(v[i]);
      }
    };
    if constexpr (ONE) {
#pragma unroll
      for (int i = 0; i < V; ++i) next[i].unpack(v[i]);
      if (row + stride < a.M) fetch(row + stride);
    }
    float mean = 0.0f, rstd = 1.0f;
    auto centre = [&](int c) {     // v = x - mean; zeros stay beyond the row's end
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!FULL && (c * V + i) * span + t >= a.units) continue;
#pragma unroll
        for (int e = 0; e < 8; e += 2) add2(v[i][e], v[i][e + 1], -mean, -mean);
      }
    };
    if constexpr (NORM) {
      double s0 = 0.0, s1 = 0.0;                  // two chains
      for (int c = 0; c < chunks; ++c) {
        if (!ONE) load(c);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            s0 += (double)v[i][e];
            s1 += (double)v[i][e + 1];
          }
      }
      mean = (float)(team.sum(s0 + s1, red_sum[0] + base) * inv_k);
      s0 = s1 = 0.0;
      for (int c = chunks - 1; c >= 0; --c) {
        if (c != chunks - 1) load(c);
        centre(c);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const double d0 = (double)v[i][e], d1 = (double)v[i][e + 1];
            s0 = fma(d0, d0, s0);
            s1 = fma(d1, d1, s1);
          }
      }
      rstd = rsqrt_rounded(team.sum(s0 + s1, red_sum[1] + base) * inv_k + (double)a.eps);
      if (t == 0 && !has_norm(mean, rstd)) report_status(a.st, NVFP4_ERR_NONFINITE);
    }
    // the row's result before its last rounding; v holds chunk c, as x - mean
    auto finish = [&](int c) {
      if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int u = (c * V + i) * span + t;
          if (!FULL && u >= a.units) continue;
          float p[8];
#pragma unroll
          for (int e = 0; e < 8; e += 2) mul2(v[i][e], v[i][e + 1], rstd, rstd);
          if (a.gamma != nullptr) {
            Raw::param(static_cast<const P*>(a.gamma), u, a.units, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = __fmul_rn(v[i][e], p[e]);
          }
          if (a.beta != nullptr) {
            Raw::param(static_cast<const P*>(a.beta), u, a.units, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = __fadd_rn(v[i][e], p[e]);
          }
        }
      }
    };
    auto reload = [&](int c) {
      load(c);
      if constexpr (NORM) centre(c);
    };
    // after the statistics pass chunk 0 is in registers; without one (and not ONE), nothing is
    if constexpr (!QUANT) {
      T* y = static_cast<T*>(a.y) + row * a.ldy;
      for (int c = 0; c < chunks; ++c) {
        if (c != 0) reload(c);
        finish(c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int u = (c * V + i) * span + t;
          if (FULL || u < a.units) Raw::store(y, u, a.units, v[i]);
        }
      }
      if (t == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
    } else {
      float top = 0.0f;
      for (int c = 0; c < chunks; ++c) {
        if ((!NORM && !ONE) || c != 0) reload(c);
        finish(c);                 // what lies beyond the row's end is zero
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; e += 2) top = max3_abs(top, v[i][e], v[i][e + 1]);
      }
      const uint32_t m = team.max(abs_key(top), red_max[turn] + base);
      const RowScale rs = row_scale(m);
      if (t == 0) {
        a.scales[row] = rs.scale;
        if (m >= 0x7F800000u) report_status(a.st, NVFP4_ERR_NONFINITE);
      }
      int8_t* codes = a.codes + row * a.ldc;
      const bool zero = rs.inv == 0.0f;
      for (int c = chunks - 1; c >= 0; --c) {
        if (c != chunks - 1) {
          reload(c);
          finish(c);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int u = (c * V + i) * span + t;
          if (FULL || u < a.units) Raw::store_codes(codes, u, a.units, zero ? make_uint2(0u, 0u) : encode8(v[i], rs.inv));
        }
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void copies_left() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Layer norm of many long rows: the steps of k_rows with fewer warps per row (two
// for 4096 elements), since a row's reductions cost every one of its warps some
// hundred instructions and a barrier.  A thread holds V units as they are in
// memory and unpacks them for each pass; the next row arrives meanwhile in the
// thread's own part of shared memory (cp.async: it waits for its own copies
// alone).  Gain and bias are in shared memory as fp32, laid out for loads of whole
// lines.  Bound: instruction issue and the conversions to binary64 still (8192 x
// 4096 bf16 with fp32 parameters: 31 us, its bytes 20.5; 8192 x 8192: 57 and 41;
// 4096 x 4096 fp32: 25 and 20.5).  Sixteen units a thread, one warp a row, spill:
// 58 us.
constexpr int kNormThreads = 512, kNormSmem = 224 * 1024;

template <typename T, typename P, bool QUANT, int V, bool FULL>
__global__ void __launch_bounds__(kNormThreads, 1) k_norm_rows(const RowArgs a) {
  using U = Unit<T>;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  float* gain = reinterpret_cast<float*>(norm_smem);     // elements 0-3 of every unit, then 4-7
  float* bias = gain + a.units * 8;
  __shared__ double red_sum[2][kNormThreads / 32];
  __shared__ uint32_t red_max[2][kNormThreads / 32];
  const int warps = a.warps, index = (threadIdx.x >> 5) / warps, lane = threadIdx.x & 31;
  const int warp = (threadIdx.x >> 5) - index * warps;
  const int teams = (blockDim.x >> 5) / warps, base = index * warps, span = warps * 32, t = warp * 32 + lane;
  const uint32_t row_bytes = (uint32_t)a.units * 8u * (uint32_t)sizeof(T);
  const uint8_t* stage = norm_smem + (uint32_t)a.units * 64u + (uint32_t)index * row_bytes;
  const int64_t stride = (int64_t)gridDim.x * teams, first = (int64_t)blockIdx.x * teams + index;
  const double inv_k = 1.0 / (8.0 * (double)a.units);
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  auto issue = [&](int64_t row) {
    if (row < a.M) {
      const uint8_t* x = reinterpret_cast<const uint8_t*>(static_cast<const T*>(a.x) + row * a.ldx);
      const uint32_t dst = tc::saddr(stage);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int u = i * span + t;
        if (!FULL && u >= a.units) continue;
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
          const uint32_t off = (uint32_t)(u + h * a.units) * 16u;
          copy16(dst + off, x + off);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  issue(first);
  for (int u = threadIdx.x; u < a.units; u += blockDim.x) {
    float g[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f}, b[8] = {};
    if (a.gamma != nullptr) U::param(static_cast<const P*>(a.gamma), u, a.units, g);
    if (a.beta != nullptr) U::param(static_cast<const P*>(a.beta), u, a.units, b);
    Unit<float>::store(gain, u, a.units, g);
    Unit<float>::store(bias, u, a.units, b);
  }
  __syncthreads();
  auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(span) : "memory"); };
  auto total = [&](double x, double* slot) {
    x = warp_sum_f64(x);
    if (warps == 1) return x;
    if (lane == 0) slot[warp] = x;
    sync();
    x = slot[0];
    for (int w = 1; w < warps; ++w) x += slot[w];
    return x;
  };
  int turn = 0;
  for (int64_t row = first; row < a.M; row += stride, turn ^= 1) {
    copies_left<0>();
    U held[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = i * span + t;
      if (FULL || u < a.units) held[i].load(reinterpret_cast<const T*>(stage), u, a.units);
      else held[i].zero();
    }
    double s[4] = {0.0, 0.0, 0.0, 0.0};                   // chains
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v[8];
      held[i].unpack(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e & 3] += (double)v[e];
    }
    issue(row + stride);                                  // the row has been read
    const float mean = (float)(total((s[0] + s[1]) + (s[2] + s[3]), red_sum[0] + base) * inv_k);
    s[0] = s[1] = s[2] = s[3] = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      held[i].forget();
      if (!FULL && i * span + t >= a.units) continue;
      float v[8];
      held[i].unpack(v);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        add2(v[e], v[e + 1], -mean, -mean);
        const double d0 = (double)v[e], d1 = (double)v[e + 1];
        s[e & 3] = fma(d0, d0, s[e & 3]);
        s[(e + 1) & 3] = fma(d1, d1, s[(e + 1) & 3]);
      }
    }
    const float rstd =
        rsqrt_rounded(total((s[0] + s[1]) + (s[2] + s[3]), red_sum[1] + base) * inv_k + (double)a.eps);
    if (t == 0 && !has_norm(mean, rstd)) report_status(a.st, NVFP4_ERR_NONFINITE);
    auto result = [&](int i, float (&v)[8]) {             // before its last rounding
      const int u = i * span + t;
      float p[8];
      held[i].forget();
      held[i].unpack(v);
      Unit<float>::param(gain, u, a.units, p);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        add2(v[e], v[e + 1], -mean, -mean);
        mul2(v[e], v[e + 1], rstd, rstd);
        v[e] = __fmul_rn(v[e], p[e]);
        v[e + 1] = __fmul_rn(v[e + 1], p[e + 1]);
      }
      Unit<float>::param(bias, u, a.units, p);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(v[e], p[e]);
    };
    if constexpr (!QUANT) {
      T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!FULL && i * span + t >= a.units) continue;
        float v[8];
        result(i, v);
        U::store(y, i * span + t, a.units, v);
      }
      if (t == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
    } else {
      float top = 0.0f, v[V][8];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!FULL && i * span + t >= a.units) continue;
        result(i, v[i]);
#pragma unroll
        for (int e = 0; e < 8; e += 2) top = max3_abs(top, v[i][e], v[i][e + 1]);
      }
      uint32_t m = __reduce_max_sync(0xFFFFFFFFu, abs_key(top));
      if (warps > 1) {
        if (lane == 0) red_max[turn][base + warp] = m;
        sync();
        m = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? red_max[turn][base + lane] : 0u);
      }
      const RowScale rs = row_scale(m);
      if (t == 0) {
        a.scales[row] = rs.scale;
        if (m >= 0x7F800000u) report_status(a.st, NVFP4_ERR_NONFINITE);
      }
      int8_t* codes = a.codes + row * a.ldc;
      const bool zero = rs.inv == 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!FULL && i * span + t >= a.units) continue;
        U::store_codes(codes, i * span + t, a.units, zero ? make_uint2(0u, 0u) : encode8(v[i], rs.inv));
      }
    }
  }
  copies_left<0>();
}

cudaLaunchConfig_t dependent_launch(dim3 grid, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute* at) {
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T, typename P, bool NORM, bool QUANT, int V, bool ONE, bool FULL = false>
cudaError_t run_rows(RowArgs a, int num_sms, cudaStream_t stream) {
  if constexpr (ONE && !FULL)
    if (a.units % (32 * V) == 0) return run_rows<T, P, NORM, QUANT, V, ONE, true>(a, num_sms, stream);
  auto kern = k_rows<T, P, NORM, QUANT, V, ONE, FULL>;
  a.warps = ONE ? (a.units + 32 * V - 1) / (32 * V) : 32;
  const int teams = std::max(1, 4 / a.warps), threads = 32 * a.warps * teams;
  const int64_t groups = (a.M + teams - 1) / teams;
  // persistent when rows fit: as many CTAs as are resident at once, by registers
  // (8192 x 4096 bf16 with 1.6 waves of them instead: 43 us, 37 so)
  static std::atomic<int> known;
  const int regs = i8::asked_once(&known, 128, [&] {
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, kern) == cudaSuccess) return fa.numRegs;
    (void)cudaGetLastError();
    return -1;
  });
  const int ctas = std::max(1, std::min(2048 / threads, 65536 / ((regs + 7) / 8 * 8 * threads)));
  const int64_t grid = std::min<int64_t>(groups, ONE ? (int64_t)num_sms * ctas : (int64_t)1 << 30);
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = dependent_launch(dim3((unsigned)grid), threads, 0, stream, &at);
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, typename P, bool QUANT, int V, bool FULL>
cudaError_t run_norm_rows(RowArgs a, int num_sms, cudaStream_t stream) {
  a.warps = (a.units + 32 * V - 1) / (32 * V);
  if (a.warps > kNormThreads / 32) return cudaErrorNotSupported;
  const int64_t row = (int64_t)a.units * 8 * (int64_t)sizeof(T), params = (int64_t)a.units * 64;
  const int teams = (int)std::min<int64_t>({kNormThreads / 32 / a.warps, a.warps == 1 ? 16 : 15, (kNormSmem - params) / row});
  if (teams < 1) return cudaErrorNotSupported;
  static tc::SmemOnce once;
  const cudaError_t e = once.set(k_norm_rows<T, P, QUANT, V, FULL>, kNormSmem);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>((a.M + teams - 1) / teams, num_sms);
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg =
      dependent_launch(dim3((unsigned)grid), 32 * a.warps * teams, (size_t)(params + teams * row), stream, &at);
  return cudaLaunchKernelEx(&cfg, k_norm_rows<T, P, QUANT, V, FULL>, a);
}

// Ten or five units per thread if that leaves none idle and eight does not.  Where
// none of them fills the warps, the checks of the row's end cost registers (76 bytes
// spilled, 272 into 8 bits), and k_rows is the faster one (4096 rows of 9216 bf16: 46
// us, 55 here, into 8 bits 52 and 74; of 13824 fp32 into 8 bits 111 and 125), except
// for fp32 rows (11008: 101, 65 here), for bf16 rows with fp32 parameters that take
// four warps and more (7168: 52 and 39; 5632: 30 and 34), and into 8 bits where four
// warps a row fill the CTA (4096 rows of 7168 fp32: 67 and 58; 1500 of 6656: 28 and
// 25.3; not so just past a wave of 592 rows: 600 of 7168 15 and 19).
template <typename T, typename P, bool QUANT>
cudaError_t launch_norm_rows(const RowArgs& a, int num_sms, cudaStream_t stream) {
  if (a.units % 256 == 0) return run_norm_rows<T, P, QUANT, 8, true>(a, num_sms, stream);
  if constexpr (!QUANT)
    if (a.units % 320 == 0) return run_norm_rows<T, P, QUANT, 10, true>(a, num_sms, stream);
  if (a.units % 160 == 0) return run_norm_rows<T, P, QUANT, 5, true>(a, num_sms, stream);
  const bool four = a.units > 768 && a.units <= 1024;
  if (QUANT ? !four : sizeof(T) == 2 && (sizeof(P) == 2 || a.units <= 768)) return cudaErrorNotSupported;
  return run_norm_rows<T, P, QUANT, 8, false>(a, num_sms, stream);
}

// Units per thread.  Many: fewer warps share a row's reductions, and a thread has
// more bytes on their way (quantizer, 8192 x 14336 bf16: eight 54 us, four 67;
// norm, 8192 x 8192 bf16: eight 68, four 77, two 86 us).  Few: more warps per row,
// for latency and where rows are few (300 rows of 4096 into 8 bits: two 4.9,
// four 5.7 us).  The norm holds shorter rows better in four units (5120 bf16: 44
// us, eight 53) and fp32 in two (4096: 25.5, four 27.6 us); eight units of fp32
// do not fit in registers.
template <typename T, typename P, bool NORM, bool QUANT>
cudaError_t launch_rows(const RowArgs& a, int num_sms, cudaStream_t stream) {
  constexpr bool BF16 = sizeof(T) == 2;
  auto fits = [&](int v) { return a.units <= max_threads(v) * v; };
  // k_norm_rows: from 16 KB a row on (4800 x 8192 bf16: 39 us, k_rows 44; into 8 bits
  // 44 and 50; 4800 x 4096 bf16: 22.8 and 19.5), and where k_rows would read fp32
  // parameters beside bf16 rows, two lines a load (8192 x 4096: 31 and 37 us), but
  // from 4096 rows: 3000 x 4096 16.5 and 16.3, 1400 x 4096 12.7 and 9.2.
  const int64_t row_bytes = (int64_t)a.units * 8 * (int64_t)sizeof(T);
  if constexpr (NORM)
    if (a.M > 3 * (int64_t)num_sms && (row_bytes >= 16384 || (sizeof(P) > sizeof(T) && row_bytes >= 8192 && a.M >= 4096))) {
      const cudaError_t e = launch_norm_rows<T, P, QUANT>(a, num_sms, stream);
      if (e != cudaErrorNotSupported) return e;
    }
  int v = 4;
  if (a.M <= num_sms) v = 1;
  else if (NORM && a.M <= 3 * (int64_t)num_sms) v = 2;
  else if (BF16) v = a.units >= (NORM ? 1024 : 512) ? 8 : 4;
  else if (NORM) v = a.units <= 512 ? 2 : 4;
  v = std::min(v, (a.units + 31) / 32);                // no more than fill a warp
  if (v <= 1 && fits(1)) return run_rows<T, P, NORM, QUANT, 1, true>(a, num_sms, stream);
  if (v <= 2 && fits(2)) return run_rows<T, P, NORM, QUANT, 2, true>(a, num_sms, stream);
  if (v <= 4 && fits(4)) return run_rows<T, P, NORM, QUANT, 4, true>(a, num_sms, stream);
  if constexpr (BF16)
    if (fits(8)) return run_rows<T, P, NORM, QUANT, 8, true>(a, num_sms, stream);
  return run_rows<T, P, NORM, QUANT, 4, false>(a, num_sms, stream);
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
// The threads of a row keep the running dgamma and dbeta of their own columns in
// registers over all rows they meet; a CTA writes them once, as one row of the
// workspace, and k_ln_params sums those rows.  Every order of summation is fixed.
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

// A CTA of up to 512 threads works on `teams` rows at a time.  Each thread copies
// its own units of x and dy into shared memory `stages` rows ahead (cp.async: a
// thread waits for its own copies alone, so neither barriers nor registers are
// spent on what is on its way), reads them once for the row's sums and the
// parameters' gradients and once more for dx.  gamma waits in shared memory too:
// from L1, which the ring leaves too small for it, 8192 x 8192 fp32 took 227 us.
// Bound: bytes (8192 x 8192 fp32: 127 us, 6.3 TB/s; bf16: 93 us, where half the
// bytes go with as many instructions).
constexpr int kBwdThreads = 512, kBwdSmem = 224 * 1024, kBwdMaxStages = 4;

template <typename T, typename P, int V>
__global__ void __launch_bounds__(kBwdThreads, 1) k_ln_backward_rows(const BwdArgs a, int warps, int stages) {
  using U = Unit<T>;
  extern __shared__ __align__(16) uint8_t bwd_smem[];
  float* gain = reinterpret_cast<float*>(bwd_smem);            // gamma, or ones
  uint8_t* ring_raw = bwd_smem + (size_t)a.units * 32;
  __shared__ float2 red[2][kMaxWarps];
  Team team;
  team.warps = warps;
  team.index = (threadIdx.x >> 5) / warps;
  team.warp = (threadIdx.x >> 5) - team.index * warps;
  team.lane = threadIdx.x & 31;
  const int teams = (blockDim.x >> 5) / warps, base = team.index * warps;
  const int t = team.warp * 32 + team.lane, span = warps * 32;
  const uint32_t row_bytes = (uint32_t)a.units * 8u * (uint32_t)sizeof(T);
  uint8_t* ring = ring_raw + (size_t)team.index * stages * 2 * row_bytes;
  const int64_t stride = (int64_t)gridDim.x * teams;
  const float inv_k = 1.0f / (8.0f * (float)a.units);
  float dg[V][8], db[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = db[i][e] = 0.0f;
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  auto issue = [&](int64_t row, int stage) {
    if (row < a.M) {
      const T* x = static_cast<const T*>(a.x) + row * a.ldx;
      const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
      const uint32_t dst = tc::saddr(ring + (size_t)stage * 2 * row_bytes);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int u = i * span + t;
        if (u >= a.units) continue;
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
          const uint32_t off = (uint32_t)(u + h * a.units) * 16u;
          copy16(dst + off, reinterpret_cast<const uint8_t*>(x) + off);
          copy16(dst + row_bytes + off, reinterpret_cast<const uint8_t*>(dy) + off);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int64_t first = (int64_t)blockIdx.x * teams + team.index;
  for (int s = 0; s < stages; ++s) issue(first + s * stride, s);
  for (int u = threadIdx.x; u < a.units; u += blockDim.x) {
    float v[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (a.gamma != nullptr) U::param(static_cast<const P*>(a.gamma), u, a.units, v);
    U::store_param(gain, u, a.units, v);
  }
  __syncthreads();
  float mean = 0.0f, rstd = 0.0f;
  if (first < a.M) { mean = a.mean[first]; rstd = a.rstd[first]; }
  int turn = 0, stage = 0;
  for (int64_t row = first; row < a.M; row += stride, turn ^= 1) {
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (row + stride < a.M) { next_mean = a.mean[row + stride]; next_rstd = a.rstd[row + stride]; }
    if (stages == 4) copies_left<3>();
    else if (stages == 3) copies_left<2>();
    else copies_left<1>();
    const T* xs = reinterpret_cast<const T*>(ring + (size_t)stage * 2 * row_bytes);
    const T* ds = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(xs) + row_bytes);
    // xh and g = dy * gamma of unit u
    auto unit = [&](int u, float (&xh)[8], float (&dyv)[8], float (&g)[8]) {
      U w;
      w.load(xs, u, a.units);
      w.unpack(xh);
      w.load(ds, u, a.units);
      w.unpack(dyv);
      U::param(gain, u, a.units, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[e] = (xh[e] - mean) * rstd;
        g[e] *= dyv[e];
      }
    };
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = i * span + t;
      if (u >= a.units) continue;
      float xh[8], dyv[8], g[8];
      unit(u, xh, dyv, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s.x += g[e];
        s.y = fmaf(g[e], xh[e], s.y);
        dg[i][e] = fmaf(dyv[e], xh[e], dg[i][e]);
        db[i][e] += dyv[e];
      }
    }
    if (a.dx != nullptr) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
        s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
      }
      if (warps > 1) {
        float2* slot = red[turn] + base;
        if (team.lane == 0) slot[team.warp] = s;
        // one named barrier per team
        asm volatile("bar.sync %0, %1;" ::"r"(team.index + 1), "r"(span) : "memory");
        s = slot[0];
        for (int w = 1; w < warps; ++w) {
          s.x += slot[w].x;
          s.y += slot[w].y;
        }
      }
      const float c1 = s.x * inv_k, c2 = s.y * inv_k;
      T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int u = i * span + t;
        if (u >= a.units) continue;
        float xh[8], dyv[8], g[8], o[8];
        unit(u, xh, dyv, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rstd * (g[e] - fmaf(xh[e], c2, c1));
        U::store(dx, u, a.units, o);
      }
    }
    issue(row + stages * stride, stage);
    if (++stage == stages) stage = 0;
    mean = next_mean;
    rstd = next_rstd;
  }
  if (a.part == nullptr) return;
  copies_left<0>();
  float* pg = a.part + (int64_t)blockIdx.x * 16 * a.units;     // [dgamma | dbeta]
  float* pb = pg + (int64_t)8 * a.units;
  if (teams == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = i * span + t;
      if (u >= a.units) continue;
      U::store_param(pg, u, a.units, dg[i]);
      U::store_param(pb, u, a.units, db[i]);
    }
    return;
  }
  // the teams' sums, one after another, in the ring's place
  float* sum = reinterpret_cast<float*>(ring_raw);
  for (int k = 0; k < teams; ++k) {
    __syncthreads();
    if (team.index != k) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = i * span + t;
      if (u >= a.units) continue;
      if (k > 0) {
        float v[8];
        U::param(sum, u, a.units, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[i][e] += v[e];
        U::param(sum + a.units * 8, u, a.units, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) db[i][e] += v[e];
      }
      float* to_g = k == teams - 1 ? pg : sum;
      float* to_b = k == teams - 1 ? pb : sum + a.units * 8;
      U::store_param(to_g, u, a.units, dg[i]);
      U::store_param(to_b, u, a.units, db[i]);
    }
  }
}

// Small inputs, in one launch: dgamma and dbeta need no sums over a row, so the
// first CTAs take rows, for dx, and the rest take columns, for the parameters'
// gradients, reading x and dy a second time (from L2).  A column CTA takes 32
// bytes of every row: a warp four rows at a time, eight lanes of a word each; its
// warps' sums are joined in shared memory in their order.  Bound: latency (333 x
// 5120 bf16: 7.6 us; its bytes, once, 1.6).
constexpr int kSmallThreads = 512;

template <typename T, typename P, int V>
__global__ void __launch_bounds__(kSmallThreads, 2) k_ln_backward_small(const BwdArgs a, int warps, int row_ctas, float* dgamma,
                                                                         float* dbeta) {
  using U = Unit<T>;
  constexpr int C = 4 / (int)sizeof(T);               // columns per lane
  __shared__ float2 red[kSmallThreads / 32];
  __shared__ float sums[2][kSmallThreads / 32][8 * C];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  if ((int)blockIdx.x < row_ctas) {
    const int index = w / warps, base = index * warps, span = warps * 32, t = (w - base) * 32 + lane;
    const int64_t row = (int64_t)blockIdx.x * (kSmallThreads / 32 / warps) + index;
    if (index >= kSmallThreads / 32 / warps || row >= a.M) return;     // whole teams
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float xh[V][8], g[V][8];
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = i * span + t;
      if (u >= a.units) continue;
      U p, q;
      p.load(x, u, a.units);
      q.load(dy, u, a.units);
      float gm[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
      if (a.gamma != nullptr) U::param(static_cast<const P*>(a.gamma), u, a.units, gm);
      p.unpack(xh[i]);
      q.unpack(g[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[i][e] = (xh[i][e] - mean) * rstd;
        g[i][e] *= gm[e];
        s.x += g[i][e];
        s.y = fmaf(g[i][e], xh[i][e], s.y);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
      s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
    }
    if (warps > 1) {
      if (lane == 0) red[w] = s;
      asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(span) : "memory");
      s = red[base];
      for (int k = 1; k < warps; ++k) {
        s.x += red[base + k].x;
        s.y += red[base + k].y;
      }
    }
    const float inv_k = 1.0f / (8.0f * (float)a.units), c1 = s.x * inv_k, c2 = s.y * inv_k;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int u = i * span + t;
      if (u >= a.units) continue;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd * (g[i][e] - fmaf(xh[i][e], c2, c1));
      U::store(dx, u, a.units, o);
    }
    return;
  }
  const int col = ((int)blockIdx.x - row_ctas) * 8 * C + (lane & 7) * C;   // K is a multiple of 8 * C
  float sg[C] = {}, sb[C] = {};
#pragma unroll 4
  for (int64_t row = w * 4 + (lane >> 3); row < a.M; row += kSmallThreads / 8) {
    const uint32_t xw = *reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.x) + row * a.ldx + col);
    const uint32_t dw = *reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.dy) + row * a.lddy + col);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float xv[C], dv[C];
    if constexpr (C == 2) {
      xv[0] = __uint_as_float(xw << 16); xv[1] = __uint_as_float(xw & 0xFFFF0000u);
      dv[0] = __uint_as_float(dw << 16); dv[1] = __uint_as_float(dw & 0xFFFF0000u);
    } else {
      xv[0] = __uint_as_float(xw);
      dv[0] = __uint_as_float(dw);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      sg[c] = fmaf(dv[c], (xv[c] - mean) * rstd, sg[c]);
      sb[c] += dv[c];
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      sg[c] += __shfl_xor_sync(0xFFFFFFFFu, sg[c], o);
      sb[c] += __shfl_xor_sync(0xFFFFFFFFu, sb[c], o);
    }
    if (lane < 8) {
      sums[0][w][lane * C + c] = sg[c];
      sums[1][w][lane * C + c] = sb[c];
    }
  }
  __syncthreads();
  if (threadIdx.x < 16 * C) {
    const int which = threadIdx.x / (8 * C), c = threadIdx.x % (8 * C);
    float v = sums[which][0][c];
#pragma unroll
    for (int k = 1; k < kSmallThreads / 32; ++k) v += sums[which][k][c];
    float* out = which == 0 ? dgamma : dbeta;
    if (out != nullptr) out[((int)blockIdx.x - row_ctas) * 8 * C + c] = v;
  }
}

// Rows too long for that ring (bf16 from K = 16400 on, fp32 from 11472).
// Bound: its reads, once per column chunk with nothing loaded ahead (4096 x 14336
// fp32: 270 us, its bytes once 108; 4096 x 16400 bf16: 352 and 62).
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
      Unit<T> w;
      w.load(x, u, a.units);
      w.unpack(xv);
      w.load(dy, u, a.units);
      w.unpack(dyv);
      float gm[8];
      if (a.gamma != nullptr) Unit<T>::param(static_cast<const P*>(a.gamma), u, a.units, gm);
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
        Unit<T>::store(dx, u, a.units, o);
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
      Unit<T>::store_param(pg, u, a.units, dg[i]);
      Unit<T>::store_param(pb, u, a.units, db[i]);
    }
  }
}

// dgamma / dbeta = sum over the workspace's rows: 32 columns per CTA, one warp
// per 32nd row, joined in shared memory in the order of the warps.
__global__ void __launch_bounds__(1024) k_ln_params(const float* part, int parts, int64_t K, float* dgamma,
                                                    float* dbeta) {
  __shared__ float red[32][33];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + l;   // column of [dgamma | dbeta]; 2 K is a multiple of 32
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  float v[(kLnMaxParts + 31) / 32];
#pragma unroll
  for (int i = 0; i < (kLnMaxParts + 31) / 32; ++i)
    v[i] = w + 32 * i < parts ? part[(int64_t)(w + 32 * i) * 2 * K + c] : 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < (kLnMaxParts + 31) / 32; ++i) s += v[i];
  red[w][l] = s;
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += red[i][l];
    float* out = c < K ? dgamma : dbeta;
    if (out != nullptr) out[c < K ? c : c - K] = s;
  }
}

template <typename T, typename P, int V>
cudaError_t run_backward_rows(const BwdArgs& a, int warps, int teams, int stages, int parts, cudaStream_t stream) {
  static tc::SmemOnce once;
  cudaError_t e = once.set(k_ln_backward_rows<T, P, V>, kBwdSmem);
  if (e != cudaSuccess) return e;
  const size_t row = (size_t)a.units * 8 * sizeof(T), sums = teams > 1 ? (size_t)a.units * 64 : 0;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = dependent_launch(dim3((unsigned)parts), 32 * warps * teams,
                                                  (size_t)a.units * 32 + std::max((size_t)teams * stages * 2 * row, sums), stream, &at);
  return cudaLaunchKernelEx(&cfg, k_ln_backward_rows<T, P, V>, a, warps, stages);
}

template <typename T, typename P>
cudaError_t run_backward_small(const BwdArgs& a, float* dgamma, float* dbeta, cudaStream_t stream) {
  const int v = a.units > kSmallThreads / 2 ? 2 : 1;         // units per thread
  const int warps = (a.units + 32 * v - 1) / (32 * v), teams = kSmallThreads / 32 / warps;
  const int row_ctas = a.dx != nullptr ? (int)((a.M + teams - 1) / teams) : 0;
  const int col_ctas = dgamma != nullptr || dbeta != nullptr ? a.units * (int)sizeof(T) / 4 : 0;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = dependent_launch(dim3((unsigned)(row_ctas + col_ctas)), kSmallThreads, 0, stream, &at);
  return cudaLaunchKernelEx(&cfg, v == 2 ? k_ln_backward_small<T, P, 2> : k_ln_backward_small<T, P, 1>, a, warps, row_ctas,
                            dgamma, dbeta);
}

// *parts: rows of the workspace that were written.
template <typename T, typename P>
cudaError_t run_backward(const BwdArgs& a, int num_sms, int* parts, cudaStream_t stream) {
  const int most = std::min(num_sms, kLnMaxParts);
  // Units per thread: four, for more rows at a time (8192 x 8192 bf16: four 93 us,
  // two 112), but two for short rows (8192 x 1024: 19 us, four 23) and where four
  // leave a team no room for two rows in shared memory (8192 x 8192 fp32).
  for (int v = a.units < 256 ? 2 : 4; v >= 2; v /= 2) {
    const int warps = (a.units + 32 * v - 1) / (32 * v);
    if (warps > kBwdThreads / 32) break;
    const int teams = std::min(kBwdThreads / 32 / warps, 15);
    const int64_t per_stage = (int64_t)teams * 2 * a.units * 8 * (int64_t)sizeof(T);
    const int stages = (int)std::min<int64_t>(kBwdMaxStages, (kBwdSmem - (int64_t)a.units * 32) / per_stage);
    if (stages < 2) continue;
    *parts = (int)std::min<int64_t>(most, (a.M + teams - 1) / teams);
    if (v == 4) return run_backward_rows<T, P, 4>(a, warps, teams, stages, *parts, stream);
    return run_backward_rows<T, P, 2>(a, warps, teams, stages, *parts, stream);
  }
  const int threads = std::min(512, (a.units + 63) / 64 * 32);
  *parts = (int)std::min<int64_t>(most, a.M);
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = dependent_launch(
      dim3((unsigned)*parts, (unsigned)((a.units + 2 * threads - 1) / (2 * threads))), threads, 0, stream, &at);
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
  BwdArgs a{};
  a.dy = n.dy; a.lddy = n.lddy; a.x = n.x; a.ldx = n.ldx; a.gamma = n.gamma;
  a.mean = n.mean; a.rstd = n.rstd; a.dx = n.dx; a.lddx = n.lddx;
  const bool params = n.dgamma != nullptr || n.dbeta != nullptr;
  a.part = params ? n.part : nullptr;
  a.M = n.M; a.units = (int)(n.K / 8);
  // k_ln_backward_small while reading x and dy twice costs less than the second
  // launch and the partial sums: 333 x 5120 bf16 7.6 us, the two kernels 12.6; 64 x
  // 4096 3.2 and 7.3; 1000 x 8192 (33 MB) 21 and 27; 2000 x 2048 14.0 and 15.6; but
  // 4000 x 256 10.4 and 8.4, 1500 x 5120 fp32 (61 MB) 37 and 26.
  if (n.M <= 2048 && 2 * n.M * n.K * (n.dt == NVFP4_BF16 ? 2 : 4) <= (36ll << 20) && a.units <= 2 * kSmallThreads) {
    if (n.dt == NVFP4_BF16)
      return n.pdt == NVFP4_BF16 ? run_backward_small<__nv_bfloat16, __nv_bfloat16>(a, n.dgamma, n.dbeta, stream)
                                 : run_backward_small<__nv_bfloat16, float>(a, n.dgamma, n.dbeta, stream);
    return n.pdt == NVFP4_BF16 ? run_backward_small<float, __nv_bfloat16>(a, n.dgamma, n.dbeta, stream)
                               : run_backward_small<float, float>(a, n.dgamma, n.dbeta, stream);
  }
  int parts = 0;
  cudaError_t e;
  if (n.dt == NVFP4_BF16)
    e = n.pdt == NVFP4_BF16 ? run_backward<__nv_bfloat16, __nv_bfloat16>(a, num_sms, &parts, stream)
                            : run_backward<__nv_bfloat16, float>(a, num_sms, &parts, stream);
  else
    e = n.pdt == NVFP4_BF16 ? run_backward<float, __nv_bfloat16>(a, num_sms, &parts, stream)
                            : run_backward<float, float>(a, num_sms, &parts, stream);
  if (e != cudaSuccess || !params) return e;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = dependent_launch(dim3((unsigned)(2 * n.K / 32)), 1024, 0, stream, &at);
  return cudaLaunchKernelEx(&cfg, k_ln_params, (const float*)a.part, parts, n.K, n.dgamma, n.dbeta);
}

}  // namespace nvfp4
