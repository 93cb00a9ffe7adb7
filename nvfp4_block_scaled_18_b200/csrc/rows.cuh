// Device helpers of the row-wise kernels (layer norm, 8-bit quantizer): a team
// of W warps owns one row, each thread holds V units of 8 elements of it.
#pragma once

#include "common.cuh"

namespace nvfp4 {
namespace rows {

constexpr int kMaxWarps = 32;   // warps of one CTA

// A team of warps.  `slot` is its area for one reduction (one word per warp); the
// caller alternates slots so that a slot is written again only after a later
// barrier of the same team.
struct Team {
  int warps;      // W: warps of the team
  int index;      // team within the CTA
  int warp;       // warp within the team
  int lane;
  __device__ __forceinline__ void sync() const {
    // one named barrier per team (at most two of several warps); barrier 0 stays the CTA's own
    if (index == 0) asm volatile("bar.sync 1, %0;" ::"r"(warps * 32) : "memory");
    else asm volatile("bar.sync 2, %0;" ::"r"(warps * 32) : "memory");
  }
  // Sum over the team: within each warp by shuffles, then every thread adds the
  // warps' sums from shared memory (fewer instructions than a second round of
  // shuffles up to about ten warps).
  __device__ __forceinline__ double sum(double v, double* slot) const {
    v = warp_sum_f64(v);
    if (warps == 1) return v;
    if (lane == 0) slot[warp] = v;
    sync();
    v = slot[0];
    for (int w = 1; w < warps; ++w) v += slot[w];
    return v;
  }
  __device__ __forceinline__ uint32_t max(uint32_t v, uint32_t* slot) const {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (warps == 1) return v;
    if (lane == 0) slot[warp] = v;
    sync();
    return __reduce_max_sync(0xFFFFFFFFu, lane < warps ? slot[lane] : 0u);
  }
};

// Two fp32 additions or products, each rounded once, in one instruction.  A packed
// product that feeds a packed sum is contracted by the compiler all the same
// (codes then differ in one of 5e4): such pairs stay with __fmul_rn and __fadd_rn.
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ void mul2(float& a, float& b, float c, float d) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}
// max(m, |a|, |b|); a NaN stays.
__device__ __forceinline__ float max3_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}
// fl32(1 / sqrt(x)) for x >= 0: the fp32 estimate and two Newton steps in
// binary64, within 2^-48 of the exact value before its one rounding; outside the
// estimate's range the library's functions.
__device__ __forceinline__ float rsqrt_rounded(double x) {
  if (x > 1e-30 && x < 1e30) {
    double r = (double)rsqrtf((float)x);
    const double h = 0.5 * x;
    r = r * fma(-h * r, r, 1.5);
    r = r * fma(-h * r, r, 1.5);
    return (float)r;
  }
  return (float)(1.0 / sqrt(x));
}

// Whether a row's statistics give it a norm: both finite, and rstd not the 0 that
// comes of a difference from the mean beyond fp32.
__device__ __forceinline__ bool has_norm(float mean, float rstd) {
  return abs_key(mean) < 0x7F800000u && abs_key(rstd) - 1u < 0x7F7FFFFFu;
}

// A unit is eight elements of a row, and what one thread handles at a time: of
// bf16 rows 16 bytes, elements 8u..8u+7; of fp32 rows two runs of 16 bytes, one
// from each half of the row, elements 4u..4u+3 and K/2 + 4u..K/2 + 4u+3, so that
// a warp's loads and stores are whole lines (with 32 bytes a lane every store
// touched its sectors twice).  `units` = K / 8.
//
// Plain loads, not the read-only path: the preceding kernel may still be writing
// when this one starts.
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xFFFF0000u);
  v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  v[4] = __uint_as_float(w.z << 16); v[5] = __uint_as_float(w.z & 0xFFFF0000u);
  v[6] = __uint_as_float(w.w << 16); v[7] = __uint_as_float(w.w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack8(const float4& a, const float4& b, float (&v)[8]) {
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Element i of an array of V, by a 32-bit byte offset from a uniform base.
template <typename V, typename B>
__device__ __forceinline__ const V& at(const B* base, int i) {
  return *reinterpret_cast<const V*>(reinterpret_cast<const char*>(base) + (uint32_t)i * (uint32_t)sizeof(V));
}
template <typename V, typename B>
__device__ __forceinline__ V& at(B* base, int i) {
  return *reinterpret_cast<V*>(reinterpret_cast<char*>(base) + (uint32_t)i * (uint32_t)sizeof(V));
}

template <typename T> struct Unit;
template <> struct Unit<__nv_bfloat16> {
  using T = __nv_bfloat16;
  uint4 w;                       // as it is in memory: what a row on its way occupies
  __device__ __forceinline__ void load(const T* row, int u, int) { w = at<uint4>(row, u); }
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void unpack(float (&v)[8]) const { unpack8(w, v); }
  // unpacked again after this, not kept unpacked
  __device__ __forceinline__ void forget() { asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)); }
  static __device__ __forceinline__ void store(T* row, int u, int, const float (&v)[8]) {
    at<uint4>(row, u) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
  static __device__ __forceinline__ void store_codes(int8_t* row, int u, int, uint2 c) { at<uint2>(row, u) = c; }
  // the unit's elements of a parameter vector
  static __device__ __forceinline__ void param(const __nv_bfloat16* p, int u, int, float (&v)[8]) {
    unpack8(at<uint4>(p, u), v);
  }
  static __device__ __forceinline__ void param(const float* p, int u, int, float (&v)[8]) {
    unpack8(at<float4>(p, 2 * u), at<float4>(p, 2 * u + 1), v);
  }
  static __device__ __forceinline__ void store_param(float* p, int u, int, const float (&v)[8]) {
    at<float4>(p, 2 * u) = make_float4(v[0], v[1], v[2], v[3]);
    at<float4>(p, 2 * u + 1) = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <> struct Unit<float> {
  using T = float;
  float4 a, b;
  __device__ __forceinline__ void load(const T* row, int u, int units) {
    a = at<float4>(row, u);
    b = at<float4>(row, u + units);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void unpack(float (&v)[8]) const { unpack8(a, b, v); }
  __device__ __forceinline__ void forget() {
    asm volatile("" : "+f"(a.x), "+f"(a.y), "+f"(a.z), "+f"(a.w), "+f"(b.x), "+f"(b.y), "+f"(b.z), "+f"(b.w));
  }
  static __device__ __forceinline__ void store(T* row, int u, int units, const float (&v)[8]) {
    at<float4>(row, u) = make_float4(v[0], v[1], v[2], v[3]);
    at<float4>(row, u + units) = make_float4(v[4], v[5], v[6], v[7]);
  }
  static __device__ __forceinline__ void store_codes(int8_t* row, int u, int units, uint2 c) {
    at<uint32_t>(row, u) = c.x;
    at<uint32_t>(row, u + units) = c.y;
  }
  static __device__ __forceinline__ void param(const __nv_bfloat16* p, int u, int units, float (&v)[8]) {
    const uint2 x = at<uint2>(p, u), y = at<uint2>(p, u + units);
    unpack8(make_uint4(x.x, x.y, y.x, y.y), v);
  }
  static __device__ __forceinline__ void param(const float* p, int u, int units, float (&v)[8]) {
    unpack8(at<float4>(p, u), at<float4>(p, u + units), v);
  }
  static __device__ __forceinline__ void store_param(float* p, int u, int units, const float (&v)[8]) { store(p, u, units, v); }
};

// rint(v * inv) of eight values as packed bytes.  |v * inv| <= 128, so adding
// 1.5 * 2^23 rounds the (already rounded) product to the nearest integer, ties
// to even, and leaves it in two's complement in the sum's low byte.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], inv), 12582912.0f));
  const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return make_uint2(lo, hi);
}

// Rows whose largest magnitude is below this have scale 0 and codes 0
// (127 / amax would leave the normal range not far below).
#define NVFP4_I8_MIN_AMAX 0x1p-110f

struct RowScale {
  float scale, inv;
};
// Scale and multiplier of a row from the key of its largest magnitude: NaN and
// multiplier 0 when the row holds a NaN or an infinity.
__device__ __forceinline__ RowScale row_scale(uint32_t amax_key) {
  if (amax_key >= 0x7F800000u) return RowScale{__uint_as_float(0x7FFFFFFFu), 0.0f};
  const float amax = __uint_as_float(amax_key);
  if (amax < NVFP4_I8_MIN_AMAX) return RowScale{0.0f, 0.0f};
  return RowScale{__fdiv_rn(amax, 127.0f), __fdiv_rn(127.0f, amax)};
}

}  // namespace rows
}  // namespace nvfp4
