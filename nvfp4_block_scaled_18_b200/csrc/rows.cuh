// Device helpers of the row-wise kernels (layer norm, 8-bit quantizer): a team
// of W warps owns one row, each thread holds V units of 8 elements of it.
#pragma once

#include "common.cuh"

namespace nvfp4 {
namespace rows {

constexpr int kMaxTeams = 8;    // rows a CTA works on at a time
constexpr int kMaxWarps = 32;   // warps of one CTA

// Sum or maximum over a team.  `slot` is the team's area for this reduction
// (one word per warp); the caller alternates slots so that a slot is written
// again only after a later barrier of the same team.
struct Team {
  int warps;      // W: warps of the team
  int index;      // team within the CTA
  int warp;       // warp within the team
  int lane;
  __device__ __forceinline__ void sync() const {
    // one named barrier per team; barrier 0 stays the CTA's own
    asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(warps * 32) : "memory");
  }
  __device__ __forceinline__ double sum(double v, double* slot) const {
    v = warp_sum_f64(v);
    if (warps == 1) return v;
    if (lane == 0) slot[warp] = v;
    sync();
    return warp_sum_f64(lane < warps ? slot[lane] : 0.0);
  }
  __device__ __forceinline__ uint32_t max(uint32_t v, uint32_t* slot) const {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (warps == 1) return v;
    if (lane == 0) slot[warp] = v;
    sync();
    return __reduce_max_sync(0xFFFFFFFFu, lane < warps ? slot[lane] : 0u);
  }
};

// Eight consecutive elements as fp32 (16-byte aligned).  Plain loads, not the
// read-only path: the preceding kernel may still be writing when this one starts.
__device__ __forceinline__ void fetch8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  v[4] = __uint_as_float(u.z << 16); v[5] = __uint_as_float(u.z & 0xFFFF0000u);
  v[6] = __uint_as_float(u.w << 16); v[7] = __uint_as_float(u.w & 0xFFFF0000u);
}
__device__ __forceinline__ void fetch8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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
