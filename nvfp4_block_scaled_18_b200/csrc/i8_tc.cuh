// tcgen05 wrappers of the 8-bit integer linear's kernels (kind::i8).
#pragma once

#include <atomic>

#include "tcgen05.cuh"

namespace nvfp4 {
namespace tc {

// One lane of a converged warp, the same each time.  Roles are run by whole
// warps that branch only around the issuing instructions: the operands of
// tcgen05.mma then stay in uniform registers.  With the role in a single
// lane's branch a stage of four MMAs took 460 ns to issue, whatever their size.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A warp's bounded wait for something far off (a whole tile's MMAs): one lane
// polls, sleeping in between, and the others wait for it, so that the pollers do
// not compete with the copies and the MMAs for shared memory.  True for every
// lane when the phase came.
template <bool CLUSTER = false, bool DRAIN = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, WaitState* w, int* st) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    auto poll = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (!poll()) {
      const uint64_t t0 = globaltimer();
      while (!poll()) {
        if (!DRAIN && wait_aborted(w)) { ok = 0; break; }
        if (globaltimer() - t0 > w->limit_ns) {
          wait_raise(w);
          report_status(st, NVFP4_ERR_TIMEOUT);
          ok = 0;
          break;
        }
        __nanosleep(20);
      }
    }
  }
  ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
  // the lanes that did not poll observe the phase too: it is over, so this does not wait
  if (ok) ok = __all_sync(0xFFFFFFFFu, CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity));
  return ok != 0;
}

// What is added where there is no bias: x + -0 is x, the sign of a zero included.
constexpr float kNoBias = -0.0f;

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

// 4 or 16 columns of this warp's TMEM lane quadrant.
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
// Bulk copy into the shared memory of another CTA of the cluster; its bytes
// count on an mbarrier there (both addresses from mapa_shared).
__device__ __forceinline__ void copy_to_peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t remote_bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(remote_bar)
               : "memory");
}

// A kernel's shared-memory limit, raised once per device (the call takes a
// microsecond; for devices from the 64th on it is made every time).
struct SmemOnce {
  std::atomic<uint64_t> done{0};
  template <typename F>
  cudaError_t set(F kern, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit != 0 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// 2-D tensor map over int8 rows (rows x K, row pitch ld bytes): boxes of 128
// bytes x box_rows rows, 128-byte swizzle, zero fill out of range.
bool encode_i8_map(CUtensorMap* map, const int8_t* p, int64_t rows, int64_t K, int64_t ld, uint32_t box_rows);

}  // namespace tc
}  // namespace nvfp4
