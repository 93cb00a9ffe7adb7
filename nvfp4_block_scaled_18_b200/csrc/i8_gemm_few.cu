// 8-bit integer linear for few tokens, sm_100a: the operands of i8_gemm.cu swapped.
//
// Y^T = W A^T: 128 rows of W are the tensor cores' M, the tokens (padded to NP)
// their N, so one pass over W serves all tokens.  W's bytes are the bound; to
// keep every SM loading, the ks CTAs of a thread-block cluster split K.  The
// sums are int32, so splitting and joining them changes nothing.
//
// Grid: ks * ceil(N / 128) CTAs, ks consecutive ones a cluster.  256 threads:
// warp 0 loads W and token tiles by TMA into a ring; warp 1 issues
// the MMAs.  Then every CTA owns a run of T tokens.  All warps move the others'
// part of the 128 x NP int32 partial from TMEM to the idle ring, one bulk copy
// per owner sends it on (stores into a peer's shared memory, 16 bytes a lane,
// took 3 us for 32 KB), and each owner adds what it was sent to its own
// accumulator, scales the sums and writes Y, 32 consecutive columns a store.
//
// Programmatic dependent launch: before griddepcontrol.wait the kernel sets up
// and asks L2 to prefetch the first ring of W tiles; it loads nothing else.
// Every mbarrier wait is bounded; every CTA reaches every cluster barrier.
//
// Bound: W's bytes, read at 6.7 TB/s between the first tile (1 us after the start)
// and the last; joining K's parts and writing Y takes 2 us (16 tokens) to 4 us (128)
// more (61 x 5120 x 27648: 27.3 us, 5.3 TB/s over all; 16 x 14336 x 4096: 12.1 us).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "i8_plan.h"
#include "i8_tc.cuh"
#include "kernels.h"

namespace nvfp4 {
using namespace tc;
namespace {

constexpr int THREADS = 256;
using i8::BK;
using i8::W_ROWS;
template <int NP, int CTAS> using Cfg = i8::FewCfg<NP, CTAS>;

struct Params {
  const float* a_scales;
  const float* w_scales;
  const float* bias;
  void* y;
  int64_t ldy;
  int M, N;
  int per_owner;      // T: tokens of an owner, a multiple of G
  int land;           // byte offset of the arriving partial sums from the ring's start
  int k_steps;        // stages of work along K: ceil(K / 128)
  int* st;
  uint64_t wait_ns;
  int hold;
};

template <int NP, int CTAS, bool BF16OUT>
__global__ void __launch_bounds__(THREADS, 1)
    k_i8_few(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
  using C = Cfg<NP, CTAS>;
  using Out = std::conditional_t<BF16OUT, __nv_bfloat16, float>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ __align__(16) float token_scale[NP];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int* part = reinterpret_cast<const int*>(smem + p.land);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::RING + (C::OVERLAY ? 0 : C::PART));
  uint64_t* full = bars;
  uint64_t* empty = bars + C::STAGES;
  uint64_t* acc_full = bars + 2 * C::STAGES;
  uint64_t* landed = acc_full + 1;        // the others' partial sums
  WaitState* ws = reinterpret_cast<WaitState*>(landed + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ws + 1);

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), ks = (int)cluster_nctarank();
  const int n0 = (int)(blockIdx.x / ks) * W_ROWS;
  const int s0 = (int)((int64_t)rank * p.k_steps / ks), s1 = (int)((int64_t)(rank + 1) * p.k_steps / ks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(saddr(&full[s]), 1);
      mbar_init(saddr(&empty[s]), 1);
    }
    mbar_init(saddr(acc_full), 1);
    mbar_init(saddr(landed), 1);
    ws->abort = 0;
    ws->limit_ns = p.wait_ns;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmW) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmX) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int g = s0; g < min(s1, s0 + C::STAGES); ++g) prefetch_l2_tile_2d(&tmW, g * BK, n0);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (!C::OVERLAY && ks > 1) cluster_arrive_relaxed();     // this CTA runs: peers may push into its partial area
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    int issued = 0;
    for (int g = s0; !p.hold && g < s1; ++g, ++issued) {
      const int s = issued % C::STAGES;
      bool ok = mbar_wait_inline(saddr(&empty[s]), (uint32_t)((issued / C::STAGES) & 1) ^ 1u, ws, p.st);
      ok = __all_sync(0xFFFFFFFFu, ok) != 0;
      if (!ok) break;
      const uint32_t dst = saddr(smem + s * C::STAGE), bar = saddr(&full[s]);
      if (elect_one()) {                                   // bytes past K arrive as zeros
        mbar_expect_tx(bar, C::STAGE);
        tma_load_2d(dst, &tmW, g * BK, n0, bar);
        tma_load_2d(dst + C::W_BYTES, &tmX, g * BK, 0, bar);
      }
      __syncwarp();
    }
    for (int i = max(0, issued - C::STAGES); i < issued; ++i)
      (void)mbar_drain(saddr(&full[i % C::STAGES]), (uint32_t)((i / C::STAGES) & 1), ws, p.st);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t idesc = idesc_i8(W_ROWS, NP);
    for (int g = s0; g < s1; ++g) {
      const int i = g - s0, s = i % C::STAGES;
      bool ok = mbar_wait_inline(saddr(&full[s]), (uint32_t)((i / C::STAGES) & 1), ws, p.st);
      ok = __all_sync(0xFFFFFFFFu, ok) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = saddr(smem + s * C::STAGE);
      const uint64_t da = desc_sw128(base), db = desc_sw128(base + C::W_BYTES);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_i8<1>(tmem, da + (uint64_t)(2 * k), db + (uint64_t)(2 * k), idesc, (i > 0 || k > 0) ? 1u : 0u);
        commit<1>(saddr(&empty[s]));
      }
      __syncwarp();
    }
    if (elect_one()) commit<1>(saddr(acc_full));      // every MMA issued has completed
  }
  __syncwarp();
  // this thread's column of Y and its scale, loaded while the MMAs run
  const int q = warp & 3, half = warp >> 2, row = q * 32 + lane, n = n0 + row;
  float sw = 0.0f, bias = kNoBias;
  if (n < p.N) {
    sw = p.w_scales[n];
    if (p.bias != nullptr) bias = p.bias[n];
  }
  for (int m = threadIdx.x; m < p.M; m += THREADS) token_scale[m] = p.a_scales[m];
  const bool ok = warp_wait<false, true>(saddr(acc_full), 0u, ws, p.st);
  tc_fence_after();
  const bool have = __all_sync(0xFFFFFFFFu, ok && !wait_aborted(ws)) != 0;
  const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16);
  constexpr int G = C::G;
  const int T = p.per_owner, groups = (p.M + G - 1) / G;       // G tokens each
  const int own0 = min(groups, rank * T / G), own1 = min(groups, (rank + 1) * T / G);
  bool arrived = true;
  if (ks > 1) {
    if (threadIdx.x == 0) {
      const int bytes = (ks - 1) * (own1 - own0) * G * 512;
      mbar_expect_tx(saddr(landed), (uint32_t)bytes);
    }
    int* stage = reinterpret_cast<int*>(smem);                 // [token, this CTA's own left out][row]
    for (int j = half; j < groups; j += 2) {
      if (j >= own0 && j < own1) continue;                     // uniform across the warp
      uint32_t v[G] = {};
      if (have) {
        tmem_ld_n(acc + (uint32_t)(j * G), v);
        tmem_ld_wait();
      }
      int* to = stage + (j < own0 ? j : j - (own1 - own0)) * G * W_ROWS + row;
#pragma unroll
      for (int i = 0; i < G; ++i) to[i * W_ROWS] = (int)v[i];
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (C::OVERLAY) cluster_sync();                            // every ring of the cluster is idle
    else cluster_wait();                                       // every peer has started
    if (threadIdx.x < ks && (int)threadIdx.x != rank) {
      const int o = (int)threadIdx.x, o0 = min(groups, o * T / G), o1 = min(groups, (o + 1) * T / G);
      if (o1 > o0) {
        const uint32_t from = saddr(stage + (o < rank ? o0 : o0 - (own1 - own0)) * G * W_ROWS);
        const uint32_t to = saddr(smem + p.land) + (uint32_t)((rank < o ? rank : rank - 1) * (o1 - o0) * G * 512);
        copy_to_peer(mapa_shared(to, (uint32_t)o), from, (uint32_t)((o1 - o0) * G * 512), mapa_shared(saddr(landed), (uint32_t)o));
      }
    }
    __syncwarp();
    arrived = warp_wait<true, true>(saddr(landed), 0u, ws, p.st);
    cluster_arrive();                // what this CTA was sent is here: the senders may leave
  } else {
    __syncthreads();                 // token_scale
  }
  for (int j = own0 + half; j < own1; j += 2) {
    uint32_t v[G] = {};
    if (have) {
      tmem_ld_n(acc + (uint32_t)(j * G), v);
      tmem_ld_wait();
    }
    for (int src = 0; src < ks - 1; ++src) {
      const int* from = part + (size_t)(src * (own1 - own0) + (j - own0)) * G * W_ROWS + row;
#pragma unroll
      for (int i = 0; i < G; ++i) v[i] += (uint32_t)from[i * W_ROWS];
    }
    // the stores' addresses are the bulk of this loop's instructions: one running pointer
    Out* y = static_cast<Out*>(p.y) + (int64_t)(j * G) * p.ldy + n;
    const int left = n < p.N ? p.M - j * G : 0;
    const float4* ts = reinterpret_cast<const float4*>(token_scale + j * G);
#pragma unroll
    for (int i = 0; i < G; i += 4) {
      const float4 t = ts[i / 4];
      const float s4[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int e = 0; e < 4; ++e, y += p.ldy) {
        const float f = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn((int)v[i + e]), s4[e]), sw), bias);
        if (i + e < left) {
          if constexpr (BF16OUT) *y = __float2bfloat16_rn(f);
          else *y = f;
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
  }
  if (ks > 1) {
    cluster_wait();                  // what this CTA sent has arrived
    if (!arrived) (void)warp_wait<true, true>(saddr(landed), 0u, ws, p.st);    // given up before: all has been sent by now
  }
}

template <int NP, int CTAS>
cudaLaunchConfig_t few_config(unsigned grid, int ks, cudaStream_t stream, cudaLaunchAttribute (&at)[2]) {
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)ks; at[1].val.clusterDim.y = 1; at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Cfg<NP, CTAS>::SMEM;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cfg;
}

// Stands in for k_i8_few in questions of occupancy, never launched: the device counts
// one CTA per SM for any kernel that allocates tensor memory, and two run.
__global__ void __launch_bounds__(THREADS) k_few_shape() {}
SmemOnce shape_once;

// Clusters of ks CTAs, CTAS per SM, that the device holds at once: asked once per
// device and split, since the GPCs' sizes differ (148 SMs held 33 clusters of four
// at one CTA per SM, 132 CTAs, and 71 at two; 36 of them at one took two waves, 64 x
// 4500 x 28672 41 us, in three parts 26).  The answer is what fits, not what the
// device achieves each time: 56 clusters of five at two per SM still take a second
// wave (5 x 7168 x 14336 21 us, 57 tiles in four parts 18.8).
template <int NP, int CTAS>
int clusters_at_once(int ks, int num_sms) {
  static std::atomic<int> cache[16][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 16;
  // not known: a low guess, which only splits K less
  return i8::asked_once(dev < 16 ? &cache[dev][ks] : nullptr, std::max(1, num_sms * CTAS / ks / 2), [&] {
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = few_config<NP, CTAS>((unsigned)(num_sms * 8 / ks * ks), ks, nullptr, at);
    cfg.dynamicSmemBytes += NP * 4;               // the static part
    int n = 0;
    if (shape_once.set(k_few_shape, 232448) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, k_few_shape, &cfg) == cudaSuccess)
      return n;
    (void)cudaGetLastError();                     // the call goes on without the answer
    return -1;
  });
}

// The largest split of K whose clusters fit one wave (16 x 4096 x 14336 in 32
// clusters of eight 12.4 us, of four 13.7; 5 x 5888 x 14336 in 46 clusters of six,
// one too many, 22.1 us, of five 15.8), whose partial sums fit and which leaves a CTA
// enough steps to pay for joining them: above 32 tokens ten (128 x 4096 x 4096: 10.1
// us split in 3, 10.6 in 4).  At two CTAs per SM not seven: 37 clusters of them are no
// faster than 37 of six (5 x 4736 x 14336: 13.8 and 13.5 us, x 2048 5.4 and 5.0).
template <int NP, int CTAS>
int choose_ks(int64_t M, int64_t tiles, int k_steps, int num_sms) {
  return i8::split_of_k(tiles, k_steps, NP > 32 ? 10 : 1,
                        [&](int k) { return !(CTAS == 2 && k == 7) && Cfg<NP, CTAS>::fits((int)M, k); },
                        [&](int k) { return clusters_at_once<NP, CTAS>(k, num_sms); });
}

template <int NP, int CTAS, bool BF16OUT>
cudaError_t launch_np(const I8GemmArgs& g, int num_sms, cudaStream_t stream) {
  using C = Cfg<NP, CTAS>;
  const int64_t tiles = (g.N + W_ROWS - 1) / W_ROWS;
  const int k_steps = (int)((g.K + BK - 1) / BK);
  const int ks = choose_ks<NP, CTAS>(g.M, tiles, k_steps, num_sms);
  if (tiles * ks > INT32_MAX) return cudaErrorNotSupported;
  CUtensorMap tmW, tmX;
  if (!encode_i8_map(&tmW, g.w, g.N, g.K, g.ldw, W_ROWS) || !encode_i8_map(&tmX, g.a, g.M, g.K, g.lda, NP))
    return cudaErrorInvalidValue;
  Params p{};
  p.a_scales = g.a_scales; p.w_scales = g.w_scales; p.bias = g.bias; p.y = g.y; p.ldy = g.ldy;
  p.M = (int)g.M; p.N = (int)g.N; p.k_steps = k_steps; p.st = g.st;
  p.per_owner = C::per_owner((int)g.M, ks);
  p.land = C::OVERLAY ? C::RING - (ks - 1) * p.per_owner * 512 : C::RING;
  const WaitTest wt = wait_test();
  p.wait_ns = wt.limit_ns; p.hold = wt.hold;
  auto kern = k_i8_few<NP, CTAS, BF16OUT>;
  static SmemOnce once;
  cudaError_t e = once.set(kern, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t cfg = few_config<NP, CTAS>((unsigned)(tiles * ks), ks, stream, at);
  return cudaLaunchKernelEx(&cfg, kern, tmW, tmX, p);
}

// One CTA per SM has a ring twice as deep, two per SM twice the CTAs to split K
// into.  More than one wave: two (216 row tiles of 5120: 28 us).  Up to 32
// tokens the tails are short and two win wherever K is split (5 x 4096 x 4096:
// 6.4 us, one per SM 6.9; 16 x 14336 x 4096, not split: 13.0 and 12.1 us); above,
// one per SM wins throughout (128 x 5120 x 5120: 11.6 us, two per SM 15.5).
template <int NP, bool BF16OUT>
cudaError_t launch_ctas(const I8GemmArgs& g, int num_sms, cudaStream_t stream) {
  const int64_t tiles = (g.N + W_ROWS - 1) / W_ROWS;
  const bool one = tiles <= num_sms && (NP > 32 || tiles * 2 > num_sms);
  return one ? launch_np<NP, 1, BF16OUT>(g, num_sms, stream) : launch_np<NP, 2, BF16OUT>(g, num_sms, stream);
}

template <bool BF16OUT>
cudaError_t launch_out(const I8GemmArgs& g, int num_sms, cudaStream_t stream) {
  if (g.M <= 16) return launch_ctas<16, BF16OUT>(g, num_sms, stream);
  if (g.M <= 32) return launch_ctas<32, BF16OUT>(g, num_sms, stream);
  if (g.M <= 64) return launch_ctas<64, BF16OUT>(g, num_sms, stream);
  if (g.M <= 128) return launch_ctas<128, BF16OUT>(g, num_sms, stream);
  return launch_np<256, 1, BF16OUT>(g, num_sms, stream);
}

}  // namespace

double i8_gemm_few_ns(int64_t M, int64_t N, int64_t K, int num_sms) {
  const int64_t tiles = (N + W_ROWS - 1) / W_ROWS;
  const int k_steps = (int)((K + BK - 1) / BK), ks = choose_ks<256, 1>(M, tiles, k_steps, num_sms);
  return i8::few_ns(tiles, k_steps, ks, num_sms);
}

cudaError_t launch_i8_gemm_few(const I8GemmArgs& g, int num_sms, cudaStream_t stream) {
  if (g.M > 256) return cudaErrorNotSupported;
  return g.y_bf16 ? launch_out<true>(g, num_sms, stream) : launch_out<false>(g, num_sms, stream);
}

}  // namespace nvfp4
