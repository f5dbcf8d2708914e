// ring.cuh -- bounded waits and bulk copies of the kernels that stream row
// slices through a ring of shared-memory slots (fused_tma.cu, quant_tma.cu,
// norm_backward_tma.cu).
#pragma once

#include "car_device.cuh"

namespace car {
namespace {

// Dynamic shared memory that the pipeline kernels' instances are allowed, the
// most a CTA can have.  The allowance belongs to the kernel, not to a handle:
// were it each handle's own need, a handle made later with a smaller ring
// would take it from the earlier ones.
constexpr int kMaxDynamicSmem = 227 * 1024;

// Threads that issue the bulk copies of a CTA in the kernels whose CTAs work on
// several rows at a time, where it divides the ring's slots.
constexpr int kProducers = 2;

// 16-byte vectors per consumer thread for rows of `vecs` vectors (at most
// 2048), where a CTA's 512 threads are cut into teams of whole warps, one row
// each: the preferred number, unless another of 2 to `most` leaves clearly
// fewer of the threads' places empty (by a tenth).
inline int team_threads(int vecs, int vpt) { return ((vecs + vpt - 1) / vpt + 31) / 32 * 32; }
inline double team_use(int vecs, int vpt) {
  const int t = team_threads(vecs, vpt);
  return t > 512 ? 0.0 : (double)(512 / t) * vecs / (512.0 * vpt);
}
inline int team_vectors(int vecs, int prefer, int most) {
  int best = prefer;
  double use = team_use(vecs, prefer) + 0.1;
  for (int vpt = 2; vpt <= most; vpt++) {
    if (team_use(vecs, vpt) > use) {
      best = vpt;
      use = team_use(vecs, vpt);
    }
  }
  return best;
}

// A row of weights in shared memory, widened (WIDE, 16-bit types): the vectors'
// halves lie in two planes of float4, so that a warp that takes consecutive
// vectors reads either without bank conflicts.  By the first `threads` threads.
template <int DT, bool WIDE>
__device__ __forceinline__ void weight_to_shared(const uint4* __restrict__ weight, int vecs, int threads, uint8_t* s) {
  for (int v = threadIdx.x; v < vecs; v += threads) {
    const uint4 w = __ldg(weight + v);
    if constexpr (WIDE) {
      float f[8];
      Pack<DT>::widen(w, f);
      reinterpret_cast<float4*>(s)[v] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(s)[vecs + v] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      reinterpret_cast<uint4*>(s)[v] = w;
    }
  }
}
__device__ __forceinline__ void lds_wide(const uint8_t* s, int vecs, int v, float2 (&f)[4]) {
  const float4 a = reinterpret_cast<const float4*>(s)[v], b = reinterpret_cast<const float4*>(s)[vecs + v];
  f[0] = make_float2(a.x, a.y);
  f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y);
  f[3] = make_float2(b.z, b.w);
}

// Wait for the barrier phase with the given parity; false when the CTA is
// aborting or the wait ran past kWaitLimitNs.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (uint32_t i = 1; i < (1u << 30); i++) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0 && (*abort || globaltimer() - t0 > kWaitLimitNs)) return false;
  }
  return false;
}
// Same, ignoring the abort flag (used while draining on the way out).
__device__ __forceinline__ bool wait_bounded_cluster(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (uint32_t i = 1; i < (1u << 30); i++) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((i & 63u) == 0 && (*abort || globaltimer() - t0 > kWaitLimitNs)) return false;
  }
  return false;
}
__device__ __forceinline__ bool wait_bounded_drain(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (uint32_t i = 1; i < (1u << 30); i++) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0 && globaltimer() - t0 > kWaitLimitNs) return false;
  }
  return false;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ uint4 lds16(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

}  // namespace
}  // namespace car
