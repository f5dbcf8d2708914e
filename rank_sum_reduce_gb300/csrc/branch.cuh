// branch.cuh -- what the kernels of a block's branch share (branch_rows.cu,
// branch_tma.cuh, branch_backward.cu, branch_backward_tma.cuh, dropout.cu): the
// dropout's generator, and the sums over a row that is split over warps and a
// cluster of CTAs.
#pragma once

#include "branch.h"
#include "car_device.cuh"

namespace car {
namespace {

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011, section 4.3): ten rounds of two wide products, for the 8
// elements of one counter.  A launch has one key and one offset, and there are
// fewer than 2^32 counters (a handle's data is at most 2^35 bytes), so three of the
// counter's four words are the same for all threads: one product of the first round
// and one of the second are too.  They are taken out of the loops (DropState); the
// other 18, at a quarter of the rate of other instructions, are what the generator
// costs (W = 1, M = 16389, N = 4096 bf16 with both norms: forward 82 us without
// dropout, 97 with it, backward 126 and 148).
struct DropState {
  uint32_t k0, k1;   // the key
  uint32_t z, y, hi, lo;
};
__device__ __forceinline__ DropState drop_state(const DropParams& d) {  // after the wait for the grids it depends on
  const uint64_t offset = d.offset + (d.offset_dev ? *static_cast<const volatile uint64_t*>(d.offset_dev) : 0ull);
  DropState s;
  s.k0 = d.key0;
  s.k1 = d.key1;
  const uint64_t b = (uint64_t)(uint32_t)offset * 0xCD9E8D57u;
  const uint64_t a = (uint64_t)((uint32_t)(b >> 32) ^ s.k0) * 0xD2511F53u;  // of the second round
  s.z = (uint32_t)(offset >> 32) ^ s.k1;
  s.y = (uint32_t)b ^ (s.k0 + 0x9E3779B9u);
  s.hi = (uint32_t)(a >> 32) ^ (s.k1 + 0xBB67AE85u);
  s.lo = (uint32_t)a;
  return s;
}
__device__ __forceinline__ uint4 philox4x32_10(const DropState& s, uint32_t counter) {
  const uint64_t a1 = (uint64_t)counter * 0xD2511F53u;
  const uint64_t b2 = (uint64_t)((uint32_t)(a1 >> 32) ^ s.z) * 0xCD9E8D57u;
  uint4 c = make_uint4((uint32_t)(b2 >> 32) ^ s.y, (uint32_t)b2, s.hi ^ (uint32_t)a1, s.lo);
#pragma unroll
  for (uint32_t r = 2; r < 10; r++) {
    const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
    c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ (s.k0 + r * 0x9E3779B9u), (uint32_t)b,
                   (uint32_t)(a >> 32) ^ c.w ^ (s.k1 + r * 0xBB67AE85u), (uint32_t)a);
  }
  return c;
}

// The 16 random bits of the E elements of the vector `v` of the [M, N] problem
// (v counts 16-byte vectors), two in a word.  A 16-bit type has one counter per
// vector; an fp32 vector is half of one's eight elements.
template <int E>
__device__ __forceinline__ void drop_bits(const DropState& s, int64_t v, uint32_t (&bits)[E / 2]) {
  const uint4 w = philox4x32_10(s, (uint32_t)(E == 8 ? v : v >> 1));
  if constexpr (E == 8) {
    bits[0] = w.x;
    bits[1] = w.y;
    bits[2] = w.z;
    bits[3] = w.w;
  } else {
    bits[0] = (v & 1) ? w.z : w.x;
    bits[1] = (v & 1) ? w.w : w.y;
  }
}

// The same, not to be put off until the bits are used: they are computed here, while
// the row's data is on its way.
template <int E>
__device__ __forceinline__ void drop_bits_here(const DropState& s, int64_t v, uint32_t (&bits)[E / 2]) {
  drop_bits<E>(s, v, bits);
#pragma unroll
  for (int e = 0; e < E / 2; e++) asm volatile("" : "+r"(bits[e]));
}

// Element pair of a word: kept, and scaled, where its 16 bits as the upper half of
// a word exceed the limit; else 0 (selected, not multiplied, so that what is
// dropped may be anything).
__device__ __forceinline__ float2 drop2(const DropParams& d, uint32_t bits, float2 x) {
  const float2 s = mul2(x, make_float2(d.scale, d.scale));
  return make_float2((bits << 16) > d.limit ? s.x : 0.f, bits > d.limit ? s.y : 0.f);
}

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <int DT>
__device__ __forceinline__ void widen2(uint4 v, float2 (&f)[Pack<DT>::kN / 2]) {
  float t[Pack<DT>::kN];
  Pack<DT>::widen(v, t);
#pragma unroll
  for (int e = 0; e < Pack<DT>::kN / 2; e++) f[e] = make_float2(t[2 * e], t[2 * e + 1]);
}
template <int DT>
__device__ __forceinline__ uint4 narrow2(const float2 (&f)[Pack<DT>::kN / 2]) {
  float t[Pack<DT>::kN];
#pragma unroll
  for (int e = 0; e < Pack<DT>::kN / 2; e++) t[2 * e] = f[e].x, t[2 * e + 1] = f[e].y;
  return Pack<DT>::narrow(t);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Sums over a row in the row kernels: warps, then the CTA, then the cluster's
// CTAs, as in fused_rows.cuh.  Every warp adds the warp partials itself, and
// every thread the CTAs', in the same order, so all of the row hold the same
// bits.  `x` counts the exchanges of the CTA; what exchange x writes is next
// written in exchange x + 2, after the CTA's barrier of x + 1, which a thread
// reaches only once it has read x's.
struct RowSums {
  float warp[2][3][32];
  float4 part[2][8];    // the cluster's partials
  uint64_t bar[2];
};

__device__ __forceinline__ void row_sums_init(RowSums& s, int cluster) {  // one thread, before a barrier
  if (cluster > 1) {
    mbar_init(&s.bar[0], 1);
    mbar_init(&s.bar[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
}

// A CTA's wait for its peers' partials; err's bits are car_sync's.
struct ClusterWait {
  int crank;
  uint64_t wait_ns;
  unsigned int* err;
};

// v, the CTA's sums in every thread, becomes the cluster's; NaN for a thread whose
// wait for its peers runs out (it then waits until their partials have landed,
// bounded again, so that none reaches a CTA that has exited and the phases stay in
// step).
template <int NS>
__device__ __forceinline__ void cluster_sums(RowSums& s, float (&v)[NS], uint32_t x, int cluster, const ClusterWait& peers) {
  const int lane = threadIdx.x & 31;
  const uint32_t b = x & 1u, par = (x >> 1) & 1u;
  if (threadIdx.x < 32) {
    constexpr uint32_t bytes = NS == 1 ? 4u : NS == 2 ? 8u : 16u;
    if (lane == 0) mbar_arrive_expect_tx(&s.bar[b], bytes * (uint32_t)cluster);
    if (lane < cluster) {
      const uint32_t to = map_rank(&s.part[b][peers.crank], (uint32_t)lane), bar = map_rank(&s.bar[b], (uint32_t)lane);
      if constexpr (NS == 1) st_async_f32(to, v[0], bar);
      if constexpr (NS > 1) st_async_v2_b32(to, __float_as_uint(v[0]), __float_as_uint(v[1]), bar);
      if constexpr (NS > 2) st_async_v2_b32(to + 8u, __float_as_uint(v[2]), 0u, bar);
    }
  }
  if (wait_cluster_phase(&s.bar[b], par, peers.wait_ns)) {
#pragma unroll
    for (int i = 0; i < NS; i++) v[i] = reinterpret_cast<const float*>(&s.part[b][0])[i];
    for (int r = 1; r < cluster; r++) {
#pragma unroll
      for (int i = 0; i < NS; i++) v[i] += reinterpret_cast<const float*>(&s.part[b][r])[i];
    }
  } else {
    atomicOr(peers.err, 1u);
#pragma unroll
    for (int i = 0; i < NS; i++) v[i] = __int_as_float(0x7fc00000);
    if (!wait_cluster_phase(&s.bar[b], par)) atomicOr(peers.err, 2u);
  }
}

// v becomes the sums over the row, in the row kernels.
template <int NS>
__device__ __forceinline__ void row_sums(RowSums& s, float (&v)[NS], uint32_t x, int cluster, const ClusterWait& peers) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < NS; i++) {
    v[i] = warp_total(v[i]);
    if (lane == 0) s.warp[x & 1u][i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NS; i++) v[i] = warp_total(lane < nwarps ? s.warp[x & 1u][i][lane] : 0.f);
  if (cluster > 1) cluster_sums(s, v, x, cluster, peers);
}

}  // namespace
}  // namespace car
