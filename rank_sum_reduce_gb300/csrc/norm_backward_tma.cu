// norm_backward_tma.cu -- backward of rank sum + residual add + RMSNorm for
// many rows, with the rows streamed into shared memory by TMA bulk copies.
// Same operation as norm_backward.cu, in the manner of the forward's pipeline
// kernel (fused_tma.cu): one persistent CTA per SM, a producer thread that
// keeps a ring of slices in flight -- dy_0 .. dy_{W-1}, h, dres -- and
// consumer warps that fold them into fp32 accumulators in rank order.
//
// A CTA takes tiles of `teams` consecutive rows (tile blockIdx.x, blockIdx.x +
// grid, ...).  A tile's rows lie next to each other in every buffer, so one
// bulk copy brings the same slice of all of them: one thread issues about one
// copy per 0.3 us whatever its size, so short rows need their slices joined to
// keep HBM busy.  Each team of consumer warps owns one row of the tile, with
// its own statistic and barrier: while one team is in the serial part of its
// row another folds.
//
// h stays in registers (packed) from the statistic to the gradient, or, with
// more than three vectors per thread, in its slot; the dres slice is only
// waited for after the statistic and is read from its slot there.  The weight
// row lies in shared memory, the weight gradient of a team's rows in its
// registers for the whole kernel; the teams' are added in shared memory at the
// end, one partial per CTA.  Every mbarrier wait is bounded, as in the forward.
#include "car_launch.h"
#include "ring.cuh"

namespace car {
namespace {

struct BackwardTmaParams {
  RankPtrs dy;
  const uint8_t* h;
  const uint8_t* dres;  // may be null
  const uint4* weight;
  uint4* dx;
  float* partial;       // [grid, N], or null
  unsigned int* err;
  float eps;
  float inv_cols;
  int64_t rows;
  int row_bytes;
  int vec_per_row;
  int slots;
  int slices;           // of a tile: W ranks, h, dres
  int teams;            // rows of a tile
  uint32_t producers;   // 1 or 2
  int team_threads;     // multiple of 32
  int nranks;
};

__device__ __forceinline__ const uint8_t* slice_source(const BackwardTmaParams& p, int q) {
  return q < p.nranks ? static_cast<const uint8_t*>(p.dy.p[q]) : (q == p.nranks ? p.h : p.dres);
}
// Bytes of one slice of the tile that starts at `row`.
__device__ __forceinline__ uint32_t tile_bytes(const BackwardTmaParams& p, int64_t row) {
  const int64_t left = p.rows - row;
  return (uint32_t)(left < p.teams ? left : p.teams) * (uint32_t)p.row_bytes;
}

// Producer `who` of p.producers, each in a warp of its own: issues every
// p.producers-th copy of the CTA's sequence (copy c fills slot c % S as its use
// c / S), then waits for the copies that it issued.  S is a multiple of
// p.producers, so a slot is always filled by the same one: a producer that
// could run ahead of a slot's previous use would take that use's parity for
// its own.  Two measured up to 4 % faster than one with eight ranks and more,
// four slower (W = 16, M = 512, N = 8192 bf16 31.4 / 30.9 / 30.9 us, W = 4, M =
// 2000 40.7 / 40.8 / 45.9); h and dres loaded by the consumers instead were
// slower too (W = 8, M = 512 20.4 against 19.8).
__device__ __forceinline__ void produce(const BackwardTmaParams& p, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                        volatile int* s_abort, uint32_t who) {
  const int S = p.slots;
  const size_t stride = (size_t)p.teams * p.row_bytes;
  int slot = 0;
  uint32_t phase = 0;
  uint64_t issued = 0;
  bool ok = true;
  for (int64_t row = (int64_t)blockIdx.x * p.teams; row < p.rows && ok; row += (int64_t)gridDim.x * p.teams) {
    const int64_t off = row * (int64_t)p.row_bytes;
    const uint32_t bytes = tile_bytes(p, row);
    for (int q = 0; q < p.slices; q++) {
      if (((uint32_t)issued & (p.producers - 1u)) == who) {
        if (issued >= (uint64_t)S && !wait_bounded(&empty[slot], phase ^ 1u, s_abort)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[slot], bytes);
        bulk_load(ring + slot * stride, slice_source(p, q) + off, bytes, &full[slot]);
      }
      issued++;
      if (++slot == S) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  if (!ok) {
    atomicOr(p.err, 1u);
    *s_abort = 1;
  }
  const int used = issued < (uint64_t)S ? (int)issued : S;
  for (int k = 0; k < used; k++) {  // copy number c is use c / S of slot c % S
    const uint64_t c = issued - 1 - (uint64_t)k;
    if (((uint32_t)c & (p.producers - 1u)) != who) continue;
    if (!wait_bounded_drain(&full[c % (uint64_t)S], (uint32_t)((c / (uint64_t)S) & 1u))) atomicOr(p.err, 1u);
  }
}

// The lower half of the warp adds one sum, the upper half another; both to all
// lanes: five shuffles where two sums after one another take eight.
__device__ __forceinline__ float2 half_sums(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  const float other = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
  return (threadIdx.x & 16) ? make_float2(other, v) : make_float2(v, other);
}
__device__ __forceinline__ float2 warp_sum2(float a, float b) {
  const bool upper = threadIdx.x & 16;
  const float other = __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
  return half_sums(__fadd_rn(upper ? b : a, other));
}

// The weight row lies widened in shared memory where that costs no slots: every
// vector is used twice, and widening takes eight instructions of the hundred or
// so that a vector needs, where the instructions are what bounds rows of few
// ranks (with the sums' shared shuffles W = 1, M = 16389, N = 4096 87.0 -> 82.5
// us, W = 4, M = 4085, N = 10488 100.5 -> 92.2).  Three vectors per thread gain
// nothing more by it (W = 3, N = 10000 43.4 / 43.3), four lose (W = 4, N = 14000
// 138 / 168).
template <int DT, int VPT>
constexpr bool kWideWeight = DT != kFP32 && VPT == 2;
template <int DT, int VPT>
__device__ __forceinline__ int weight_row_bytes(int row_bytes) {
  return VPT > 4 ? 0 : kWideWeight<DT, VPT> ? 2 * row_bytes : row_bytes;
}

// VPT: vectors per consumer thread.  Two for rows of up to 1024 vectors: with
// one, the fixed work of a row (two sums over the warp, a barrier, addresses)
// is done twice as often (W = 1, M = 16389, N = 4096 bf16: 82 against 135 us).
// Three for longer rows, and where two would leave a third of the threads
// without a row (W = 8, M = 1500, N = 4400: 27.4 against 34.4; N = 7000, where
// two fit better, 43.0 against 39.6).  Four only for rows that three do not
// hold: in 16 bits the accumulators leave little room to overlap (N = 4400:
// 36.3).  Five to eight above that, as few as 512 threads need (W = 1, M = 3000,
// N = 9000: five 81 us, six 98, eight 115), in fp32 alone: more than four
// 16-bit vectors' accumulators would not fit in registers.  Of 96, which leave
// room for a CTA of 18 warps, four 16-bit vectors spill 36 bytes, six, seven and
// eight fp32 ones 28, 52 and 340.
template <int DT, int VPT>
__device__ __forceinline__ void consume(const BackwardTmaParams& p, uint8_t* ring, const uint8_t* s_weight, uint64_t* full,
                                        uint64_t* empty, uint64_t* rowbar, uint64_t* done, float2* s_warp,
                                        volatile int* s_abort) {
  constexpr int E = Pack<DT>::kN;
  const int S = p.slots, T = p.team_threads, n = p.nranks;
  const int team = threadIdx.x / T, tid = threadIdx.x - team * T;
  const int warp = tid >> 5, lane = threadIdx.x & 31, nwarps = T >> 5;
  const size_t stride = (size_t)p.teams * p.row_bytes;
  const uint8_t* mine = ring + (size_t)team * p.row_bytes + 16 * tid;  // this thread's first vector in slot 0
  rowbar += team;
  s_warp += team * 2 * nwarps;
  float2 dw[VPT][E / 2];
  bool ok[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    ok[k] = tid + k * T < p.vec_per_row;
#pragma unroll
    for (int e = 0; e < E / 2; e++) dw[k][e] = make_float2(0.f, 0.f);
  }
  int slot = 0;
  uint32_t phase = 0, it = 0;
  bool failed = false;
  auto advance = [&] {
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
  };
  auto release = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    advance();
  };
  auto widen2 = [](uint4 v, float2 (&f)[E / 2]) {
    float t[E];
    Pack<DT>::widen(v, t);
#pragma unroll
    for (int e = 0; e < E / 2; e++) f[e] = make_float2(t[2 * e], t[2 * e + 1]);
  };
  auto weight = [&](int k, float2 (&f)[E / 2]) {
    const int v = tid + k * T;
    if constexpr (kWideWeight<DT, VPT>) lds_wide(s_weight, p.vec_per_row, v, f);
    else if constexpr (VPT <= 4) widen2(lds16(s_weight + 16 * v), f);
    else widen2(__ldg(p.weight + v), f);
  };
  for (int64_t tile = (int64_t)blockIdx.x * p.teams; tile < p.rows; tile += (int64_t)gridDim.x * p.teams) {
    const int64_t row = tile + team;
    if (row >= p.rows) {  // a team without a row in the last tile only lets the slots go
      for (int q = 0; q < p.slices && !failed; q++) {
        failed = !wait_bounded(&full[slot], phase, s_abort);
        if (!failed) release();
      }
      break;
    }
    constexpr bool HELD = VPT > 3;  // h is read again from its slot
    float2 g[VPT][E / 2];
    uint4 hv[HELD ? 1 : VPT];
    float2 ss = make_float2(0.f, 0.f), c = make_float2(0.f, 0.f);
    for (int q = 0; q < n; q++) {
      if (!wait_bounded(&full[slot], phase, s_abort)) {
        failed = true;
        break;
      }
      const uint8_t* sl = mine + slot * stride;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (ok[k]) {
          float2 t[E / 2];
          widen2(lds16(sl + 16 * k * T), t);
#pragma unroll
          for (int e = 0; e < E / 2; e++) g[k][e] = q == 0 ? t[e] : add2(g[k][e], t[e]);
        }
      }
      release();
    }
    if (failed || !wait_bounded(&full[slot], phase, s_abort)) {
      failed = true;
      break;
    }
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        const uint4 v = lds16(mine + slot * stride + 16 * k * T);
        if constexpr (!HELD) hv[k] = v;
        float2 hf[E / 2], wf[E / 2];
        widen2(v, hf);
        weight(k, wf);
#pragma unroll
        for (int e = 0; e < E / 2; e++) {
          ss = fma2(hf[e], hf[e], ss);
          c = fma2(mul2(g[k][e], wf[e]), hf[e], c);
        }
      }
    }
    const int hslot = slot;
    if constexpr (HELD) {
      advance();
    } else {
      release();
    }
    // row statistics: every warp adds the team's warp partials itself, in the
    // same order; they are double-buffered by row parity
    float2 sum = warp_sum2(ss.x + ss.y, c.x + c.y);
    if (nwarps > 1) {
      float2* sw = s_warp + nwarps * (it & 1u);
      if (lane == 0) {
        sw[warp] = sum;
        mbar_arrive(rowbar);
      }
      if (!wait_bounded(rowbar, it & 1u, s_abort)) {
        failed = true;
        break;
      }
      sum = half_sums((lane & 15) < nwarps ? reinterpret_cast<const float*>(sw)[2 * (lane & 15) + (lane >> 4)] : 0.f);
    }
    it++;
    const float rms = rsqrtf(fmaf(sum.x, p.inv_cols, p.eps));
    const float m = __fmul_rn(__fmul_rn(sum.y, p.inv_cols), rms);
    const float2 rms2 = make_float2(rms, rms), m2 = make_float2(-m, -m);
    if (p.dres && !wait_bounded(&full[slot], phase, s_abort)) {
      failed = true;
      break;
    }
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        float2 hf[E / 2], wf[E / 2], df[E / 2];
        float o[E];
        widen2(HELD ? lds16(mine + hslot * stride + 16 * k * T) : hv[HELD ? 0 : k], hf);
        weight(k, wf);
        widen2(p.dres ? lds16(mine + slot * stride + 16 * k * T) : make_uint4(0u, 0u, 0u, 0u), df);
#pragma unroll
        for (int e = 0; e < E / 2; e++) {
          const float2 u = mul2(hf[e], rms2);
          dw[k][e] = fma2(g[k][e], u, dw[k][e]);
          const float2 x = fma2(rms2, fma2(u, m2, mul2(g[k][e], wf[e])), df[e]);
          o[2 * e] = x.x;
          o[2 * e + 1] = x.y;
        }
        st16(p.dx + row * (int64_t)p.vec_per_row + tid + k * T, Pack<DT>::narrow(o));
      }
    }
    if constexpr (HELD) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[hslot]);
    }
    if (p.dres) release();
  }
  if (!p.partial) {
    if (failed) {
      atomicOr(p.err, 1u);
      *s_abort = 1;
    }
    return;
  }
  // The weight gradients of the teams, added in team order by the first one:
  // the others leave theirs in the ring once every team is past its last slot.
  if (p.teams > 1 && !failed) {
    if (lane == 0) mbar_arrive(&done[0]);
    failed = !wait_bounded(&done[0], 0u, s_abort);
    if (!failed) {
      float* at = reinterpret_cast<float*>(ring) + (size_t)(team - 1) * p.vec_per_row * E;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (ok[k] && team > 0) {
#pragma unroll
          for (int e = 0; e < E / 2; e += 2)
            *reinterpret_cast<float4*>(at + (tid + k * T) * E + 2 * e) =
                make_float4(dw[k][e].x, dw[k][e].y, dw[k][e + 1].x, dw[k][e + 1].y);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&done[1]);
      failed = !wait_bounded(&done[1], 0u, s_abort);
    }
  }
  if (failed) {
    atomicOr(p.err, 1u);
    *s_abort = 1;
    return;
  }
  if (team > 0) return;
  float* to = p.partial + blockIdx.x * (int64_t)p.vec_per_row * E;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    if (ok[k]) {
      const int col = (tid + k * T) * E;
#pragma unroll
      for (int e = 0; e < E / 2; e += 2) {
        float4 a = make_float4(dw[k][e].x, dw[k][e].y, dw[k][e + 1].x, dw[k][e + 1].y);
        for (int t = 1; t < p.teams; t++) {
          const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring) +
                                                            (size_t)(t - 1) * p.vec_per_row * E + col + 2 * e);
          a.x += b.x;
          a.y += b.y;
          a.z += b.z;
          a.w += b.w;
        }
        *reinterpret_cast<float4*>(to + col + 2 * e) = a;
      }
    }
  }
}

template <int DT, int VPT>
__global__ void __launch_bounds__(512 + 32 * kProducers, 1) reduce_rmsnorm_backward_tma_kernel(const BackwardTmaParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int S = p.slots;
  uint8_t* s_weight = smem + (size_t)S * p.teams * p.row_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_weight + weight_row_bytes<DT, VPT>(p.row_bytes));
  uint64_t* empty = full + S;
  uint64_t* rowbar = empty + S;             // [16], by team
  uint64_t* done = rowbar + 16;             // [2]
  float2* s_warp = reinterpret_cast<float2*>(done + 2);  // [teams][2][warps of a team]: 32 at most
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_warp + 32);
  const int consumers = p.teams * p.team_threads, nwarps = consumers >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], (uint32_t)nwarps);
    }
    for (int t = 0; t < p.teams; t++) mbar_init(&rowbar[t], (uint32_t)(p.team_threads >> 5));
    mbar_init(&done[0], (uint32_t)nwarps);
    mbar_init(&done[1], (uint32_t)nwarps);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the first tile into L2 while the previous grid of the stream finishes
  const int64_t first = (int64_t)blockIdx.x * p.teams;
  if (warp == nwarps && lane < p.slices)
    prefetch_l2(slice_source(p, lane) + first * (int64_t)p.row_bytes, tile_bytes(p, first));
  __syncthreads();
  pdl_wait_and_release();
  if (warp >= nwarps) {
    if (lane == 0) produce(p, smem, full, empty, s_abort, warp - nwarps);
  } else {
    if constexpr (VPT <= 4) {
      weight_to_shared<DT, kWideWeight<DT, VPT>>(p.weight, p.vec_per_row, consumers, s_weight);
      asm volatile("bar.sync 1, %0;" ::"r"(consumers) : "memory");
    }
    consume<DT, VPT>(p, smem, s_weight, full, empty, rowbar, done, s_warp, s_abort);
  }
}

using BackwardTmaFn = void (*)(const BackwardTmaParams);

template <int DT>
BackwardTmaFn pick_vpt(int vpt) {
  if (vpt == 2) return reduce_rmsnorm_backward_tma_kernel<DT, 2>;
  if (vpt == 3) return reduce_rmsnorm_backward_tma_kernel<DT, 3>;
  if (vpt == 4) return reduce_rmsnorm_backward_tma_kernel<DT, 4>;
  if constexpr (DT == kFP32) {
    if (vpt == 5) return reduce_rmsnorm_backward_tma_kernel<DT, 5>;
    if (vpt == 6) return reduce_rmsnorm_backward_tma_kernel<DT, 6>;
    if (vpt == 7) return reduce_rmsnorm_backward_tma_kernel<DT, 7>;
    return reduce_rmsnorm_backward_tma_kernel<DT, 8>;
  }
  return nullptr;
}
BackwardTmaFn pick(int dtype, int vpt) {
  switch (dtype) {
    case kBF16: return pick_vpt<kBF16>(vpt);
    case kFP16: return pick_vpt<kFP16>(vpt);
    default: return pick_vpt<kFP32>(vpt);
  }
}

constexpr int kRingBudget = 224 * 1024;  // ring and weight row

}  // namespace

bool backward_tma_shape(int dtype, int64_t rows, int vec_per_row, int num_sms, int W, TeamShape* out) {
  const int row_bytes = vec_per_row * 16;
  const int vpt = vec_per_row > 2048 ? (vec_per_row + 511) / 512 : team_vectors(vec_per_row, 2, vec_per_row > 1536 ? 4 : 3);
  if (vpt > (dtype == kFP32 ? 8 : 4)) return false;
  out->vpt = vpt;
  out->use = team_use(vec_per_row, vpt);
  out->team_threads = team_threads(vec_per_row, vpt);
  if (out->team_threads > 512) return false;
  const int teams = 512 / out->team_threads;
  out->teams = teams;
  // about one tile's slices in flight, as in the forward, and an even number
  const int slice = teams * row_bytes, weights = vpt > 4 ? 0 : vpt == 2 && dtype != kFP32 ? 2 * row_bytes : row_bytes;
  int slots = W + 2 < 6 ? 6 : (W + 3) / 2 * 2;
  if (slots > (kRingBudget - weights) / slice) slots = (kRingBudget - weights) / slice;
  if (slots > 4) slots -= slots % kProducers;
  out->producers = slots % kProducers == 0 ? kProducers : 1;
  out->slots = slots;
  const int64_t tiles = (rows + teams - 1) / teams;
  out->grid = (int)(tiles < num_sms ? tiles : num_sms);
  // the ring also takes the teams' weight gradients at the end
  if (slots < 2 || (int64_t)(teams - 1) * vec_per_row * 8 * 4 > (int64_t)slots * slice) return false;
  out->smem = slots * slice + weights + (2 * slots + 18) * 8 + 32 * 8 + 16;
  return true;
}

cudaError_t backward_tma_prepare(int dtype, const TeamShape& sh) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(pick(dtype, sh.vpt)), cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kMaxDynamicSmem);
}

cudaError_t launch_backward_tma(int dtype, int W, const RankPtrs& dy, const void* h, const void* weight, float eps,
                                const void* dres, void* dx, float* dweight, float* workspace, unsigned int* err,
                                int64_t rows, int64_t cols, int vec_per_row, const TeamShape& sh, cudaStream_t s) {
  BackwardTmaParams p;
  p.dy = dy;
  p.h = static_cast<const uint8_t*>(h);
  p.dres = static_cast<const uint8_t*>(dres);
  p.weight = static_cast<const uint4*>(weight);
  p.dx = static_cast<uint4*>(dx);
  p.partial = dweight ? (sh.grid > 1 ? workspace : dweight) : nullptr;
  p.err = err;
  p.eps = eps;
  p.inv_cols = 1.f / (float)cols;
  p.rows = rows;
  p.row_bytes = vec_per_row * 16;
  p.vec_per_row = vec_per_row;
  p.slots = sh.slots;
  p.slices = W + 1 + (dres ? 1 : 0);
  p.teams = sh.teams;
  p.producers = (uint32_t)sh.producers;
  p.team_threads = sh.team_threads;
  p.nranks = W;
  const unsigned threads = (unsigned)(sh.teams * sh.team_threads + 32 * sh.producers);
  cudaError_t e = launch_pdl(pick(dtype, sh.vpt), (unsigned)sh.grid, threads, (size_t)sh.smem, s, 1, p);
  if (e != cudaSuccess || !dweight || sh.grid == 1) return e;
  return launch_sum_partials(workspace, dweight, sh.grid, cols, s);
}

}  // namespace car
