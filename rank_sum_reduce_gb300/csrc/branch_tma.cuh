// branch_tma.cuh -- a block's branch (branch_rows.cu) for many rows: the rank
// slices and the residual (and a gate of each row's own) stream through a ring
// of shared-memory stages (branch_ring.cuh), the sum of a row stays in registers
// over both of its exchanges, and while one team of warps waits for its row's
// sums another folds.
//
// The rows of weights, and a gate of all rows, lie in shared memory as they are.
//
// What bounds it: HBM with two and more ranks and enough rows (W = 4, M = 8191, N =
// 8192 bf16 with both norms 133 us, 1.04 of a copy's rate; W = 8, M = 3040 83, 0.97; own
// gates W = 2, M = 8192, N = 4096 64, 0.92; W = 1, M = 16389, N = 4096 82, 0.97); with
// few rows per SM whole rows (W = 8, M = 512, N = 8192 17.4, 0.85: 3.4 rows per SM); rows
// that CTAs share, with one rank, their exchanges (N = 16384, M = 1216 32-33, 0.72): a
// CTA has one team then, so nothing folds while the row waits; with one rank and dropout
// instructions (97, 0.82); without a norm W = 1, M = 16389 takes 91 us, longer than with
// one: the CTAs then ask for more of HBM at once (see branch_ring_fit).
#pragma once

#include "branch_ring.cuh"

namespace car {

struct BranchTmaParams {
  RankPtrs in;
  const uint8_t* residual;
  const uint4* weight;
  const uint4* norm_weight;
  const uint4* gate;        // may be null
  uint4* residual_out;
  uint4* norm_out;
  uint4* ar_out;            // may be null
  unsigned int* err;
  DropParams drop;
  float residual_scale;
  float eps, norm_eps;
  float inv_cols;
  int gate_from;
  uint32_t gate_span;       // rows that share a gate row
  unsigned long long wait_ns;  // as in the row kernels, where CTAs share a row
  unsigned long long delay_ns;
  int64_t delay_row;
  int delay_cta;
  RingPlan ring;
};

using BranchTmaFn = void (*)(const BranchTmaParams);
BranchTmaFn branch_tma_bf16(int vpt, bool split, bool norm, int gate, bool drop);
BranchTmaFn branch_tma_fp16(int vpt, bool split, bool norm, int gate, bool drop);
BranchTmaFn branch_tma_fp32(int vpt, bool split, bool norm, int gate, bool drop);

namespace {

__device__ __forceinline__ const uint8_t* slice_source(const BranchTmaParams& p, int q) {
  return q < p.ring.ranks ? static_cast<const uint8_t*>(p.in.p[q])
                          : q == p.ring.ranks ? p.residual : reinterpret_cast<const uint8_t*>(p.gate);
}

// Weight row i (0: weight, 1: norm_weight, 2: a gate of all rows), vector v of this
// CTA's.
__device__ __forceinline__ uint4 weight_at(const BranchTmaParams& p, const uint8_t* s_rows, int i, int v) {
  return lds16(s_rows + 16 * (i * p.ring.chunk + v));
}

template <int DT, int VPT, bool SPLIT, bool NORM, int GATE, bool DROP>
__device__ __forceinline__ void consume(const BranchTmaParams& p, const Part<SPLIT>& part, const uint8_t* ring, const uint8_t* s_rows,
                                        RingShared& s) {
  constexpr int E = Pack<DT>::kN;
  constexpr bool SHARED = GATE == kGateShared;
  const RingPlan& rp = p.ring;
  const bool rows = SHARED && p.gate_from == kFromRows;
  const int T = rp.team_threads, V = part.V;
  const int team = threadIdx.x / T, tid = threadIdx.x - team * T;
  const uint32_t stride = slice_stride(rp);
  const uint8_t* mine = ring + (size_t)team * rp.row_bytes;  // the row in stage 0
  const ClusterWait peers{part.crank, p.wait_ns, p.err};
  const DropState state = drop_state(p.drop);
  bool ok[VPT];
  int col[VPT], at[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    ok[k] = tid + k * T < V;
    col[k] = min(tid + k * T, V - 1);
    at[k] = 16 * col[k];
  }
  RingReader in(rp, s, p.err);
  uint32_t x = 0;
  // With a norm behind the block the second sum of the team's last row travels with the
  // first one of the row after it, so a row passes one barrier instead of two, and its
  // norm_out is stored then: bf16 W = 1, M = 1216, N = 16384 (two CTAs a row) 41.3 ->
  // 35.6 us, M = 1000, N = 32768 (four) 69.9 -> 59.1, M = 8192, N = 1024 16.2 -> 15.2;
  // with many ranks it costs a little (W = 16, M = 1000, N = 4096 26.8 -> 27.6).
  constexpr bool DEFER = NORM;
  float2 last[DEFER ? VPT : 1][E / 2];
  float last_ss = 0.f;
  int64_t last_base = -1;
  auto finish = [&](const float2(&h)[VPT][E / 2], int64_t base, float sum) {
    const float2 r = both(rsqrtf(fmaf(sum, p.inv_cols, p.eps)));
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      float2 f[E / 2];
      widen2<DT>(weight_at(p, s_rows, 0, col[k]), f);
#pragma unroll
      for (int e = 0; e < E / 2; e++) f[e] = mul2(mul2(h[k][e], r), f[e]);
      if (ok[k]) st16(p.norm_out + base + col[k], narrow2<DT>(f));
    }
  };
  for (Tiles<false> t(rp, part); t.more(rp); t.next(rp)) {
    if (team >= t.count(rp)) {
      in.skip();
      continue;
    }
    const int row = t.row + team;
    const int64_t base = (int64_t)row * rp.vec_per_row + part.col0;
    // a shared gate row from L2, asked for before the row's waits where registers allow
    constexpr bool EARLY = SHARED && VPT * E <= 16;
    uint4 gv[EARLY ? VPT : 1];
    const uint4* grow = rows ? p.gate + (int64_t)((uint32_t)row / p.gate_span) * rp.vec_per_row + part.col0 : nullptr;
    if (EARLY && rows) {
#pragma unroll
      for (int k = 0; k < VPT; k++) gv[EARLY ? k : 0] = __ldg(grow + col[k]);
    }
    // the mask's bits, before the row's waits where registers allow: a chain of ten
    // dependent products that would stand between its two exchanges
    constexpr bool BITS_FIRST = DROP && VPT * E <= 16;
    uint32_t bits[BITS_FIRST ? VPT : 1][E / 2];
    if constexpr (BITS_FIRST) {
#pragma unroll
      for (int k = 0; k < VPT; k++) drop_bits_here<E>(state, base + col[k], bits[BITS_FIRST ? k : 0]);
    }
    float2 z[VPT][E / 2];
    const uint8_t* held = ring_rank_sum<DT, VPT, false>(rp, in, mine, ok, at, z);
    if (in.failed) {
#pragma unroll
      for (int k = 0; k < VPT; k++) ok[k] = false;
    }
    if (p.ar_out) {
#pragma unroll
      for (int k = 0; k < VPT; k++)
        if (ok[k]) st16(p.ar_out + base + col[k], narrow2<DT>(z[k]));
    }
    // test hook: this whole CTA reaches the row's first exchange late
    if (SPLIT && part.crank == p.delay_cta && row == p.delay_row) spin_ns(p.delay_ns);
    float2 inv = both(1.f);
    if constexpr (NORM) {
      float v[DEFER ? 2 : 1] = {0.f};
      if constexpr (DEFER) v[DEFER ? 1 : 0] = last_ss;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) ss = fma2(z[k][e], z[k][e], ss);
        v[0] += ok[k] ? ss.x + ss.y : 0.f;
      }
      team_sums<SPLIT>(rp, s, team, x++, v, peers);
      inv = both(rsqrtf(fmaf(v[0], p.inv_cols, p.norm_eps)));
      if constexpr (DEFER) {
        if (last_base >= 0) finish(last, last_base, v[DEFER ? 1 : 0]);
      }
    }
    float hh = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      float2 f[E / 2];
      if constexpr (NORM) {
        // keeps the vectors' arithmetic apart: all at once the CTAs' stores come in
        // bursts where HBM is the limit (W = 1, M = 16389, N = 4096 84.4 us, with this
        // 82.0; N = 5120, W = 2 with one gate row and dropout 76.7 and 72.2)
        __syncwarp();
        widen2<DT>(weight_at(p, s_rows, 1, col[k]), f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[k][e] = mul2(mul2(z[k][e], inv), f[e]);
      }
      if constexpr (GATE != kGateNone) {
        widen2<DT>(GATE == kGateOwn ? lds16(held + stride + at[k])
                   : rows           ? (EARLY ? gv[EARLY ? k : 0] : __ldg(grow + col[k]))
                                    : weight_at(p, s_rows, 2, col[k]),
                   f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[k][e] = mul2(z[k][e], f[e]);
      }
      if constexpr (DROP) {
        if constexpr (!BITS_FIRST) drop_bits<E>(state, base + col[k], bits[0]);
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[k][e] = drop2(p.drop, bits[BITS_FIRST ? k : 0][e], z[k][e]);
      }
      widen2<DT>(lds16(held + at[k]), f);
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < E / 2; e++) {
        z[k][e] = fma2(both(p.residual_scale), f[e], z[k][e]);
        ss = fma2(z[k][e], z[k][e], ss);
      }
      hh += ok[k] ? ss.x + ss.y : 0.f;
      if (ok[k]) st16(p.residual_out + base + col[k], narrow2<DT>(z[k]));
    }
    in.release();
    if constexpr (DEFER) {
#pragma unroll
      for (int k = 0; k < VPT; k++) {
#pragma unroll
        for (int e = 0; e < E / 2; e++) last[k][e] = z[k][e];
      }
      last_base = base;
      last_ss = hh;
    } else {
      float v[1] = {hh};
      team_sums<SPLIT>(rp, s, team, x++, v, peers);
      finish(z, base, v[0]);
    }
  }
  if constexpr (DEFER) {
    if (last_base >= 0) {
      float v[1] = {last_ss};
      team_sums<SPLIT>(rp, s, team, x++, v, peers);
      finish(last, last_base, v[0]);
    }
  }
}

template <int DT, int VPT, bool SPLIT, bool NORM, int GATE, bool DROP>
__global__ void __launch_bounds__(kRingThreads, 1)
    reduce_branch_residual_rmsnorm_tma_kernel(const __grid_constant__ BranchTmaParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RingShared s;
  const RingPlan& rp = p.ring;
  const Part<SPLIT> part(rp);
  uint8_t* s_rows = smem + (size_t)rp.stages * rp.group * slice_stride(rp);
  const int consumers = rp.teams * rp.team_threads, V = part.V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ring_init(rp, s);
  // the first tile into L2 while the previous grid of the stream finishes
  const Tiles<false> first(rp, part);
  if (warp == kRingConsumers / 32 && lane < rp.ranks + rp.held && first.more(rp))
    prefetch_l2(slice_source(p, lane) + first.row * (int64_t)rp.row_bytes + part.col0 * 16,
                (uint32_t)first.count(rp) * (uint32_t)V * 16u);
  if constexpr (SPLIT) cluster_barrier();  // the peers' barriers too
  else __syncthreads();
  pdl_wait_and_release();
  if (warp >= kRingConsumers / 32) {
    take_registers<false>();
    const int who = warp - kRingConsumers / 32;
    if (lane == 0 && who < rp.producers) ring_produce<false>(rp, part, smem, s, who, p.err, [&](int q) { return slice_source(p, q); });
  } else {
    take_registers<true>();
    if (threadIdx.x >= consumers) return;
    uint4* to = reinterpret_cast<uint4*>(s_rows);
    for (int v = threadIdx.x; v < V; v += consumers) {
      to[v] = __ldg(p.weight + part.col0 + v);
      if constexpr (NORM) to[rp.chunk + v] = __ldg(p.norm_weight + part.col0 + v);
      if (GATE && p.gate && p.gate_from == kFromFactor) to[2 * rp.chunk + v] = __ldg(p.gate + part.col0 + v);
    }
    consumers_barrier(rp);
    consume<DT, VPT, SPLIT, NORM, GATE, DROP>(p, part, smem, s_rows, s);
  }
}

template <int DT, int VPT, bool SPLIT, bool NORM, int GATE>
BranchTmaFn pick_drop(bool drop) {
  return drop ? reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, SPLIT, NORM, GATE, true>
              : reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, SPLIT, NORM, GATE, false>;
}
template <int DT, int VPT, bool SPLIT, bool NORM>
BranchTmaFn pick_gate(int gate, bool drop) {
  return gate == kGateNone     ? pick_drop<DT, VPT, SPLIT, NORM, kGateNone>(drop)
         : gate == kGateShared ? pick_drop<DT, VPT, SPLIT, NORM, kGateShared>(drop)
                               : pick_drop<DT, VPT, SPLIT, NORM, kGateOwn>(drop);
}
template <int DT, int VPT, bool SPLIT>
BranchTmaFn pick_norm(bool norm, int gate, bool drop) {
  return norm ? pick_gate<DT, VPT, SPLIT, true>(gate, drop) : pick_gate<DT, VPT, SPLIT, false>(gate, drop);
}
// The instance of a type, in a file of its own: they compile side by side.
template <int DT>
BranchTmaFn pick_instance(int vpt, bool split, bool norm, int gate, bool drop) {
  if (split) return pick_norm<DT, 2, true>(norm, gate, drop);
  if (vpt == 3) return pick_norm<DT, 3, false>(norm, gate, drop);
  return pick_norm<DT, 2, false>(norm, gate, drop);
}

}  // namespace
}  // namespace car
