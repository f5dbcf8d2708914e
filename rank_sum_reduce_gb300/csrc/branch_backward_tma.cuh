// branch_backward_tma.cuh -- backward of a block's branch (branch_backward.cu)
// for many rows: the slices dy_0 .. dy_{W-1}, h, the stored sum, the skip
// gradient and a gate of each row's own stream through a ring of shared-memory
// stages (branch_ring.cuh).  The sum of dy stays in registers and becomes dh, dz
// and v in turn; the others are read again from their stage, which is held to the
// row's end.
//
// The weight and the factor norm_weight * gate row lie in shared memory, in fp32, or
// packed (PACK; not the product) where two tiles do not fit and the ring gets deeper:
// bf16 with both norms, W = 4, M = 1216, N = 16384 81.5 us in fp32, 67.0 packed; M =
// 2000, N = 8192 62.2 and 53.4; W = 8, M = 512 29.0 and 27.5.  Where two tiles fit it
// changes little (W = 1, M = 1216, N = 16384 58.7 and 58.4, with dropout 65.4 and 67.0).
// In an instance of its own: chosen at run time it spills (W = 1, M = 16389, N = 4096
// with dropout 147 us against 169).
//
// The factor is made anew for each gate row: two barriers and an L2 latency, which cost
// less than the gate read from L2 and another product for every row even where four
// rows share one (bf16 with norms, W = 1, M = 16384, N = 4096: 16 gate rows 146 us
// against 166, 4096 of them 238 against 255; W = 4, M = 2048, N = 2048 fp32, a gate
// row for each row, 59 against 64).
//
// Column sums.  A thread sums g u and t (or gate t, where no gate row is shared)
// over its team's rows in registers.  Where rows share a gate row, tiles end with
// it: the teams' sums of t are then added in shared memory in team order, leave
// as dgate or as a partial of the span (as in the row kernel), and gate * t is
// added to the span's partial of dnorm_weight, where each column has one owner.
// (That sum in shared memory left the ring no room for two tiles: W = 1, M = 1216, N =
// 16384 bf16 with norms and one gate row 87 us against 66.)
#pragma once

#include "branch_ring.cuh"

namespace car {

struct BranchBackwardTmaParams {
  RankPtrs dy;
  const uint8_t* h;
  const uint8_t* ar;         // may be null
  const uint8_t* dres;       // may be null
  const uint4* weight;
  const uint4* norm_weight;
  const uint4* gate;         // may be null
  uint4* dx;
  uint4* dresidual;          // may be null
  uint4* dgate_own;          // [M, N], or null
  float* dgate;              // as in the row kernel
  float* part_w;
  float* part_w1;
  float* part_gate;
  unsigned int* err;
  DropParams drop;
  float residual_scale;
  float eps, norm_eps;
  float inv_cols;
  uint32_t gate_span;        // rows that share a gate row
  uint32_t first_vec;        // of the [M, N] problem's vectors: this launch's first
  bool shared;               // t is summed by gate row
  int factor_at, sums_at;    // the factor and the teams' sums behind the weight, in bytes
  unsigned long long wait_ns;  // as in the row kernels, where CTAs share a row
  unsigned long long delay_ns;
  int64_t delay_row;
  int delay_cta;
  int a_at, d_at, g_at;      // the stored sum, dres and gate behind h in their stage, in bytes
  RingPlan ring;
};

using BackwardTmaFn = void (*)(const BranchBackwardTmaParams);
BackwardTmaFn branch_backward_tma_bf16(bool split, bool norm, int gate, bool drop);
BackwardTmaFn branch_backward_tma_fp16(bool split, bool norm, int gate, bool drop);
BackwardTmaFn branch_backward_tma_fp32(bool split, bool norm, int gate, bool drop);
// With a norm, weights packed.
BackwardTmaFn branch_backward_tma_packed_bf16(bool split, int gate, bool drop);
BackwardTmaFn branch_backward_tma_packed_fp16(bool split, int gate, bool drop);

namespace {

// Slices of a tile: the ranks, h, then those of ar, dres and the gate that there are.
__device__ __forceinline__ const uint8_t* slice_source(const BranchBackwardTmaParams& p, int q) {
  if (q < p.ring.ranks) return static_cast<const uint8_t*>(p.dy.p[q]);
  q -= p.ring.ranks;
  if (q == 0) return p.h;
  if (p.ar && --q == 0) return p.ar;
  if (p.dres && --q == 0) return p.dres;
  return reinterpret_cast<const uint8_t*>(p.gate);
}

// A row of weights in shared memory, and vector v of it.
template <int DT, bool PACK>
__device__ __forceinline__ void weights_to_shared(const uint4* __restrict__ row, int vecs, int threads, uint8_t* to) {
  if constexpr (PACK)
    for (int v = threadIdx.x; v < vecs; v += threads) reinterpret_cast<uint4*>(to)[v] = __ldg(row + v);
  else
    row_to_shared<DT>(row, nullptr, vecs, threads, to);
}
template <int DT, bool PACK>
__device__ __forceinline__ void weight_at(const uint8_t* row, int vecs, int v, float2 (&f)[Pack<DT>::kN / 2]) {
  if constexpr (PACK) widen2<DT>(lds16(row + 16 * v), f);
  else row_from_shared<DT>(row, vecs, v, f);
}

template <int DT, int VPT, bool SPLIT, bool NORM, int GATE, bool DROP, bool PACK>
__device__ __forceinline__ void consume(const BranchBackwardTmaParams& p, const Part<SPLIT>& part, const uint8_t* ring, const uint8_t* s_rows,
                                        uint8_t* s_factor, float4* s_comb, RingShared& s) {
  constexpr int E = Pack<DT>::kN;
  constexpr bool SHARED = GATE == kGateShared;
  constexpr bool FACTOR = NORM || SHARED;  // dz is multiplied by a factor row: norm_weight, the gate row or both
  // Else they spill (bf16 with norms: W = 1, M = 8192, N = 2048, own gates and dropout 47.8
  // us with branches, 65.3 without; W = 8, M = 608, N = 16384, eight gate rows 66 and 70);
  // own gates without dropout do not (M = 1216, N = 16384 70 and 64).
  constexpr bool BRANCHES = E == 8 && (SHARED || (NORM && GATE == kGateOwn && DROP));
  const RingPlan& rp = p.ring;
  const bool shared = SHARED && p.shared;
  const int T = rp.team_threads, V = part.V, teams = SPLIT ? 1 : rp.teams;
  const ClusterWait peers{part.crank, p.wait_ns, p.err};
  const int team = SPLIT ? 0 : threadIdx.x / T, tid = threadIdx.x - team * T;
  const uint8_t* mine = ring + (size_t)team * rp.row_bytes;  // the row in stage 0
  float2 dw[VPT][E / 2], ts[VPT][E / 2];
  bool ok[VPT];
  int col[VPT], at[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    ok[k] = tid + k * T < V;
    col[k] = min(tid + k * T, V - 1);
    at[k] = 16 * col[k];
#pragma unroll
    for (int e = 0; e < E / 2; e++) dw[k][e] = ts[k][e] = make_float2(0.f, 0.f);
  }
  // Adds the teams' sums of every column in team order and hands each column's
  // four to `take`, in the same thread every time.
  auto combine = [&](float2 (&acc)[VPT][E / 2], auto take) {
    if (teams == 1) {
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (ok[k]) {
#pragma unroll
          for (int e = 0; e < E / 2; e += 2)
            take(col[k] * (E / 4) + e / 2, make_float4(acc[k][e].x, acc[k][e].y, acc[k][e + 1].x, acc[k][e + 1].y));
        }
      }
      return;
    }
    float4* to = s_comb + (size_t)team * V * (E / 4);
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
#pragma unroll
        for (int e = 0; e < E / 2; e += 2)
          to[col[k] * (E / 4) + e / 2] = make_float4(acc[k][e].x, acc[k][e].y, acc[k][e + 1].x, acc[k][e + 1].y);
      }
    }
    consumers_barrier(rp);
    for (int i = threadIdx.x; i < V * (E / 4); i += teams * T) {
      float4 a = s_comb[i];
      for (int k = 1; k < teams; k++) {
        const float4 b = s_comb[(size_t)k * V * (E / 4) + i];
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
      }
      take(i, a);
    }
    consumers_barrier(rp);  // before the teams' next sums
  };
  // Columns 4 i .. 4 i + 3 of a row of T.
  auto four = [&](const uint4* row, int i) {
    if constexpr (E == 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(row) + i);
      return f;
    } else {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(row) + i);
      float f[8];
      Pack<DT>::widen(make_uint4(w.x, w.y, 0u, 0u), f);
      return make_float4(f[0], f[1], f[2], f[3]);
    }
  };
  auto plane = [&] { return (int64_t)part.group * rp.vec_per_row * (E / 4) + part.col0 * (E / 4); };
  // ts holds all rows of gate row b (whole), or those of this span: its first gate row
  // (slot 0) or its last (1)
  auto flush = [&](uint32_t b, bool whole, int slot) {
    float4* out = nullptr;
    if (p.dgate)
      out = reinterpret_cast<float4*>(whole ? p.dgate : p.part_gate) +
            (whole ? (int64_t)b : 2 * (int64_t)part.group + slot) * rp.vec_per_row * (E / 4) + part.col0 * (E / 4);
    combine(ts, [&](int i, float4 t) {
      if (NORM && p.part_w1) {
        const float4 g = four(p.gate + (int64_t)b * rp.vec_per_row + part.col0, i);
        float4* to = reinterpret_cast<float4*>(p.part_w1) + plane() + i;
        float4 d = slot == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *to;
        d.x = fmaf(g.x, t.x, d.x);
        d.y = fmaf(g.y, t.y, d.y);
        d.z = fmaf(g.z, t.z, d.z);
        d.w = fmaf(g.w, t.w, d.w);
        *to = d;
      }
      if (!out) return;
      if (NORM && whole) {
        const float4 w = four(p.norm_weight + part.col0, i);
        t = make_float4(t.x * w.x, t.y * w.y, t.z * w.z, t.w * w.w);
      }
      out[i] = t;
    });
#pragma unroll
    for (int k = 0; k < VPT; k++) {
#pragma unroll
      for (int e = 0; e < E / 2; e++) ts[k][e] = make_float2(0.f, 0.f);
    }
  };

  RingReader in(rp, s, p.err);
  uint32_t x = 0;
  for (Tiles<SHARED> t(rp, part); t.more(rp);) {
    const int tile = t.row;
    if (team >= t.count(rp)) {
      in.skip();
    } else {
      const int row = tile + team;
      const int64_t base = (int64_t)row * rp.vec_per_row + part.col0;
      float2 g[VPT][E / 2];
      const uint8_t* held = ring_rank_sum<DT, VPT, BRANCHES>(rp, in, mine, ok, at, g);
      if (in.failed) {
#pragma unroll
        for (int k = 0; k < VPT; k++) ok[k] = false;
      }
      // test hook: this whole CTA reaches the row's first exchange late
      if (SPLIT && part.crank == p.delay_cta && row == p.delay_row) spin_ns(p.delay_ns);
      float hh = 0.f, gwh = 0.f, aa = 0.f;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (!BRANCHES || ok[k]) {
          float2 hf[E / 2], wf[E / 2], sh = make_float2(0.f, 0.f), sg = sh, sa = sh;
          widen2<DT>(lds16(held + at[k]), hf);
          weight_at<DT, PACK>(s_rows, V, col[k], wf);
#pragma unroll
          for (int e = 0; e < E / 2; e++) {
            sh = fma2(hf[e], hf[e], sh);
            sg = fma2(mul2(g[k][e], wf[e]), hf[e], sg);
          }
          if constexpr (NORM) {
            widen2<DT>(lds16(held + p.a_at + at[k]), hf);
#pragma unroll
            for (int e = 0; e < E / 2; e++) sa = fma2(hf[e], hf[e], sa);
          }
          hh += ok[k] ? sh.x + sh.y : 0.f;
          gwh += ok[k] ? sg.x + sg.y : 0.f;
          aa += ok[k] ? sa.x + sa.y : 0.f;
        }
      }
      float v[NORM ? 3 : 2];
      v[0] = hh;
      v[1] = gwh;
      if constexpr (NORM) v[NORM ? 2 : 0] = aa;
      team_sums<SPLIT>(rp, s, team, x++, v, peers);
      const float r = rsqrtf(fmaf(v[0], p.inv_cols, p.eps));
      const float2 m = both(-__fmul_rn(__fmul_rn(v[1], p.inv_cols), r));
      const float2 qn = NORM ? both(rsqrtf(fmaf(v[NORM ? 2 : 0], p.inv_cols, p.norm_eps))) : both(1.f);
      float vu = 0.f;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (!BRANCHES || ok[k]) {
          float2 hf[E / 2], f[E / 2], d[E / 2];
          widen2<DT>(lds16(held + at[k]), hf);
          weight_at<DT, PACK>(s_rows, V, col[k], f);
#pragma unroll
          for (int e = 0; e < E / 2; e++) {
            const float2 u = mul2(hf[e], both(r));
            dw[k][e] = fma2(g[k][e], u, dw[k][e]);
            g[k][e] = fma2(u, m, mul2(g[k][e], f[e]));
          }
          widen2<DT>(p.dres ? lds16(held + p.d_at + at[k]) : make_uint4(0u, 0u, 0u, 0u), d);
#pragma unroll
          for (int e = 0; e < E / 2; e++) g[k][e] = fma2(both(r), g[k][e], d[e]);  // dh
          if (p.dresidual) {
#pragma unroll
            for (int e = 0; e < E / 2; e++) d[e] = mul2(g[k][e], both(p.residual_scale));
            if (ok[k]) st16(p.dresidual + base + col[k], narrow2<DT>(d));
          }
          if constexpr (DROP) {
            uint32_t bits[E / 2];
            uint4 st;
            uint32_t first;
            // read here each time, so that it takes no registers between rows
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(st.x), "=r"(st.y), "=r"(st.z), "=r"(st.w)
                         : "r"(smem_addr(&s.drop)));
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(first) : "r"(smem_addr(&s.first_vec)));
            drop_bits<E>(DropState{p.drop.key0, p.drop.key1, st.x, st.y, st.z, st.w}, first + (uint32_t)base + (uint32_t)col[k], bits);
#pragma unroll
            for (int e = 0; e < E / 2; e++) g[k][e] = drop2(p.drop, bits[e], g[k][e]);  // dz
          }
          float2 u1[E / 2];
          if (NORM || (GATE && p.ar)) {
            widen2<DT>(lds16(held + p.a_at + at[k]), u1);
            if constexpr (NORM) {
#pragma unroll
              for (int e = 0; e < E / 2; e++) u1[e] = mul2(u1[e], qn);
            }
          }
          if constexpr (FACTOR) weight_at<DT, PACK && !SHARED>(s_factor, V, col[k], f);
          if constexpr (GATE == kGateOwn) {
            widen2<DT>(lds16(held + p.g_at + at[k]), d);
            if (p.dgate_own) {
#pragma unroll
              for (int e = 0; e < E / 2; e++) {
                const float2 dt = mul2(g[k][e], u1[e]);
                hf[e] = NORM ? mul2(dt, f[e]) : dt;
              }
              if (ok[k]) st16(p.dgate_own + base + col[k], narrow2<DT>(hf));
            }
#pragma unroll
            for (int e = 0; e < E / 2; e++) g[k][e] = mul2(g[k][e], d[e]);
          }
          if (NORM || shared) {
#pragma unroll
            for (int e = 0; e < E / 2; e++) ts[k][e] = fma2(g[k][e], u1[e], ts[k][e]);
          }
          if constexpr (FACTOR) {
#pragma unroll
            for (int e = 0; e < E / 2; e++) g[k][e] = mul2(g[k][e], f[e]);  // v
          }
          if constexpr (NORM) {
            float2 sv = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < E / 2; e++) sv = fma2(g[k][e], u1[e], sv);
            vu += ok[k] ? sv.x + sv.y : 0.f;
          } else {
            if (ok[k]) st16(p.dx + base + col[k], narrow2<DT>(g[k]));
          }
        }
      }
      if constexpr (NORM) {
        float w[1] = {vu};
        team_sums<SPLIT>(rp, s, team, x++, w, peers);
        // u1 * mean = a * (q * mean)
        const float2 mean = both(-__fmul_rn(__fmul_rn(w[0], p.inv_cols), qn.x));
#pragma unroll
        for (int k = 0; k < VPT; k++) {
          if (!BRANCHES || ok[k]) {
            float2 af[E / 2];
            widen2<DT>(lds16(held + p.a_at + at[k]), af);
#pragma unroll
            for (int e = 0; e < E / 2; e++) af[e] = mul2(qn, fma2(af[e], mean, g[k][e]));
            if (ok[k]) st16(p.dx + base + col[k], narrow2<DT>(af));
          }
        }
      }
      in.release();
    }
    const int cut = t.cut;
    t.next(rp);
    if (shared) {
      if (!rp.gate_span) {  // one gate row, tiles in strides
        if (!t.more(rp)) flush(0, part.groups == 1, 0);
      } else if (t.row == cut || !t.more(rp)) {
        // the span's rows of it are those from `lo` on, or from the span's first row
        const int b = (uint32_t)tile / p.gate_span, lo = b * (int)p.gate_span;
        const int first = (int)span_start(rp.rows, part.groups, part.group);
        flush(b, first <= lo && t.row - lo == (int)p.gate_span, first >= lo ? 0 : 1);
      }
    }
    // the next gate row's factor, once every team is through with this one's
    if (SHARED && rp.gate_span && t.row == cut && t.more(rp)) {
      if (!shared || teams == 1) consumers_barrier(rp);  // else flush() ended with one
      row_to_shared<DT>(NORM ? p.norm_weight + part.col0 : nullptr,
                        p.gate + (int64_t)((uint32_t)t.row / p.gate_span) * rp.vec_per_row + part.col0, V,
                        rp.teams * T, s_factor);
      consumers_barrier(rp);
    }
  }
  if (p.part_w) combine(dw, [&](int i, float4 a) { reinterpret_cast<float4*>(p.part_w)[plane() + i] = a; });
  if (NORM && p.part_w1 && !shared) combine(ts, [&](int i, float4 a) { reinterpret_cast<float4*>(p.part_w1)[plane() + i] = a; });
}

template <int DT, int VPT, bool SPLIT, bool NORM, int GATE, bool DROP, bool PACK>
__global__ void __launch_bounds__(kRingThreads, 1)
    reduce_branch_rmsnorm_backward_tma_kernel(const __grid_constant__ BranchBackwardTmaParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RingShared s;
  const RingPlan& rp = p.ring;
  const Part<SPLIT> part(rp);
  const int consumers = rp.teams * rp.team_threads, V = part.V;
  uint8_t* s_rows = smem + (size_t)rp.stages * rp.group * slice_stride(rp);
  uint8_t* s_factor = s_rows + p.factor_at;
  float4* s_comb = reinterpret_cast<float4*>(s_rows + p.sums_at);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ring_init(rp, s);
  const Tiles<GATE == kGateShared> first(rp, part);
  if (warp == kRingConsumers / 32 && lane < rp.ranks + rp.held && first.more(rp))
    prefetch_l2(slice_source(p, lane) + first.row * (int64_t)rp.row_bytes + part.col0 * 16,
                (uint32_t)first.count(rp) * (uint32_t)V * 16u);
  if constexpr (SPLIT) cluster_barrier();  // the peers' barriers too
  else __syncthreads();
  pdl_wait_and_release();
  if (warp >= kRingConsumers / 32) {
    take_registers<false>();
    const int who = warp - kRingConsumers / 32;
    if (lane == 0 && who < rp.producers) ring_produce<GATE == kGateShared>(rp, part, smem, s, who, p.err, [&](int q) { return slice_source(p, q); });
  } else {
    take_registers<true>();
    if (threadIdx.x >= consumers) return;
    const uint4 *weight = p.weight + part.col0, *norm_weight = NORM ? p.norm_weight + part.col0 : nullptr;
    weights_to_shared<DT, PACK>(weight, V, consumers, s_rows);
    if constexpr (GATE == kGateShared)
      row_to_shared<DT>(norm_weight, p.gate + (int64_t)((uint32_t)first.row / p.gate_span) * rp.vec_per_row + part.col0, V,
                        consumers, s_factor);
    else if constexpr (NORM)
      weights_to_shared<DT, PACK>(norm_weight, V, consumers, s_factor);
    if (DROP && threadIdx.x == 0) {
      const DropState d = drop_state(p.drop);
      s.drop = make_uint4(d.z, d.y, d.hi, d.lo);
      s.first_vec = p.first_vec;
    }
    consumers_barrier(rp);
    consume<DT, VPT, SPLIT, NORM, GATE, DROP, PACK>(p, part, smem, s_rows, s_factor, s_comb, s);
  }
}

template <int DT, bool SPLIT, bool NORM, int GATE, bool PACK>
BackwardTmaFn pick_drop(bool drop) {
  return drop ? reduce_branch_rmsnorm_backward_tma_kernel<DT, 2, SPLIT, NORM, GATE, true, PACK>
              : reduce_branch_rmsnorm_backward_tma_kernel<DT, 2, SPLIT, NORM, GATE, false, PACK>;
}
template <int DT, bool SPLIT, bool NORM, bool PACK>
BackwardTmaFn pick_gate(int gate, bool drop) {
  return gate == kGateNone     ? pick_drop<DT, SPLIT, NORM, kGateNone, PACK>(drop)
         : gate == kGateShared ? pick_drop<DT, SPLIT, NORM, kGateShared, PACK>(drop)
                               : pick_drop<DT, SPLIT, NORM, kGateOwn, PACK>(drop);
}
// The instances of a type, in files of their own: they compile side by side.
template <int DT, bool NORM, bool PACK>
BackwardTmaFn pick_split(bool split, int gate, bool drop) {
  return split ? pick_gate<DT, true, NORM, PACK>(gate, drop) : pick_gate<DT, false, NORM, PACK>(gate, drop);
}
template <int DT>
BackwardTmaFn pick_norm(bool split, bool norm, int gate, bool drop) {
  return norm ? pick_split<DT, true, false>(split, gate, drop) : pick_split<DT, false, false>(split, gate, drop);
}

}  // namespace
}  // namespace car
