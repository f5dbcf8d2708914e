// branch_backward_tma.cu -- backward of a block's branch (branch_backward.cu)
// for many rows: the slices dy_0 .. dy_{W-1}, h, the stored sum, the skip
// gradient and a gate of each row's own stream through a ring of shared-memory
// stages (branch_ring.cuh).  The sum of dy stays in registers and becomes dh, dz
// and v in turn; the others are read again from their stage, which is held to the
// row's end.
//
// Two vectors per thread: the weight and the factor norm_weight * gate (a gate of
// many rows) lie in shared memory, in fp32.  Longer rows read the weights from
// there packed, or from L2, and every gate row from L2.
//
// Column sums.  A thread sums g u and t (or gate t, where no gate row is shared)
// over its team's rows in registers.  Where rows share a gate row, tiles end with
// it: the teams' sums of t are then added in shared memory in team order, leave
// as dgate or as a partial of the span (as in the row kernel), and gate * t goes
// to dnorm_weight's sum in shared memory, where each column has one owner.
#include <algorithm>

#include "branch_ring.cuh"

namespace car {
namespace {


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
  int gate_from;
  uint32_t gate_span;        // rows that share a gate row
  bool shared;               // t is summed by gate row
  bool factor;               // dz is multiplied by a factor row: norm_weight, a gate of many rows or both
  int weight_rows;           // rows of weights in shared memory, in fp32 or packed
  int a_at, d_at, g_at;      // the stored sum, dres and gate behind h in their stage, in bytes
  RingPlan ring;
};

// Slices of a tile: the ranks, h, then those of ar, dres and the gate that there are.
__device__ __forceinline__ const uint8_t* slice_source(const BranchBackwardTmaParams& p, int q) {
  if (q < p.ring.ranks) return static_cast<const uint8_t*>(p.dy.p[q]);
  q -= p.ring.ranks;
  if (q == 0) return p.h;
  if (p.ar && --q == 0) return p.ar;
  if (p.dres && --q == 0) return p.dres;
  return reinterpret_cast<const uint8_t*>(p.gate);
}

template <int VPT>
constexpr bool kWideRows = VPT == 2;

// Weight row i (0: weight, 1: factor), vector v.
template <int DT, int VPT>
__device__ __forceinline__ void weight_at(const BranchBackwardTmaParams& p, const uint8_t* s_rows, int i, int v,
                                          float2 (&f)[Pack<DT>::kN / 2]) {
  const int V = p.ring.vec_per_row;
  if constexpr (kWideRows<VPT>)
    row_from_shared<DT>(s_rows + (size_t)i * V * Pack<DT>::kN * 4, V, v, f);
  else
    widen2<DT>(p.weight_rows ? lds16(s_rows + (size_t)i * p.ring.row_bytes + 16 * v) : __ldg((i == 0 ? p.weight : p.norm_weight) + v), f);
}

template <int DT, int VPT, bool NORM, int GATE, int DROP>
__device__ __forceinline__ void consume(const BranchBackwardTmaParams& p, const uint8_t* ring, const uint8_t* s_rows,
                                        uint8_t* s_factor, float4* s_comb, float4* s_dw1, RingShared& s) {
  constexpr int E = Pack<DT>::kN;
  constexpr bool SHARED = GATE == kGateShared || GATE == kGateAny, OWN = GATE == kGateOwn || GATE == kGateAny;
  constexpr bool BRANCHES = VPT * E > 16 || (SHARED && E == 8);
  const RingPlan& rp = p.ring;
  const bool own = OWN && (GATE == kGateOwn || p.gate_from == kFromRing), shared = SHARED && p.shared;
  const int T = rp.team_threads, V = rp.vec_per_row;
  const int team = threadIdx.x / T, tid = threadIdx.x - team * T;
  const uint8_t* mine = ring + (size_t)team * rp.row_bytes;  // the row in stage 0
  const DropState state = drop_state(p.drop);
  const int first = (int)span_start(rp.rows, gridDim.x, blockIdx.x);
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
    if (rp.teams == 1) {
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
    for (int i = threadIdx.x; i < V * (E / 4); i += rp.teams * T) {
      float4 a = s_comb[i];
      for (int k = 1; k < rp.teams; k++) {
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
  // rows [from, to) of gate row b are in ts
  auto flush = [&](uint32_t b, int from, int to) {
    const int lo = (int)(b * p.gate_span);
    const bool whole = from == lo && (uint32_t)(to - lo) == p.gate_span;
    float4* out = nullptr;
    if (p.dgate)
      out = reinterpret_cast<float4*>(whole ? p.dgate : p.part_gate) +
            (whole ? (int64_t)b : 2 * (int64_t)blockIdx.x + (from == first ? 0 : 1)) * V * (E / 4);
    combine(ts, [&](int i, float4 t) {
      const float4 g = four(p.gate + (int64_t)b * V, i);
      float4 d = s_dw1[i];
      d.x = fmaf(g.x, t.x, d.x);
      d.y = fmaf(g.y, t.y, d.y);
      d.z = fmaf(g.z, t.z, d.z);
      d.w = fmaf(g.w, t.w, d.w);
      s_dw1[i] = d;
      if (!out) return;
      if (NORM && whole) {
        const float4 w = four(p.norm_weight, i);
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
  int from = first;
  for (Tiles t(rp); t.more();) {
    const int tile = t.row;
    if (team >= t.count(rp)) {
      in.skip();
    } else {
      const int row = tile + team;
      const int64_t base = (int64_t)row * V;
      // a shared gate row from L2, asked for before the row's waits where registers allow
      constexpr bool EARLY = SHARED && VPT * E <= 16;
      const bool rows = SHARED && p.gate_from == kFromRows;
      uint4 gv[EARLY ? VPT : 1];
      const uint4* grow = rows ? p.gate + (int64_t)((uint32_t)row / p.gate_span) * V : nullptr;
      if (EARLY && rows) {
#pragma unroll
        for (int k = 0; k < VPT; k++) gv[EARLY ? k : 0] = __ldg(grow + col[k]);
      }
      float2 g[VPT][E / 2];
      const uint8_t* held = ring_rank_sum<DT, VPT, BRANCHES>(rp, in, mine, ok, at, g);
      if (in.failed) {
#pragma unroll
        for (int k = 0; k < VPT; k++) ok[k] = false;
      }
      float hh = 0.f, gwh = 0.f, aa = 0.f;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (!BRANCHES || ok[k]) {
          float2 hf[E / 2], wf[E / 2], sh = make_float2(0.f, 0.f), sg = sh, sa = sh;
          widen2<DT>(lds16(held + at[k]), hf);
          weight_at<DT, VPT>(p, s_rows, 0, col[k], wf);
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
      team_sums(rp, s, team, x++, v);
      const float r = rsqrtf(fmaf(v[0], p.inv_cols, p.eps));
      const float2 m = both(-__fmul_rn(__fmul_rn(v[1], p.inv_cols), r));
      const float2 qn = NORM ? both(rsqrtf(fmaf(v[NORM ? 2 : 0], p.inv_cols, p.norm_eps))) : both(1.f);
      float vu = 0.f;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (!BRANCHES || ok[k]) {
          float2 hf[E / 2], f[E / 2], d[E / 2];
          widen2<DT>(lds16(held + at[k]), hf);
          weight_at<DT, VPT>(p, s_rows, 0, col[k], f);
          widen2<DT>(p.dres ? lds16(held + p.d_at + at[k]) : make_uint4(0u, 0u, 0u, 0u), d);
#pragma unroll
          for (int e = 0; e < E / 2; e++) {
            const float2 u = mul2(hf[e], both(r));
            dw[k][e] = fma2(g[k][e], u, dw[k][e]);
            g[k][e] = fma2(both(r), fma2(u, m, mul2(g[k][e], f[e])), d[e]);  // dh
          }
          if (p.dresidual) {
#pragma unroll
            for (int e = 0; e < E / 2; e++) d[e] = mul2(g[k][e], both(p.residual_scale));
            if (ok[k]) st16(p.dresidual + base + col[k], narrow2<DT>(d));
          }
          if (DROP == kDropYes || (DROP == kDropAny && p.drop.active)) {
            uint32_t bits[E / 2];
            drop_bits<E>(state, base + col[k], bits);
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
          if (NORM || (SHARED && p.factor)) weight_at<DT, VPT>(p, s_rows, 1, col[k], f);
          if (own) {
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
          if (rows) {
            widen2<DT>(EARLY ? gv[EARLY ? k : 0] : __ldg(grow + col[k]), d);
#pragma unroll
            for (int e = 0; e < E / 2; e++) g[k][e] = mul2(g[k][e], d[e]);
          }
          if (NORM || (SHARED && p.factor)) {
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
        team_sums(rp, s, team, x++, w);
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
    if (shared && (t.row == cut || !t.more())) {
      flush((uint32_t)tile / p.gate_span, from, t.row);
      from = t.row;
    }
    // the next gate row's factor, once every team is through with this one's
    if (SHARED && rp.gate_span && p.gate_from == kFromFactor && t.row == cut && t.more()) {
      consumers_barrier(rp);
      row_to_shared<DT>(NORM ? p.norm_weight : nullptr, p.gate + (int64_t)((uint32_t)t.row / p.gate_span) * V, V,
                        rp.teams * T, s_factor);
      consumers_barrier(rp);
    }
  }
  const int64_t plane = (int64_t)blockIdx.x * V * (E / 4);
  if (p.part_w) combine(dw, [&](int i, float4 a) { reinterpret_cast<float4*>(p.part_w)[plane + i] = a; });
  if (p.part_w1) {
    float4* to = reinterpret_cast<float4*>(p.part_w1) + plane;
    if (!shared)
      combine(ts, [&](int i, float4 a) { to[i] = a; });
    else if (rp.teams > 1)
      for (int i = threadIdx.x; i < V * (E / 4); i += rp.teams * T) to[i] = s_dw1[i];
    else
      combine(ts, [&](int i, float4) { to[i] = s_dw1[i]; });
  }
}

// 16-bit types with more than four vectors per thread and fp32 with more than six,
// whose sums would not fit in registers, stay with the row kernel.
template <int DT, int VPT, bool NORM, int GATE, int DROP>
__global__ void __launch_bounds__(kRingThreads, 1)
    reduce_branch_rmsnorm_backward_tma_kernel(const __grid_constant__ BranchBackwardTmaParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ RingShared s;
  const RingPlan& rp = p.ring;
  constexpr int E = Pack<DT>::kN;
  const int consumers = rp.teams * rp.team_threads, V = rp.vec_per_row;
  uint8_t* s_rows = smem + (size_t)rp.stages * rp.group * rp.teams * rp.row_bytes;
  float4* s_dw1 = reinterpret_cast<float4*>(s_rows + (size_t)p.weight_rows * (kWideRows<VPT> ? V * E * 4 : rp.row_bytes));
  float4* s_comb = s_dw1 + (p.shared ? V * (E / 4) : 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ring_init(rp, s);
  const Tiles first(rp);
  if (warp == kRingConsumers / 32 && lane < rp.ranks + rp.held && first.more())
    prefetch_l2(slice_source(p, lane) + first.row * (int64_t)rp.row_bytes, (uint32_t)first.count(rp) * (uint32_t)rp.row_bytes);
  __syncthreads();
  pdl_wait_and_release();
  if (warp >= kRingConsumers / 32) {
    take_registers<false>();
    const int who = warp - kRingConsumers / 32;
    if (lane == 0 && who < rp.producers) ring_produce(rp, smem, s, who, p.err, [&](int q) { return slice_source(p, q); });
  } else {
    take_registers<true>();
    if (threadIdx.x >= consumers) return;
    if constexpr (kWideRows<VPT>) {
      row_to_shared<DT>(p.weight, nullptr, V, consumers, s_rows);
      if (NORM || p.factor)
        row_to_shared<DT>(NORM ? p.norm_weight : nullptr,
                          p.gate && p.gate_from == kFromFactor ? p.gate + (int64_t)((uint32_t)first.row / p.gate_span) * V : nullptr,
                          V, consumers, s_rows + (size_t)V * E * 4);
    } else if (p.weight_rows) {
      for (int v = threadIdx.x; v < V; v += consumers) {
        reinterpret_cast<uint4*>(s_rows)[v] = __ldg(p.weight + v);
        if constexpr (NORM) reinterpret_cast<uint4*>(s_rows)[V + v] = __ldg(p.norm_weight + v);
      }
    }
    if (p.shared)
      for (int i = threadIdx.x; i < V * (E / 4); i += consumers) s_dw1[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    consumers_barrier(rp);
    consume<DT, VPT, NORM, GATE, DROP>(p, smem, s_rows, s_rows + (size_t)V * E * 4, s_comb, s_dw1, s);
  }
}

using BackwardTmaFn = void (*)(const BranchBackwardTmaParams);

template <int DT, int VPT, bool NORM>
BackwardTmaFn pick_parts(int gate, bool drop) {
  if constexpr (VPT == 2) {
    if (gate == kGateNone)
      return drop ? reduce_branch_rmsnorm_backward_tma_kernel<DT, 2, NORM, kGateNone, kDropYes>
                  : reduce_branch_rmsnorm_backward_tma_kernel<DT, 2, NORM, kGateNone, kDropNone>;
    if (gate == kGateShared)
      return drop ? reduce_branch_rmsnorm_backward_tma_kernel<DT, 2, NORM, kGateShared, kDropYes>
                  : reduce_branch_rmsnorm_backward_tma_kernel<DT, 2, NORM, kGateShared, kDropNone>;
    return drop ? reduce_branch_rmsnorm_backward_tma_kernel<DT, 2, NORM, kGateOwn, kDropYes>
                : reduce_branch_rmsnorm_backward_tma_kernel<DT, 2, NORM, kGateOwn, kDropNone>;
  } else {
    if (gate == kGateNone && !drop) return reduce_branch_rmsnorm_backward_tma_kernel<DT, VPT, NORM, kGateNone, kDropNone>;
    return reduce_branch_rmsnorm_backward_tma_kernel<DT, VPT, NORM, kGateAny, kDropAny>;
  }
}
template <int DT, bool NORM>
BackwardTmaFn pick_vpt(int vpt, int gate, bool drop) {
  if (vpt == 2) return pick_parts<DT, 2, NORM>(gate, drop);
  if (vpt == 3) return pick_parts<DT, 3, NORM>(gate, drop);
  if (vpt == 4) return pick_parts<DT, 4, NORM>(gate, drop);
  if constexpr (DT == kFP32) {
    if (vpt == 5) return pick_parts<DT, 5, NORM>(gate, drop);
    if (vpt == 6) return pick_parts<DT, 6, NORM>(gate, drop);
  }
  return nullptr;
}
BackwardTmaFn pick(int dtype, int vpt, bool norm, int gate, bool drop) {
  switch (dtype) {
    case kBF16: return norm ? pick_vpt<kBF16, true>(vpt, gate, drop) : pick_vpt<kBF16, false>(vpt, gate, drop);
    case kFP16: return norm ? pick_vpt<kFP16, true>(vpt, gate, drop) : pick_vpt<kFP16, false>(vpt, gate, drop);
    default: return norm ? pick_vpt<kFP32, true>(vpt, gate, drop) : pick_vpt<kFP32, false>(vpt, gate, drop);
  }
}

constexpr int kSharedBudget = 222 * 1024;  // ring and what lies beside it; RingShared is static

// Where a call's weights and slices lie; the bytes beside the ring: the weights, the
// sum of dnorm_weight behind a shared gate, the teams' sums.
bool fit(int dtype, int W, const BranchArgs& br, const BranchGradArgs& g, int64_t rows, int vec_per_row, const TeamShape& sh,
         BranchBackwardTmaParams* p, int* beside) {
  const bool norm = br.norm_weight != nullptr, wide = sh.vpt == 2, own = br.gate && br.gate_span == 0;
  // A shared gate row is part of the factor where its rows are worth the two barriers
  // and the L2 latency of making the next one's: W = 1, M = 16384, N = 4096 bf16 with
  // norms, 1024 rows a gate row, 145 us against 151 with the gate read from L2 for
  // every row; M = 13332, N = 1160 fp16, 1111 rows, 40.6 against 42.3.
  const bool folded = wide && br.gate && !own && (br.gate_span == rows || br.gate_span * vec_per_row >= 8192);
  p->gate_from = !br.gate || folded ? kFromFactor : own ? kFromRing : kFromRows;
  p->factor = norm || folded;
  p->shared = br.gate && !own && (g.dgate || g.dnorm_weight);
  RingPlan& rp = p->ring;
  rp.rows = (int)rows;
  rp.row_bytes = vec_per_row * 16;
  rp.vec_per_row = vec_per_row;
  rp.ranks = W;
  rp.teams = sh.teams;
  rp.team_threads = sh.team_threads;
  rp.gate_span = p->shared || (folded && br.gate_span < rows) ? (uint32_t)br.gate_span : 0;
  const int slice = sh.teams * rp.row_bytes, floats = dtype == kFP32 ? rp.row_bytes : 2 * rp.row_bytes;
  rp.held = 1;
  p->a_at = p->d_at = p->g_at = 0;
  if (g.ar) p->a_at = slice * rp.held++;
  if (g.dres) p->d_at = slice * rp.held++;
  if (own) p->g_at = slice * rp.held++;
  p->weight_rows = p->factor ? 2 : 1;
  const int sums = (p->shared ? floats : 0) + (sh.teams > 1 ? sh.teams * floats : 0);
  *beside = sums + p->weight_rows * (wide ? floats : rp.row_bytes);
  if (branch_ring_fit(kSharedBudget - *beside, &rp)) return true;
  if (wide) return false;
  p->weight_rows = 0;
  *beside = sums;
  return branch_ring_fit(kSharedBudget - sums, &rp);
}

}  // namespace

bool branch_backward_tma_shape(int dtype, int64_t rows, int vec_per_row, int num_sms, TeamShape* out) {
  const int vpt = vec_per_row > 2048 ? (vec_per_row + 511) / 512 : team_vectors(vec_per_row, 2, vec_per_row > 1536 ? 4 : 3);
  if (vpt > (dtype == kFP32 ? 6 : 4)) return false;
  out->vpt = vpt;
  out->use = team_use(vec_per_row, vpt);
  out->team_threads = team_threads(vec_per_row, vpt);
  if (out->team_threads > 512) return false;
  // as many as a CTA has rows, so that few rows are spread over the SMs
  out->teams = (int)std::min<int64_t>(512 / out->team_threads, (rows + num_sms - 1) / num_sms);
  out->grid = (int)std::min<int64_t>((rows + out->teams - 1) / out->teams, num_sms);
  return true;
}

bool branch_backward_tma_fits(int dtype, int W, const BranchArgs& br, const BranchGradArgs& g, int64_t rows, int vec_per_row,
                              const TeamShape& sh) {
  BranchBackwardTmaParams p;
  int beside;
  return fit(dtype, W, br, g, rows, vec_per_row, sh, &p, &beside);
}

cudaError_t branch_backward_tma_prepare(int dtype, const TeamShape& sh) {
  for (int parts = 0; parts < 12; parts++) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(pick(dtype, sh.vpt, parts & 1, parts >> 2, parts & 2)),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBudget);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_branch_backward_tma(int dtype, int W, const RankPtrs& dy, const BranchArgs& br, const BranchGradArgs& g,
                                       const void* weight, float eps, unsigned int* err, int64_t rows, int64_t cols,
                                       int vec_per_row, const TeamShape& sh, cudaStream_t s) {
  BranchBackwardTmaParams p;
  int beside;
  if (!fit(dtype, W, br, g, rows, vec_per_row, sh, &p, &beside)) return cudaErrorInvalidValue;
  const bool one = sh.grid == 1, own = br.gate && br.gate_span == 0;
  p.dy = dy;
  p.h = static_cast<const uint8_t*>(g.h);
  p.ar = static_cast<const uint8_t*>(g.ar);
  p.dres = static_cast<const uint8_t*>(g.dres);
  p.weight = static_cast<const uint4*>(weight);
  p.norm_weight = static_cast<const uint4*>(br.norm_weight);
  p.gate = static_cast<const uint4*>(br.gate);
  p.dx = static_cast<uint4*>(g.dx);
  p.dresidual = static_cast<uint4*>(g.dresidual);
  p.dgate_own = own ? static_cast<uint4*>(g.dgate) : nullptr;
  p.dgate = own ? nullptr : static_cast<float*>(g.dgate);
  const size_t plane = (size_t)sh.grid * (size_t)cols;
  p.part_w = g.dweight ? (one ? g.dweight : g.workspace) : nullptr;
  p.part_w1 = g.dnorm_weight ? (one ? g.dnorm_weight : g.workspace + plane) : nullptr;
  p.part_gate = one ? nullptr : g.workspace + 2 * plane;
  p.err = err;
  p.drop = br.drop;
  p.residual_scale = br.residual_scale;
  p.eps = eps;
  p.norm_eps = br.norm_eps;
  p.inv_cols = 1.f / (float)cols;
  p.gate_span = (uint32_t)std::max<int64_t>(br.gate_span, 1);
  const RingPlan& rp = p.ring;
  cudaError_t e = launch_pdl(pick(dtype, sh.vpt, br.norm_weight != nullptr, gate_kind(br), br.drop.active), (unsigned)sh.grid,
                             (unsigned)kRingThreads, (size_t)rp.stages * rp.group * rp.teams * rp.row_bytes + beside, s, 1, p);
  return e == cudaSuccess ? launch_branch_sums(br, g, dtype, sh.grid, rows, cols, s) : e;
}

}  // namespace car
