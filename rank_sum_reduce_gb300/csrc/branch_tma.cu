// branch_tma.cu -- a block's branch (branch_rows.cu) for many rows: the rank
// slices and the residual (and a gate of each row's own) stream through a ring
// of shared-memory stages (branch_ring.cuh), the sum of a row stays in registers
// over both of its exchanges, and while one team of warps waits for its row's
// sums another folds.
//
// The rows of weights, and a gate of all rows, lie in shared memory as they are, or
// in L2 where they would leave the ring less than six slices.
#include <algorithm>

#include "branch_ring.cuh"

namespace car {
namespace {

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
  bool packed;              // the rows of weights lie in shared memory
  uint32_t gate_span;       // rows that share a gate row (kGateRows)
  RingPlan ring;
};

__device__ __forceinline__ const uint8_t* slice_source(const BranchTmaParams& p, int q) {
  return q < p.ring.ranks ? static_cast<const uint8_t*>(p.in.p[q])
                          : q == p.ring.ranks ? p.residual : reinterpret_cast<const uint8_t*>(p.gate);
}

// Weight row i (0: weight, 1: norm_weight, 2: a gate of all rows), vector v.
__device__ __forceinline__ uint4 weight_at(const BranchTmaParams& p, const uint8_t* s_rows, int i, int v) {
  return p.packed ? lds16(s_rows + (size_t)i * p.ring.row_bytes + 16 * v)
                  : __ldg((i == 0 ? p.weight : i == 1 ? p.norm_weight : p.gate) + v);
}

template <int DT, int VPT, bool NORM, int GATE, int DROP>
__device__ __forceinline__ void consume(const BranchTmaParams& p, const uint8_t* ring, const uint8_t* s_rows, RingShared& s) {
  constexpr int E = Pack<DT>::kN;
  constexpr bool BRANCHES = VPT > 4;
  constexpr bool SHARED = GATE == kGateShared || GATE == kGateAny, OWN = GATE == kGateOwn || GATE == kGateAny;
  const RingPlan& rp = p.ring;
  const bool own = OWN && (GATE == kGateOwn || p.gate_from == kFromRing), rows = SHARED && p.gate_from == kFromRows;
  const int T = rp.team_threads, V = rp.vec_per_row;
  const int team = threadIdx.x / T, tid = threadIdx.x - team * T;
  const uint32_t stride = (uint32_t)rp.teams * (uint32_t)rp.row_bytes;
  const uint8_t* mine = ring + (size_t)team * rp.row_bytes;  // the row in stage 0
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
  // DEFER: the second sum of the team's last row travels with the first one of the row
  // after it, so a row passes one barrier instead of two, and its norm_out is stored
  // then; where registers hold two rows.
  constexpr bool DEFER = NORM && VPT * E <= 24;
  float2 last[DEFER ? VPT : 1][E / 2];
  float last_ss = 0.f;
  int64_t last_base = -1;
  auto finish = [&](const float2(&h)[VPT][E / 2], int64_t base, float sum) {
    const float2 r = both(rsqrtf(fmaf(sum, p.inv_cols, p.eps)));
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (BRANCHES && !ok[k]) continue;
      float2 f[E / 2];
      widen2<DT>(weight_at(p, s_rows, 0, col[k]), f);
#pragma unroll
      for (int e = 0; e < E / 2; e++) f[e] = mul2(mul2(h[k][e], r), f[e]);
      if (ok[k]) st16(p.norm_out + base + col[k], narrow2<DT>(f));
    }
  };
  for (Tiles t(rp); t.more(); t.next(rp)) {
    if (team >= t.count(rp)) {
      in.skip();
      continue;
    }
    const int row = t.row + team;
    const int64_t base = (int64_t)row * V;
    // a shared gate row from L2, asked for before the row's waits where registers allow
    constexpr bool EARLY = SHARED && VPT * E <= 16;
    uint4 gv[EARLY ? VPT : 1];
    const uint4* grow = rows ? p.gate + (int64_t)((uint32_t)row / p.gate_span) * V : nullptr;
    if (EARLY && rows) {
#pragma unroll
      for (int k = 0; k < VPT; k++) gv[EARLY ? k : 0] = __ldg(grow + col[k]);
    }
    // the mask's bits, before the row's waits where registers allow: a chain of ten
    // dependent products that would stand between its two exchanges
    constexpr bool BITS_FIRST = DROP != kDropNone && VPT * E <= 16;
    uint32_t bits[BITS_FIRST ? VPT : 1][E / 2];
    if (BITS_FIRST && (DROP == kDropYes || p.drop.active)) {
#pragma unroll
      for (int k = 0; k < VPT; k++) drop_bits_here<E>(state, base + col[k], bits[BITS_FIRST ? k : 0]);
    }
    float2 z[VPT][E / 2];
    const uint8_t* held = ring_rank_sum<DT, VPT, BRANCHES>(rp, in, mine, ok, at, z);
    if (in.failed) {
#pragma unroll
      for (int k = 0; k < VPT; k++) ok[k] = false;
    }
    if (p.ar_out) {
#pragma unroll
      for (int k = 0; k < VPT; k++)
        if (ok[k]) st16(p.ar_out + base + col[k], narrow2<DT>(z[k]));
    }
    float2 inv = both(1.f);
    if constexpr (NORM) {
      float v[DEFER ? 2 : 1] = {0.f};
      if constexpr (DEFER) v[DEFER ? 1 : 0] = last_ss;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (BRANCHES && !ok[k]) continue;
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) ss = fma2(z[k][e], z[k][e], ss);
        v[0] += ok[k] ? ss.x + ss.y : 0.f;
      }
      team_sums(rp, s, team, x++, v);
      inv = both(rsqrtf(fmaf(v[0], p.inv_cols, p.norm_eps)));
      if constexpr (DEFER) {
        if (last_base >= 0) finish(last, last_base, v[DEFER ? 1 : 0]);
      }
    }
    float hh = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (BRANCHES && !ok[k]) continue;
      float2 f[E / 2];
      if constexpr (NORM) {
        widen2<DT>(weight_at(p, s_rows, 1, col[k]), f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[k][e] = mul2(mul2(z[k][e], inv), f[e]);
      }
      if (GATE && (GATE != kGateAny || p.gate)) {
        widen2<DT>(own ? lds16(held + stride + at[k]) : rows ? (EARLY ? gv[EARLY ? k : 0] : __ldg(grow + col[k])) : weight_at(p, s_rows, 2, col[k]), f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[k][e] = mul2(z[k][e], f[e]);
      }
      if (DROP == kDropYes || (DROP == kDropAny && p.drop.active)) {
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
      team_sums(rp, s, team, x++, v);
      finish(z, base, v[0]);
    }
  }
  if constexpr (DEFER) {
    if (last_base >= 0) {
      float v[1] = {last_ss};
      team_sums(rp, s, team, x++, v);
      finish(last, last_base, v[0]);
    }
  }
}

template <int DT, int VPT, bool NORM, int GATE, int DROP>
__global__ void __launch_bounds__(kRingThreads, 1)
    reduce_branch_residual_rmsnorm_tma_kernel(const __grid_constant__ BranchTmaParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ RingShared s;
  const RingPlan& rp = p.ring;
  uint8_t* s_rows = smem + (size_t)rp.stages * rp.group * rp.teams * rp.row_bytes;
  const int consumers = rp.teams * rp.team_threads, V = rp.vec_per_row;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ring_init(rp, s);
  // the first tile into L2 while the previous grid of the stream finishes
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
    if (p.packed) {
      for (int v = threadIdx.x; v < V; v += consumers) {
        reinterpret_cast<uint4*>(s_rows)[v] = __ldg(p.weight + v);
        if constexpr (NORM) reinterpret_cast<uint4*>(s_rows)[V + v] = __ldg(p.norm_weight + v);
        if (GATE && p.gate && p.gate_from == kFromFactor) reinterpret_cast<uint4*>(s_rows)[2 * V + v] = __ldg(p.gate + v);
      }
      consumers_barrier(rp);
    }
    consume<DT, VPT, NORM, GATE, DROP>(p, smem, s_rows, s);
  }
}

using BranchTmaFn = void (*)(const BranchTmaParams);

template <int DT, int VPT, bool NORM>
BranchTmaFn pick_parts(int gate, bool drop) {
  if constexpr (VPT == 2) {
    if (gate == kGateNone)
      return drop ? reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, NORM, kGateNone, kDropYes>
                  : reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, NORM, kGateNone, kDropNone>;
    if (gate == kGateShared)
      return drop ? reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, NORM, kGateShared, kDropYes>
                  : reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, NORM, kGateShared, kDropNone>;
    return drop ? reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, NORM, kGateOwn, kDropYes>
                : reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, NORM, kGateOwn, kDropNone>;
  } else {
    if (gate == kGateNone && !drop) return reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, NORM, kGateNone, kDropNone>;
    return reduce_branch_residual_rmsnorm_tma_kernel<DT, VPT, NORM, kGateAny, kDropAny>;
  }
}
template <int DT, bool NORM>
BranchTmaFn pick_vpt(int vpt, int gate, bool drop) {
  switch (vpt) {
    case 2: return pick_parts<DT, 2, NORM>(gate, drop);
    case 3: return pick_parts<DT, 3, NORM>(gate, drop);
    case 4: return pick_parts<DT, 4, NORM>(gate, drop);
    case 5: return pick_parts<DT, 5, NORM>(gate, drop);
    case 6: return pick_parts<DT, 6, NORM>(gate, drop);
    case 7: return pick_parts<DT, 7, NORM>(gate, drop);
    default: return pick_parts<DT, 8, NORM>(gate, drop);
  }
}
BranchTmaFn pick(int dtype, int vpt, bool norm, int gate, bool drop) {
  switch (dtype) {
    case kBF16: return norm ? pick_vpt<kBF16, true>(vpt, gate, drop) : pick_vpt<kBF16, false>(vpt, gate, drop);
    case kFP16: return norm ? pick_vpt<kFP16, true>(vpt, gate, drop) : pick_vpt<kFP16, false>(vpt, gate, drop);
    default: return norm ? pick_vpt<kFP32, true>(vpt, gate, drop) : pick_vpt<kFP32, false>(vpt, gate, drop);
  }
}

constexpr int kSharedBudget = 222 * 1024;  // ring and rows of weights; RingShared is static

// Where a call's weights lie, and its ring; the bytes beside the ring.
bool fit(int W, const BranchArgs& br, int64_t rows, int vec_per_row, const TeamShape& sh, BranchTmaParams* p, int* beside) {
  const bool column = br.gate && br.gate_span == rows;
  p->gate_from = !br.gate || column ? kFromFactor : br.gate_span == 0 ? kFromRing : kFromRows;
  RingPlan& rp = p->ring;
  rp.rows = (int)rows;
  rp.row_bytes = vec_per_row * 16;
  rp.vec_per_row = vec_per_row;
  rp.ranks = W;
  rp.held = 1 + (p->gate_from == kFromRing ? 1 : 0);
  rp.teams = sh.teams;
  rp.team_threads = sh.team_threads;
  rp.gate_span = 0;
  *beside = (column ? 3 : br.norm_weight ? 2 : 1) * rp.row_bytes;
  p->packed = branch_ring_fit(kSharedBudget - *beside, &rp) && rp.stages * rp.group >= 6;
  if (p->packed) return true;
  *beside = 0;
  return branch_ring_fit(kSharedBudget, &rp);
}

}  // namespace

// A whole tile per stage where two fit, three stages or 96 KB at most: deeper rings
// ask for more of HBM at once than helps (W = 1, M = 16389, N = 4096 bf16 without a
// norm 83 to 85 us with 64 to 96 KB in flight per SM, 94 with 192).  Else stages of
// two slices, as many as there is room for (W = 8, M = 512, N = 8192 with both norms
// 20.9, 19.6 and 18.3 us with three, four and five of them; stages of one slice 20.5
// with eight, of four 20.4 with three).
bool branch_ring_fit(int budget, RingPlan* p) {
  const int slices = p->ranks + p->held, places = budget / (p->teams * p->row_bytes);
  if (2 * slices <= places) {
    p->group = slices;
    p->tile_stages = 1;
  } else {
    p->group = std::max(p->held, 2);
    p->tile_stages = (p->ranks + p->group - 1) / p->group + 1;
  }
  p->stages = std::min(places / p->group, kMaxRingStages);
  if (p->tile_stages == 1) p->stages = std::min(p->stages, std::max(3, 96 * 1024 / (p->group * p->teams * p->row_bytes)));
  p->producers = kProducers;
  return p->stages >= 2;
}

// Two vectors per thread for rows of up to 1024 vectors, three where that fits
// clearly better or for longer ones, four only for rows that three do not hold,
// above 2048 as few as 512 threads need (see norm_backward_tma.cu).  Four vectors in
// shorter rows halve the warps that a row's exchanges pass through, and lose to the
// overlap of more of them: W = 1, M = 16389, N = 4096 bf16 with both norms 82.5 us
// with two, 92.4 with four; W = 2, M = 4000, N = 8192 50.5 and 63.
bool branch_tma_shape(int64_t rows, int vec_per_row, int num_sms, TeamShape* out) {
  const int vpt = vec_per_row > 2048 ? (vec_per_row + 511) / 512 : team_vectors(vec_per_row, 2, vec_per_row > 1536 ? 4 : 3);
  if (vpt > 8) return false;
  out->vpt = vpt;
  out->use = team_use(vec_per_row, vpt);
  out->team_threads = team_threads(vec_per_row, vpt);
  if (out->team_threads > 512) return false;
  // as many as a CTA has rows, so that few rows are spread over the SMs
  out->teams = (int)std::min<int64_t>(512 / out->team_threads, (rows + num_sms - 1) / num_sms);
  out->grid = (int)std::min<int64_t>((rows + out->teams - 1) / out->teams, num_sms);
  return true;
}

bool branch_tma_fits(int W, const BranchArgs& br, int64_t rows, int vec_per_row, const TeamShape& sh) {
  BranchTmaParams p;
  int beside;
  return fit(W, br, rows, vec_per_row, sh, &p, &beside);
}

cudaError_t branch_tma_prepare(int dtype, const TeamShape& sh) {
  for (int parts = 0; parts < 12; parts++) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(pick(dtype, sh.vpt, parts & 1, parts >> 2, parts & 2)),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBudget);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_branch_tma(int dtype, int W, const RankPtrs& in, const BranchArgs& br, const void* residual,
                              const void* weight, float eps, void* residual_out, void* norm_out, void* ar_out,
                              unsigned int* err, int64_t rows, int64_t cols, int vec_per_row, const TeamShape& sh,
                              cudaStream_t s) {
  BranchTmaParams p;
  int beside;
  if (!fit(W, br, rows, vec_per_row, sh, &p, &beside)) return cudaErrorInvalidValue;
  p.in = in;
  p.residual = static_cast<const uint8_t*>(residual);
  p.weight = static_cast<const uint4*>(weight);
  p.norm_weight = static_cast<const uint4*>(br.norm_weight);
  p.gate = static_cast<const uint4*>(br.gate);
  p.residual_out = static_cast<uint4*>(residual_out);
  p.norm_out = static_cast<uint4*>(norm_out);
  p.ar_out = static_cast<uint4*>(ar_out);
  p.err = err;
  p.drop = br.drop;
  p.residual_scale = br.residual_scale;
  p.eps = eps;
  p.norm_eps = br.norm_eps;
  p.inv_cols = 1.f / (float)cols;
  p.gate_span = (uint32_t)std::max<int64_t>(br.gate_span, 1);
  const RingPlan& rp = p.ring;
  return launch_pdl(pick(dtype, sh.vpt, br.norm_weight != nullptr, gate_kind(br), br.drop.active), (unsigned)sh.grid,
                    (unsigned)kRingThreads, (size_t)rp.stages * rp.group * rp.teams * rp.row_bytes + beside, s, 1, p);
}

}  // namespace car
