// branch_tma.cu -- a block's branch (branch_rows.cu) for many rows: the rank
// slices and the residual (and a gate of each row's own) stream through a ring
// of shared-memory stages (branch_ring.cuh), the sum of a row stays in registers
// over both of its exchanges, and while one team of warps waits for its row's
// sums another folds.
//
// Two vectors per thread: the weight and the factor norm_weight * gate (a gate of
// all rows) lie in shared memory, in fp32.  Longer rows leave the ring no room for
// that: both norms' weights lie there packed, or in L2, and the gate in L2, as for
// all rows a gate row that some of them share.
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
  float cols;
  int gate_from;
  bool factor;              // z is multiplied by a factor row: norm_weight, a gate of all rows or both
  bool packed;              // rows of weights in shared memory where they are not in fp32
  uint32_t gate_span;       // rows that share a gate row (kGateRows)
  RingPlan ring;
};

__device__ __forceinline__ const uint8_t* slice_source(const BranchTmaParams& p, int q) {
  return q < p.ring.ranks ? static_cast<const uint8_t*>(p.in.p[q])
                          : q == p.ring.ranks ? p.residual : reinterpret_cast<const uint8_t*>(p.gate);
}

template <int VPT>
constexpr bool kWideRows = VPT == 2;

// Weight row i (0: weight, 1: factor), vector v.
template <int DT, int VPT>
__device__ __forceinline__ void weight_at(const BranchTmaParams& p, const uint8_t* s_rows, int i, int v,
                                          float2 (&f)[Pack<DT>::kN / 2]) {
  const int V = p.ring.vec_per_row;
  if constexpr (kWideRows<VPT>)
    row_from_shared<DT>(s_rows + (size_t)i * V * Pack<DT>::kN * 4, V, v, f);
  else
    widen2<DT>(p.packed ? lds16(s_rows + (size_t)i * p.ring.row_bytes + 16 * v) : __ldg((i == 0 ? p.weight : p.norm_weight) + v), f);
}

template <int DT, int VPT, bool NORM, int GATE, int DROP>
__device__ __forceinline__ void consume(const BranchTmaParams& p, const uint8_t* ring, const uint8_t* s_rows, RingShared& s) {
  constexpr int E = Pack<DT>::kN;
  constexpr bool SHARED = GATE == kGateShared || GATE == kGateAny, OWN = GATE == kGateOwn || GATE == kGateAny;
  const RingPlan& rp = p.ring;
  const bool own = OWN && (GATE == kGateOwn || p.gate_from == kFromRing), rows = SHARED && p.gate_from == kFromRows;
  const int T = rp.team_threads, V = rp.vec_per_row;
  const int team = threadIdx.x / T, tid = threadIdx.x - team * T;
  const uint32_t stride = (uint32_t)rp.teams * (uint32_t)rp.row_bytes;
  const uint8_t* mine = ring + (size_t)team * rp.row_bytes + 16 * tid;  // this thread's first vector in stage 0
  const DropState state = drop_state(p.drop);
  bool ok[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) ok[k] = tid + k * T < V;
  RingReader in(rp, s);
  uint32_t x = 0;
  bool failed = false;
  for (Tiles t(rp); t.more() && !failed; t.next(rp)) {
    if (team >= t.count(rp)) {
      failed = !in.skip();
      continue;
    }
    const int row = t.row + team;
    const int64_t at = (int64_t)row * V + tid;
    float2 z[VPT][E / 2];
    const uint8_t* held = ring_rank_sum<DT, VPT>(rp, in, mine, ok, z);
    if (!held) {
      failed = true;
      break;
    }
    if (p.ar_out) {
#pragma unroll
      for (int k = 0; k < VPT; k++)
        if (ok[k]) st16(p.ar_out + at + k * T, narrow2<DT>(z[k]));
    }
    float2 inv = both(1.f);
    if constexpr (NORM) {
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (ok[k]) {
#pragma unroll
          for (int e = 0; e < E / 2; e++) ss = fma2(z[k][e], z[k][e], ss);
        }
      }
      float v[1] = {ss.x + ss.y};
      if (!team_sums(rp, s, team, x++, v)) {
        failed = true;
        break;
      }
      inv = both(rsqrtf(__fdiv_rn(v[0], p.cols) + p.norm_eps));
    }
    const uint4* grow = rows ? p.gate + (int64_t)((uint32_t)row / p.gate_span) * V + tid : nullptr;
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        float2 f[E / 2];
        if (NORM || (SHARED && p.factor)) {
          weight_at<DT, VPT>(p, s_rows, 1, tid + k * T, f);
#pragma unroll
          for (int e = 0; e < E / 2; e++) z[k][e] = mul2(NORM ? mul2(z[k][e], inv) : z[k][e], f[e]);
        }
        if (own || rows) {
          widen2<DT>(own ? lds16(held + stride + 16 * k * T) : __ldg(grow + k * T), f);
#pragma unroll
          for (int e = 0; e < E / 2; e++) z[k][e] = mul2(z[k][e], f[e]);
        }
        if (DROP == kDropYes || (DROP == kDropAny && p.drop.active)) {
          uint32_t bits[E / 2];
          drop_bits<E>(state, at + k * T, bits);
#pragma unroll
          for (int e = 0; e < E / 2; e++) z[k][e] = drop2(p.drop, bits[e], z[k][e]);
        }
        widen2<DT>(lds16(held + 16 * k * T), f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) {
          z[k][e] = fma2(both(p.residual_scale), f[e], z[k][e]);
          ss = fma2(z[k][e], z[k][e], ss);
        }
        st16(p.residual_out + at + k * T, narrow2<DT>(z[k]));
      }
    }
    in.release();
    float v[1] = {ss.x + ss.y};
    if (!team_sums(rp, s, team, x++, v)) {
      failed = true;
      break;
    }
    const float2 r = both(rsqrtf(__fdiv_rn(v[0], p.cols) + p.eps));
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        float2 f[E / 2];
        weight_at<DT, VPT>(p, s_rows, 0, tid + k * T, f);
#pragma unroll
        for (int e = 0; e < E / 2; e++) f[e] = mul2(mul2(z[k][e], r), f[e]);
        st16(p.norm_out + at + k * T, narrow2<DT>(f));
      }
    }
  }
  if (failed) {
    atomicOr(p.err, 1u);
    *static_cast<volatile int*>(&s.abort) = 1;
  }
}

template <int DT, int VPT, bool NORM, int GATE, int DROP>
__global__ void __launch_bounds__(512 + 32 * kProducers, 1)
    reduce_branch_residual_rmsnorm_tma_kernel(const __grid_constant__ BranchTmaParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ RingShared s;
  const RingPlan& rp = p.ring;
  uint8_t* s_rows = smem + (size_t)rp.stages * rp.group * rp.teams * rp.row_bytes;
  const int consumers = rp.teams * rp.team_threads, V = rp.vec_per_row;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) ring_init(rp, s);
  // the first tile into L2 while the previous grid of the stream finishes
  const Tiles first(rp);
  if (warp == consumers >> 5 && lane < rp.ranks + rp.held && first.more())
    prefetch_l2(slice_source(p, lane) + first.row * (int64_t)rp.row_bytes, (uint32_t)first.count(rp) * (uint32_t)rp.row_bytes);
  __syncthreads();
  pdl_wait_and_release();
  if (warp >= consumers >> 5) {
    if (lane == 0) ring_produce(rp, smem, s, warp - (consumers >> 5), p.err, [&](int q) { return slice_source(p, q); });
  } else {
    if constexpr (kWideRows<VPT>) {
      row_to_shared<DT>(p.weight, nullptr, V, consumers, s_rows);
      if (NORM || p.factor)
        row_to_shared<DT>(NORM ? p.norm_weight : nullptr, p.gate_from == kFromFactor ? p.gate : nullptr, V, consumers,
                          s_rows + (size_t)V * Pack<DT>::kN * 4);
      asm volatile("bar.sync 1, %0;" ::"r"(consumers) : "memory");
    } else if (p.packed) {
      for (int v = threadIdx.x; v < V; v += consumers) {
        reinterpret_cast<uint4*>(s_rows)[v] = __ldg(p.weight + v);
        if constexpr (NORM) reinterpret_cast<uint4*>(s_rows)[V + v] = __ldg(p.norm_weight + v);
      }
      asm volatile("bar.sync 1, %0;" ::"r"(consumers) : "memory");
    }
    consume<DT, VPT, NORM, GATE, DROP>(p, smem, s_rows, s);
  }
}

using BranchTmaFn = void (*)(const BranchTmaParams);

template <int DT, int VPT, bool NORM>
BranchTmaFn pick_parts(int gate, bool drop) {
  if constexpr (VPT == 2) {
    if (gate == kGateNone)
      return drop ? reduce_branch_residual_rmsnorm_tma_kernel<DT, 2, NORM, kGateNone, kDropYes>
                  : reduce_branch_residual_rmsnorm_tma_kernel<DT, 2, NORM, kGateNone, kDropNone>;
    if (gate == kGateShared)
      return drop ? reduce_branch_residual_rmsnorm_tma_kernel<DT, 2, NORM, kGateShared, kDropYes>
                  : reduce_branch_residual_rmsnorm_tma_kernel<DT, 2, NORM, kGateShared, kDropNone>;
    return drop ? reduce_branch_residual_rmsnorm_tma_kernel<DT, 2, NORM, kGateOwn, kDropYes>
                : reduce_branch_residual_rmsnorm_tma_kernel<DT, 2, NORM, kGateOwn, kDropNone>;
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
bool fit(int dtype, int W, const BranchArgs& br, int64_t rows, int vec_per_row, const BranchTeams& sh, BranchTmaParams* p,
         int* beside) {
  const bool norm = br.norm_weight != nullptr, wide = sh.vpt == 2, column = br.gate && br.gate_span == rows;
  p->gate_from = !br.gate ? kFromFactor : br.gate_span == 0 ? kFromRing : wide && column ? kFromFactor : kFromRows;
  p->factor = norm || (wide && column);
  RingPlan& rp = p->ring;
  rp.rows = (int)rows;
  rp.row_bytes = vec_per_row * 16;
  rp.vec_per_row = vec_per_row;
  rp.ranks = W;
  rp.held = 1 + (p->gate_from == kFromRing ? 1 : 0);
  rp.teams = sh.teams;
  rp.tile_rows = sh.tile_rows;
  rp.team_threads = sh.team_threads;
  rp.gate_span = 0;
  const int weights = (p->factor ? 2 : 1) * rp.row_bytes;
  p->packed = !wide;
  *beside = wide && dtype != kFP32 ? 2 * weights : weights;
  if (branch_ring_fit(kSharedBudget - *beside, &rp) && (wide || rp.stages * rp.group >= 6)) return true;
  if (wide) return false;
  p->packed = false;
  *beside = 0;
  return branch_ring_fit(kSharedBudget, &rp);
}

}  // namespace

bool branch_ring_fit(int budget, RingPlan* p) {
  const int slices = p->ranks + p->held, places = budget / (p->teams * p->row_bytes);
  if (2 * slices <= places) {
    p->group = slices;
    p->tile_stages = 1;
  } else {
    p->group = std::max(p->held, std::min(4, places / 3));
    p->tile_stages = (p->ranks + p->group - 1) / p->group + 1;
  }
  p->stages = std::min(places / p->group, kMaxRingStages);
  p->producers = kProducers;
  return p->stages >= 2;
}

// Two vectors per thread for rows of up to 1024 vectors, three where that fits
// clearly better or for longer ones, four only for rows that three do not hold,
// above 2048 as few as 512 threads need (see norm_backward_tma.cu).
bool branch_tma_shape(int64_t rows, int vec_per_row, int num_sms, BranchTeams* out) {
  const int vpt = vec_per_row > 2048 ? (vec_per_row + 511) / 512 : team_vectors(vec_per_row, 2, vec_per_row > 1536 ? 4 : 3);
  if (vpt > 8) return false;
  out->vpt = vpt;
  out->use = team_use(vec_per_row, vpt);
  out->team_threads = team_threads(vec_per_row, vpt);
  if (out->team_threads > 512) return false;
  out->teams = 512 / out->team_threads;
  out->tile_rows = (int)std::min<int64_t>(out->teams, (rows + num_sms - 1) / num_sms);  // few rows: spread over the SMs
  out->grid = (int)std::min<int64_t>((rows + out->tile_rows - 1) / out->tile_rows, num_sms);
  return true;
}

bool branch_tma_fits(int dtype, int W, const BranchArgs& br, int64_t rows, int vec_per_row, const BranchTeams& sh) {
  BranchTmaParams p;
  int beside;
  return fit(dtype, W, br, rows, vec_per_row, sh, &p, &beside);
}

cudaError_t branch_tma_prepare(int dtype, const BranchTeams& sh) {
  for (int parts = 0; parts < 12; parts++) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(pick(dtype, sh.vpt, parts & 1, parts >> 2, parts & 2)),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBudget);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_branch_tma(int dtype, int W, const RankPtrs& in, const BranchArgs& br, const void* residual,
                              const void* weight, float eps, void* residual_out, void* norm_out, void* ar_out,
                              unsigned int* err, int64_t rows, int64_t cols, int vec_per_row, const BranchTeams& sh,
                              cudaStream_t s) {
  BranchTmaParams p;
  int beside;
  if (!fit(dtype, W, br, rows, vec_per_row, sh, &p, &beside)) return cudaErrorInvalidValue;
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
  p.cols = (float)cols;
  p.gate_span = (uint32_t)std::max<int64_t>(br.gate_span, 1);
  const RingPlan& rp = p.ring;
  return launch_pdl(pick(dtype, sh.vpt, br.norm_weight != nullptr, gate_kind(br), br.drop.active), (unsigned)sh.grid,
                    (unsigned)(sh.teams * sh.team_threads + 32 * rp.producers),
                    (size_t)rp.stages * rp.group * rp.teams * rp.row_bytes + beside, s, 1, p);
}

}  // namespace car
