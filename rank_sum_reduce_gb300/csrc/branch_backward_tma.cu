// branch_backward_tma.cu -- launch shapes of the backward pipeline of a block's branch (branch_backward_tma.cuh).
#include <algorithm>

#include "branch_backward_tma.cuh"

namespace car {
namespace {

BackwardTmaFn pick(int dtype, bool split, bool norm, int gate, bool drop, bool packed) {
  switch (dtype) {
    case kBF16: return packed ? branch_backward_tma_packed_bf16(split, gate, drop) : branch_backward_tma_bf16(split, norm, gate, drop);
    case kFP16: return packed ? branch_backward_tma_packed_fp16(split, gate, drop) : branch_backward_tma_fp16(split, norm, gate, drop);
    default: return branch_backward_tma_fp32(split, norm, gate, drop);
  }
}

// Ring and what lies beside it; RingShared is static.  To the last 4 KB: where a second
// tile or a third one just fits it is worth much (W = 1, M = 8192, N = 4096 bf16 with
// norms and own gates 115 us with 222 KB, 85 with 224; W = 4, M = 2048 fp32 with one gate
// row 57 and 52).
constexpr int kSharedBudget = 224 * 1024;

// Where a call's weights and slices lie; the bytes beside the ring: the weights and the
// teams' sums.
bool fit(int dtype, int W, const BranchArgs& br, const BranchGradArgs& g, int64_t rows, int vec_per_row, const BranchTeams& sh,
         BranchBackwardTmaParams* p, int* beside, bool* packed) {
  const bool norm = br.norm_weight != nullptr, own = br.gate && br.gate_span == 0, shared = br.gate && !own;
  p->shared = shared && (g.dgate || g.dnorm_weight);
  RingPlan& rp = p->ring;
  rp.rows = (int)rows;
  rp.row_bytes = vec_per_row * 16;
  rp.vec_per_row = vec_per_row;
  rp.cluster = sh.cluster;
  rp.chunk = (vec_per_row + sh.cluster - 1) / sh.cluster;
  rp.ranks = W;
  rp.teams = sh.teams;
  rp.team_threads = sh.team_threads;
  rp.gate_span = shared && br.gate_span < rows ? (uint32_t)br.gate_span : 0;  // whatever is asked for: the same bits
  const int part_bytes = rp.chunk * 16, slice = sh.teams * part_bytes, floats = dtype == kFP32 ? part_bytes : 2 * part_bytes;
  rp.held = 1;
  p->a_at = p->d_at = p->g_at = 0;
  if (g.ar) p->a_at = slice * rp.held++;
  if (g.dres) p->d_at = slice * rp.held++;
  if (own) p->g_at = slice * rp.held++;
  // The weights in fp32 where two tiles fit beside them, else packed where that gains a stage (branch_backward_tma.cuh).
  const bool factor = norm || shared;
  auto place = [&](bool pack) {
    *packed = pack;
    p->factor_at = pack ? part_bytes : floats;
    p->sums_at = p->factor_at + (!factor ? 0 : pack && !shared ? part_bytes : floats);
    *beside = p->sums_at + (sh.teams > 1 ? sh.teams : 0) * floats;
    return branch_ring_fit(kSharedBudget - *beside, &rp);
  };
  const bool wide = place(false);
  if (dtype == kFP32 || !norm || (wide && rp.tile_stages == 1)) return wide;
  const int stages = wide ? rp.stages : 0;
  return (place(true) && (rp.tile_stages == 1 || rp.stages > stages)) || place(false);
}

}  // namespace

// Two vectors per thread, with a cluster of two CTAs a row from 1025 vectors on and of
// four from 2049: three 16-bit vectors per thread and their column sums do not fit in
// registers (W = 4, M = 4000, N = 5120 bf16 with both norms 67 us with two, though
// they leave 37 % of the threads' places empty, and 101 with three).
void branch_backward_tma_shape(int64_t rows, int vec_per_row, int num_sms, BranchTeams* out) {
  branch_teams(rows, vec_per_row, num_sms, vec_per_row > 2048 ? 4 : vec_per_row > 1024 ? 2 : 1, 2, out);
}

cudaError_t branch_backward_tma_prepare(int dtype, BranchTeams* sh) {
  int clusters = sh->grid / sh->cluster;
  for (int parts = 0; parts < 24; parts++) {
    const bool packed = parts >= 12;  // instances with a norm of the 16-bit types
    if (packed && (dtype == kFP32 || !(parts & 1))) continue;
    const void* fn = reinterpret_cast<const void*>(pick(dtype, sh->cluster > 1, parts & 1, parts % 12 >> 2, parts & 2, packed));
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBudget);
    if (e == cudaSuccess && sh->cluster > 1) e = branch_clusters(fn, sh->cluster, kSharedBudget, &clusters);
    if (e != cudaSuccess) return e;
  }
  sh->grid = clusters * sh->cluster;
  return cudaSuccess;
}

namespace {

// One launch, of `rows` rows from row `row0` of the problem on, and the sum of its partials.
cudaError_t launch_part(int dtype, int W, const RankPtrs& dy, const BranchArgs& br, const BranchGradArgs& g, const void* weight,
                        float eps, unsigned int* err, int64_t row0, int64_t rows, int64_t cols, int vec_per_row,
                        const BranchTeams& sh, const WaitHook& hook, bool add, bool add_gate, cudaStream_t s) {
  BranchBackwardTmaParams p;
  int beside;
  bool packed;
  if (!fit(dtype, W, br, g, rows, vec_per_row, sh, &p, &beside, &packed)) return cudaErrorInvalidValue;
  const int groups = sh.grid / sh.cluster;
  const bool one = groups == 1, own = br.gate && br.gate_span == 0;
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
  const size_t plane = (size_t)groups * (size_t)cols;
  p.part_w = g.dweight ? (one ? g.dweight : g.workspace) : nullptr;
  p.part_w1 = g.dnorm_weight ? (one ? g.dnorm_weight : g.workspace + plane) : nullptr;
  p.part_gate = one ? nullptr : g.workspace + 2 * plane;
  p.err = err;
  p.drop = br.drop;
  p.residual_scale = br.residual_scale;
  p.eps = eps;
  p.norm_eps = br.norm_eps;
  p.inv_cols = 1.f / (float)cols;
  p.first_vec = (uint32_t)(row0 * vec_per_row);
  p.gate_span = (uint32_t)std::max<int64_t>(br.gate_span, 1);
  p.wait_ns = hook.wait_ns;
  p.delay_ns = hook.delay_ns;
  p.delay_row = hook.delay_row - row0;
  p.delay_cta = hook.delay_cta;
  const RingPlan& rp = p.ring;
  cudaError_t e = launch_pdl(pick(dtype, sh.cluster > 1, br.norm_weight != nullptr, gate_kind(br), br.drop.active, packed), (unsigned)sh.grid,
                             (unsigned)kRingThreads, (size_t)rp.stages * rp.group * slice_stride(rp) + beside, s, (unsigned)sh.cluster, p);
  return e == cudaSuccess ? launch_branch_sums(br, g, dtype, groups, rows, cols, add, add_gate, s) : e;
}

// Rows that a thread adds to its column sums one after the other.  Each addition rounds to
// fp32, and where the terms are alike all of them the same way: off by up to 2^-13 for 2^12
// rows, and 1.6 % were measured for 3.5 million (N = 8, 1025 * 2^20 rows).  So
// a launch has at most this many for each thread, and the next one adds to what it left: N =
// 8192 has two from 77,825 rows on, N = 4096 from twice as many.  Fewer of them would mean
// more launches where rows are short (N = 8: 1.2 million rows a launch).
constexpr int64_t kSumRows = 512;
// The pipelines count rows in 32 bits, a grid's step past the last one included.
constexpr int64_t kMaxRows = 1 << 30;

}  // namespace

cudaError_t launch_branch_backward_tma(int dtype, int W, const RankPtrs& dy, const BranchArgs& br, const BranchGradArgs& g,
                                       const void* weight, float eps, unsigned int* err, int64_t rows, int64_t cols,
                                       int vec_per_row, const BranchTeams& sh, const WaitHook& hook, cudaStream_t s) {
  const bool own = br.gate && br.gate_span == 0, shared = br.gate && !own;
  const bool sums = g.dweight || g.dnorm_weight || (shared && g.dgate);
  const int64_t groups = sh.grid / sh.cluster;
  const int64_t most = sums && groups > 1 ? kSumRows * sh.teams * groups : kMaxRows;
  // Parts of whole gate rows, with which tiles end (gate rows of fewer rows than there are
  // teams leave teams out), or where one has more rows than a launch, of that one's; of nearly
  // the same size, so that each has rows for every CTA.
  const bool cut = shared && br.gate_span > most;
  const int64_t unit = shared && !cut ? br.gate_span : 1, outer = cut ? rows / br.gate_span : 1, units = rows / outer / unit;
  const int64_t tiles = sums && shared && !cut ? (unit + sh.teams - 1) / sh.teams : 0;  // of a gate row
  const int64_t per = std::max<int64_t>(tiles ? most / sh.teams / tiles : most / unit, 1);
  const int parts = (int)((units + per - 1) / per);
  const size_t row_bytes = (size_t)vec_per_row * 16;
  auto at = [](auto* p, size_t bytes) { return p ? reinterpret_cast<decltype(p)>(reinterpret_cast<uintptr_t>(p) + bytes) : p; };
  for (int64_t o = 0; o < outer; o++) {
    for (int i = 0; i < parts; i++) {
      const int64_t row0 = o * (rows / outer) + unit * span_start(units, parts, i);
      const int64_t n = unit * (span_start(units, parts, i + 1) - span_start(units, parts, i));
      const size_t off = (size_t)row0 * row_bytes, gate_row = shared ? (size_t)(row0 / br.gate_span) : 0;
      RankPtrs d = dy;
      for (int r = 0; r < W; r++) d.p[r] = at(dy.p[r], off);
      BranchArgs b = br;
      b.gate = at(br.gate, own ? off : gate_row * row_bytes);
      if (cut) b.gate_span = n;
      BranchGradArgs to = g;
      to.ar = at(g.ar, off);
      to.h = at(g.h, off);
      to.dres = at(g.dres, off);
      to.dx = at(g.dx, off);
      to.dresidual = at(g.dresidual, off);
      to.dgate = at(g.dgate, own ? off : gate_row * (size_t)cols * sizeof(float));
      const cudaError_t e = launch_part(dtype, W, d, b, to, weight, eps, err, row0, n, cols, vec_per_row, sh, hook, row0 > 0,
                                        cut && i > 0, s);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace car
