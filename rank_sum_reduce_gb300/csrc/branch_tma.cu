// branch_tma.cu -- launch shapes of the forward pipeline of a block's branch (branch_tma.cuh).
#include <algorithm>

#include "branch_tma.cuh"

namespace car {
namespace {

BranchTmaFn pick(int dtype, const BranchTeams& sh, bool norm, int gate, bool drop) {
  const bool split = sh.cluster > 1;
  switch (dtype) {
    case kBF16: return branch_tma_bf16(sh.vpt, split, norm, gate, drop);
    case kFP16: return branch_tma_fp16(sh.vpt, split, norm, gate, drop);
    default: return branch_tma_fp32(sh.vpt, split, norm, gate, drop);
  }
}

constexpr int kSharedBudget = 224 * 1024;  // ring and rows of weights; RingShared is static

// A call's ring, and the bytes beside it: the weight, norm_weight, and a gate of all rows
// behind both.  At least six slices fit beside them, whatever the call's parts.
bool fit(int W, const BranchArgs& br, int64_t rows, int vec_per_row, const BranchTeams& sh, BranchTmaParams* p, int* beside) {
  const bool column = br.gate && br.gate_span == rows;
  p->gate_from = !br.gate || column ? kFromFactor : br.gate_span == 0 ? kFromRing : kFromRows;
  RingPlan& rp = p->ring;
  rp.rows = (int)rows;
  rp.row_bytes = vec_per_row * 16;
  rp.vec_per_row = vec_per_row;
  rp.cluster = sh.cluster;
  rp.chunk = (vec_per_row + sh.cluster - 1) / sh.cluster;
  rp.ranks = W;
  rp.held = 1 + (p->gate_from == kFromRing ? 1 : 0);
  rp.teams = sh.teams;
  rp.team_threads = sh.team_threads;
  rp.gate_span = 0;
  *beside = (column ? 3 : br.norm_weight ? 2 : 1) * rp.chunk * 16;
  return branch_ring_fit(kSharedBudget - *beside, &rp);
}

}  // namespace

// A whole tile per stage where two fit, three stages or 96 KB at most: deeper rings
// ask for more of HBM at once than helps (W = 1, M = 16389, N = 4096 bf16 with both
// norms, 64, 96 and 128 KB in flight per SM: 88, 84 and 92 us; without 83, 91 and 93; own
// gates, M = 8192, 51, 54 and 57; N = 8192, M = 4000 46, 41 and 41).  Else stages of
// two slices, as many as there is room for (W = 8, M = 512, N = 8192 with both norms
// 20.9, 19.6 and 18.3 us with three, four and five of them; stages of one slice 20.5
// with eight, of four 20.4 with three).
bool branch_ring_fit(int budget, RingPlan* p) {
  const int slices = p->ranks + p->held, slice = (int)slice_stride(*p), places = budget / slice;
  if (2 * slices <= places) {
    p->group = slices;
    p->tile_stages = 1;
  } else {
    p->group = std::max(p->held, 2);
    p->tile_stages = (p->ranks + p->group - 1) / p->group + 1;
  }
  p->stages = std::min(places / p->group, kMaxRingStages);
  if (p->tile_stages == 1) p->stages = std::min(p->stages, std::max(3, 96 * 1024 / (p->group * slice)));
  p->producers = kProducers;
  return p->stages >= 2;
}

void branch_teams(int64_t rows, int vec_per_row, int num_sms, int cluster, int vpt, BranchTeams* out) {
  const int chunk = (vec_per_row + cluster - 1) / cluster;
  out->cluster = cluster;
  out->vpt = vpt;
  out->use = team_use(chunk, vpt);
  out->team_threads = team_threads(chunk, vpt);
  // as many as a CTA has rows, so that few rows are spread over the SMs
  out->teams = cluster > 1 ? 1 : (int)std::min<int64_t>(512 / out->team_threads, (rows + num_sms - 1) / num_sms);
  out->grid = (int)std::min<int64_t>((rows + out->teams - 1) / out->teams, num_sms / cluster) * cluster;
}

cudaError_t branch_clusters(const void* fn, int cluster, int smem, int* clusters) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster, 1, 1);
  cfg.blockDim = dim3(kRingThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int got = 0;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(&got, fn, &cfg);
  *clusters = std::min(*clusters, std::max(got, 1));
  return e;
}

// Two vectors per thread for rows of up to 1024 vectors, three where that fits
// clearly better (W = 1, M = 8000, N = 5120 bf16 with both norms 70 and 52 us) or for
// rows of up to 1536; from there on a cluster of two CTAs a row, of four above 2048.
// Four vectors in shorter rows halve the warps that a row's exchanges pass through,
// and lose to the overlap of more of them: W = 1, M = 16389, N = 4096 bf16 with both
// norms 82.5 us with two, 92.4 with four; W = 2, M = 4000, N = 8192 50.5 and 63.
void branch_tma_shape(int64_t rows, int vec_per_row, int num_sms, BranchTeams* out) {
  const int cluster = vec_per_row > 2048 ? 4 : vec_per_row > 1536 ? 2 : 1;
  branch_teams(rows, vec_per_row, num_sms, cluster, cluster > 1 ? 2 : team_vectors(vec_per_row, 2, 3), out);
}

cudaError_t branch_tma_prepare(int dtype, BranchTeams* sh) {
  int clusters = sh->grid / sh->cluster;
  for (int parts = 0; parts < 12; parts++) {
    const void* fn = reinterpret_cast<const void*>(pick(dtype, *sh, parts & 1, parts >> 2, parts & 2));
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBudget);
    if (e == cudaSuccess && sh->cluster > 1) e = branch_clusters(fn, sh->cluster, kSharedBudget, &clusters);
    if (e != cudaSuccess) return e;
  }
  sh->grid = clusters * sh->cluster;
  return cudaSuccess;
}

cudaError_t launch_branch_tma(int dtype, int W, const RankPtrs& in, const BranchArgs& br, const void* residual,
                              const void* weight, float eps, void* residual_out, void* norm_out, void* ar_out,
                              unsigned int* err, int64_t rows, int64_t cols, int vec_per_row, const BranchTeams& sh,
                              const WaitHook& hook, cudaStream_t s) {
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
  p.wait_ns = hook.wait_ns;
  p.delay_ns = hook.delay_ns;
  p.delay_row = hook.delay_row;
  p.delay_cta = hook.delay_cta;
  const RingPlan& rp = p.ring;
  return launch_pdl(pick(dtype, sh, br.norm_weight != nullptr, gate_kind(br), br.drop.active), (unsigned)sh.grid,
                    (unsigned)kRingThreads, (size_t)rp.stages * rp.group * slice_stride(rp) + beside, s, (unsigned)sh.cluster, p);
}

}  // namespace car
