// branch_api.cu -- C ABI of what lies between the rank sum and the residual add
// (include/car.h: car_reduce_dropout, car_reduce_branch_*): argument checks and
// launch shapes.  The kernels are in dropout.cu, branch_rows.cu, branch_tma.cu,
// branch_backward.cu and branch_backward_tma.cu.
#include <cmath>
#include <cstring>

#include "branch.h"
#include "handle.h"

using namespace car;

namespace {

bool finite_eps(float eps) { return std::isfinite(eps) && eps >= 0.f; }

car_status drop_params(const car_dropout* d, DropParams* out) {
  *out = DropParams{0, 0, 0, nullptr, false, 0, 1.f};
  if (!d) return CAR_OK;
  if (!(d->p >= 0.f && d->p <= 1.f)) return CAR_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(d->offset_dev) & 7u) return CAR_ERR_ALIGN;
  const uint64_t t = (uint64_t)std::floor((double)d->p * 65536.0 + 0.5);
  out->active = t > 0;
  out->limit = t > 0 ? (uint32_t)((t << 16) - 1) : 0;
  out->scale = t == 65536 ? 0.f : (float)(65536.0 / (65536.0 - (double)t));
  out->key0 = (uint32_t)d->seed;
  out->key1 = (uint32_t)(d->seed >> 32);
  out->offset = d->offset;
  out->offset_dev = out->active ? d->offset_dev : nullptr;
  return CAR_OK;
}

// Rows that share a row of the gate (0: each has its own); -1: not a divisor.
int64_t gate_span(const car_ctx* h, int64_t gate_rows) {
  if (gate_rows == 0) return 0;
  return gate_rows < 0 || gate_rows > h->M || h->M % gate_rows != 0 ? -1 : h->M / gate_rows;
}

car_status branch_args(const car_ctx* h, const car_branch* b, BranchArgs* out) {
  if (!b) return CAR_ERR_ARG;
  if (!std::isfinite(b->residual_scale) || (b->norm_weight && !finite_eps(b->norm_eps))) return CAR_ERR_ARG;
  if (!aligned16(b->norm_weight) || !aligned16(b->gate)) return CAR_ERR_ALIGN;
  out->norm_weight = b->norm_weight;
  out->norm_eps = b->norm_weight ? b->norm_eps : 0.f;
  out->gate = b->gate;
  out->gate_span = b->gate ? gate_span(h, b->gate_rows) : 1;
  if (out->gate_span < 0) return CAR_ERR_ARG;
  out->residual_scale = b->residual_scale;
  return drop_params(b->dropout, &out->drop);
}

size_t gate_bytes(const car_ctx* h, const BranchArgs& b) {
  return b.gate ? (size_t)(b.gate_span == 0 ? h->M : h->M / b.gate_span) * (size_t)h->N * h->es : 0;
}

// Buffers of a call: every output must be apart from all others, but for the
// inputs that it may replace (the same address, the same size).
struct Buffers {
  struct Range {
    uintptr_t at;
    size_t bytes;
    bool output, replaceable;
  };
  Range r[2 * kMaxRanks];
  int n = 0;
  void add(const void* p, size_t bytes, bool output, bool replaceable = false) {
    if (p && bytes) r[n++] = Range{reinterpret_cast<uintptr_t>(p), bytes, output, replaceable};
  }
  bool clash() const {
    for (int i = 0; i < n; i++) {
      if (!r[i].output) continue;
      for (int j = 0; j < n; j++) {
        if (i == j || r[j].at >= r[i].at + r[i].bytes || r[i].at >= r[j].at + r[j].bytes) continue;
        if (r[j].output || !r[j].replaceable || !r[i].replaceable || r[i].at != r[j].at) return true;
      }
    }
    return false;
  }
};

car_status prepare_dropout(car_ctx* h) {
  if (h->dropout_ready.load(std::memory_order_acquire)) return CAR_OK;
  std::lock_guard<std::mutex> lk(h->shapes);
  if (h->dropout_ready.load(std::memory_order_relaxed)) return CAR_OK;
  const OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_fail(on.status, "device of the handle");
  int per_sm = 0;
  cudaError_t e = dropout_occupancy(h->dtype, h->W, &per_sm);
  if (e != cudaSuccess) return cuda_fail(e, "dropout occupancy");
  const int64_t per_cta = (int64_t)kReduceThreads * dropout_vectors_per_thread(h->W);
  h->dropout_grid = (int)std::min<int64_t>((h->nvec + per_cta - 1) / per_cta, (int64_t)std::max(per_sm, 1) * h->num_sms);
  h->dropout_ready.store(true, std::memory_order_release);
  return CAR_OK;
}

bool one_vector(int, int vpt) { return vpt == 1; }
int branch_threads(int, int) { return kBranchThreads; }

// The forward's pipeline counts rows in 32 bits, a grid's step past the last one included.
constexpr int64_t kMaxPipelineRows = 1 << 30;

// When the forward's pipeline is faster than its row kernel: from so many rows per SM
// on.  Measured on GB300 (graph replay over cold inputs, bf16 with both norms; the row
// kernel's time divided by the pipeline's, over M = 152, 304, 608, 1216).
//  * Rows of more than 1024 vectors, which the row kernel has to split: N = 11072 1.40
//    to 2.60, N = 16384 1.07 to 1.91, N = 32768 1.14 to 2.32; at M = 80 0.92 to 1.42.
//  * Shorter ones: the more ranks and the shorter the row, the longer the row kernel,
//    with several CTAs per SM, keeps up.  W = 1: N = 1024 0.77, 1.02, 1.21, 1.30; N =
//    4096 0.88, 0.88, 0.97, 1.11; N = 8192 0.93, 1.04, 1.16, 1.38.  W = 4: N = 1024
//    0.77, 0.97, 0.96, 1.10; N = 4096 0.76, 1.03, 1.22, 1.33; N = 8192 1.10, 1.19,
//    1.42, 1.70.  W = 8: N = 1024 0.81, 0.86, 0.90, 0.98 (M = 2432 1.14); N = 2048
//    0.86, 0.81, 0.92, 1.11; N = 4096 0.72, 0.92, 1.14, 1.16; N = 8192 0.97, 1.16,
//    1.32, 1.42.  W = 16: N = 2048 0.68, 0.74, 0.96, 1.03; N = 4096 0.70, 0.98, 1.04,
//    1.04; N = 8192 0.97, 1.08, 1.09, 1.10.  fp32 at the same vectors per row, and
//    without the first norm, within 0.1 of these.
//  * Rank counts that the row kernel is not compiled for keep to the rule of those
//    beside them, though its instance for 16 ranks falls behind earlier: W = 3: N =
//    4096 0.82, 1.11, 1.38, 1.58 (M = 228 5.2 us against 4.4), N = 8192 1.20, 1.40,
//    1.65, 2.13 (M = 80 5.9 against 4.4); W = 6: N = 4096 0.76, 0.99, 1.21, 1.43; N =
//    8192 1.05, 1.23, 1.57, 1.72.  At M = 228 the rule also leaves a little with W = 4:
//    N = 4096 5.1 us against 4.7.
bool branch_pipeline_pays(const car_ctx* h) {
  const int V = h->vec_per_row, W = h->W;
  double rows;  // per SM
  if (V > 1024) rows = 1;
  else if (W <= 2) rows = V <= 128 ? 3 : V <= 512 ? 5 : 3;
  else if (W <= 4) rows = V <= 128 ? 5 : V <= 512 ? 3 : 1.5;
  else if (W <= 8) rows = V <= 128 ? 10 : V <= 256 ? 6 : V <= 512 ? 3 : 1.5;
  else rows = V <= 256 ? 10 : V <= 512 ? 4 : 2;
  return (double)h->M >= rows * h->num_sms && h->M <= kMaxPipelineRows;
}

// The same for the backward (M = 152, 228, 304, 608, 1216): W = 1: N = 1024 0.89, 1.10,
// 1.16, 1.41, 1.55; N = 4096 0.84, 1.11, 1.11, 1.18, 1.39; N = 8192 1.01, 0.99, 1.16, 1.40,
// 1.72.  W = 4: N = 2048 0.92, 1.18, 1.12, 1.07, 1.18; N = 8192 0.98, 0.98, 1.15, 1.41,
// 1.60.  W = 8: N = 1024 0.77, 1.06, 1.08, 1.35, 1.20; N = 4096 0.86, 0.97, 0.95, 1.11,
// 1.12; N = 8192 0.97, 0.93, 1.10, 1.19, 1.33.  W = 16: N = 4096 0.96, 1.11, 1.10, 1.21,
// 1.25.  More than 1024 vectors (M = 152, 304, 1216): N = 11072 1.30 to 2.10, N = 16384
// 1.15 to 1.81, N = 32768 1.32 to 2.25; at M = 80 0.89 to 1.23.  Rank counts that the row
// kernel is not compiled for (M = 152, 228, 304, 608): W = 3, N = 4096 1.01, 1.29, 1.25,
// 1.51; W = 6, N = 2048 1.07, 1.35, 1.33, 1.33.  So rows of up to 512 vectors would gain
// from one and a half rows per SM on already (W = 1, N = 2048, M = 228 7.4 us against 6.3;
// W = 3, N = 4096 12.0 against 9.2).
bool branch_backward_pipeline_pays(const car_ctx* h) {
  return h->M >= (h->vec_per_row > 1024 ? 1 : 2) * (int64_t)h->num_sms;
}

car_status prepare_branch(car_ctx* h) {
  if (h->branch_ready.load(std::memory_order_acquire)) return CAR_OK;
  std::lock_guard<std::mutex> lk(h->shapes);
  if (h->branch_ready.load(std::memory_order_relaxed)) return CAR_OK;
  const OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_fail(on.status, "device of the handle");
  int groups = 0;
  h->branch = row_split_shape(h->W, h->M, h->vec_per_row, h->num_sms, one_vector, branch_threads, false);
  cudaError_t e = branch_resident_groups(h->dtype, h->W, h->branch, h->num_sms, &groups);
  if (e != cudaSuccess) return cuda_fail(e, "branch occupancy");
  h->branch.groups = (int)std::max<int64_t>(1, std::min<int64_t>(h->M, groups));
  branch_tma_shape(h->M, h->vec_per_row, h->num_sms, &h->branch_tma);
  h->branch_pipeline = branch_pipeline_pays(h);
  if (h->branch_pipeline && (e = branch_tma_prepare(h->dtype, &h->branch_tma)) != cudaSuccess)
    return cuda_fail(e, "branch pipeline smem");
  h->branch_ready.store(true, std::memory_order_release);
  return CAR_OK;
}

car_status prepare_branch_backward(car_ctx* h) {
  if (h->branch_backward_ready.load(std::memory_order_acquire)) return CAR_OK;
  std::lock_guard<std::mutex> lk(h->shapes);
  if (h->branch_backward_ready.load(std::memory_order_relaxed)) return CAR_OK;
  const OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_fail(on.status, "device of the handle");
  int groups = 0;
  h->branch_backward = row_split_shape(h->W, h->M, h->vec_per_row, h->num_sms, one_vector, branch_threads, false);
  cudaError_t e = branch_backward_resident_groups(h->dtype, h->W, h->branch_backward, h->num_sms, &groups);
  if (e != cudaSuccess) return cuda_fail(e, "branch backward occupancy");
  h->branch_backward.groups = (int)std::max<int64_t>(1, std::min<int64_t>(h->M, groups));
  branch_backward_tma_shape(h->M, h->vec_per_row, h->num_sms, &h->branch_backward_tma);
  h->branch_backward_pipeline = branch_backward_pipeline_pays(h);
  if (h->branch_backward_pipeline && (e = branch_backward_tma_prepare(h->dtype, &h->branch_backward_tma)) != cudaSuccess)
    return cuda_fail(e, "branch backward pipeline smem");
  h->branch_backward_ready.store(true, std::memory_order_release);
  return CAR_OK;
}

// CTAs (or clusters) of the backward's kernel.
int workspace_groups(const car_ctx* h) {
  return h->branch_backward_pipeline ? h->branch_backward_tma.grid / h->branch_backward_tma.cluster : h->branch_backward.groups;
}

}  // namespace

extern "C" {

car_status car_reduce_dropout(car_ctx* h, const void* const* inputs, const car_dropout* drop, void* ar_out, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (!drop) return CAR_ERR_ARG;
  DropParams d;
  if ((st = drop_params(drop, &d)) != CAR_OK) return st;
  RankPtrs tbl;
  if ((st = check_table(h, inputs, &tbl)) != CAR_OK) return st;
  if ((st = check_dev(ar_out)) != CAR_OK) return st;
  if ((st = prepare_dropout(h)) != CAR_OK) return st;
  cudaError_t e = launch_dropout(h->dtype, h->W, tbl, d, ar_out, h->nvec, h->dropout_grid, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "reduce_dropout launch");
}

car_status car_reduce_branch_residual_rmsnorm(car_ctx* h, const void* const* inputs, const car_branch* branch,
                                              const void* residual, const void* weight, float eps, void* residual_out,
                                              void* norm_out, void* ar_out, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (!finite_eps(eps)) return CAR_ERR_ARG;
  BranchArgs b;
  if ((st = branch_args(h, branch, &b)) != CAR_OK) return st;
  RankPtrs tbl;
  if ((st = check_table(h, inputs, &tbl)) != CAR_OK) return st;
  if ((st = check_dev(residual)) != CAR_OK) return st;
  if ((st = check_dev(weight)) != CAR_OK) return st;
  if ((st = check_dev(residual_out)) != CAR_OK) return st;
  if ((st = check_dev(norm_out)) != CAR_OK) return st;
  if (!aligned16(ar_out)) return CAR_ERR_ALIGN;
  if (!h->fused_ok) return CAR_ERR_SIZE;
  const size_t D = (size_t)h->D, row = (size_t)h->N * h->es;
  // residual_out may replace residual, ar_out one input: anything else clashes
  Buffers at;
  for (int r = 0; r < h->W; r++) at.add(tbl.p[r] == ar_out ? nullptr : tbl.p[r], D, false);
  at.add(residual == residual_out ? nullptr : residual, D, false);
  at.add(weight, row, false);
  at.add(b.norm_weight, row, false);
  at.add(b.gate, gate_bytes(h, b), false);
  at.add(b.drop.offset_dev, 8, false);
  at.add(residual_out, D, true);
  at.add(norm_out, D, true);
  at.add(ar_out, D, true);
  if (at.clash()) return CAR_ERR_ARG;
  if ((st = prepare_branch(h)) != CAR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (h->branch_pipeline)
    e = launch_branch_tma(h->dtype, h->W, tbl, b, residual, weight, eps, residual_out, norm_out, ar_out, h->d_err, h->M, h->N,
                          h->vec_per_row, h->branch_tma, h->hook, s);
  else
    e = launch_branch(h->dtype, h->W, tbl, b, residual, weight, eps, residual_out, norm_out, ar_out, h->d_err, h->M, h->N,
                      h->vec_per_row, h->branch, h->hook, s);
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "reduce_branch_residual_rmsnorm launch");
}

size_t car_branch_workspace_bytes(car_ctx* h, const car_branch* branch) {
  if (!live(h) || !h->fused_ok) return 0;
  const bool gate = branch && branch->gate;
  const int64_t span = gate ? gate_span(h, branch->gate_rows) : 0;
  if (span < 0 || prepare_branch_backward(h) != CAR_OK) return 0;
  return branch_workspace_floats(workspace_groups(h), h->N, span > 0) * sizeof(float);
}

car_status car_reduce_branch_residual_rmsnorm_backward(car_ctx* h, const void* const* dnorm, const car_branch* branch,
                                                       const void* ar, const void* residual_out, const void* weight,
                                                       float eps, const void* dresidual_out, const car_branch_grads* out,
                                                       void* workspace, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (!finite_eps(eps) || !out) return CAR_ERR_ARG;
  BranchArgs b;
  if ((st = branch_args(h, branch, &b)) != CAR_OK) return st;
  RankPtrs tbl;
  if ((st = check_table(h, dnorm, &tbl)) != CAR_OK) return st;
  if ((st = check_dev(residual_out)) != CAR_OK) return st;
  if ((st = check_dev(weight)) != CAR_OK) return st;
  if ((st = check_dev(out->dx)) != CAR_OK) return st;
  if ((out->dnorm_weight && !b.norm_weight) || (out->dgate && !b.gate)) return CAR_ERR_ARG;
  if (!ar && (b.norm_weight || out->dgate)) return CAR_ERR_ARG;
  if (!aligned16(ar) || !aligned16(dresidual_out) || !aligned16(out->dresidual) || !aligned16(out->dweight) ||
      !aligned16(out->dnorm_weight) || !aligned16(out->dgate) || !aligned16(workspace))
    return CAR_ERR_ALIGN;
  if (!h->fused_ok) return CAR_ERR_SIZE;
  if ((st = prepare_branch_backward(h)) != CAR_OK) return st;
  const int groups = workspace_groups(h);
  const bool shared = b.gate && b.gate_span > 0;
  const bool sums = out->dweight || out->dnorm_weight || (shared && out->dgate);
  const size_t floats = sums ? branch_workspace_floats(groups, h->N, shared) : 0;
  if (floats && !workspace) return CAR_ERR_ARG;
  const size_t D = (size_t)h->D, row = (size_t)h->N * h->es;
  Buffers at;
  for (int r = 0; r < h->W; r++) at.add(tbl.p[r], D, false, true);
  at.add(ar, D, false, true);
  at.add(residual_out, D, false, true);
  at.add(dresidual_out, D, false, true);
  at.add(weight, row, false);
  at.add(b.norm_weight, row, false);
  at.add(b.gate, gate_bytes(h, b), false);
  at.add(b.drop.offset_dev, 8, false);
  at.add(out->dx, D, true, true);
  at.add(out->dresidual, D, true, true);
  at.add(out->dweight, (size_t)h->N * 4, true);
  at.add(out->dnorm_weight, (size_t)h->N * 4, true);
  at.add(out->dgate, shared ? gate_bytes(h, b) / h->es * 4 : gate_bytes(h, b), true);
  at.add(workspace, floats * sizeof(float), true);
  if (at.clash()) return CAR_ERR_ARG;
  BranchGradArgs g;
  g.ar = ar;
  g.h = residual_out;
  g.dres = dresidual_out;
  g.dx = out->dx;
  g.dresidual = out->dresidual;
  g.dweight = out->dweight;
  g.dnorm_weight = out->dnorm_weight;
  g.dgate = out->dgate;
  g.workspace = static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (h->branch_backward_pipeline)
    e = launch_branch_backward_tma(h->dtype, h->W, tbl, b, g, weight, eps, h->d_err, h->M, h->N, h->vec_per_row,
                                   h->branch_backward_tma, h->hook, s);
  else
    e = launch_branch_backward(h->dtype, h->W, tbl, b, g, weight, eps, h->d_err, h->M, h->N, h->vec_per_row,
                               h->branch_backward, h->hook, s);
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "reduce_branch_residual_rmsnorm_backward launch");
}

}  // extern "C"
