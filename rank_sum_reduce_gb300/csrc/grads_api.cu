// grads_api.cu -- the C ABI's gradient handles (include/car.h, car_grads_*):
// argument checks, the plan of chunks, launch sizes.  Everything is computed
// in the kernels of grads.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <unordered_set>
#include <vector>

#include "../../include/car.h"
#include "car_device.cuh"
#include "car_launch.h"

struct car_grads {
  int device;
  int grid, sums_grid;  // of car_grads_reduce_clip's two passes
  int once_grid;        // of car_grads_reduce_clip_once's second pass
  bool twice;           // a clipped value of car_grads_reduce_clip may be rounded twice
  int clip_grid;        // of car_grads_clip
  int store_grid;       // of car_grads_reduce: with one rank another kernel than the first pass's
  void* memory;  // one allocation: chunks, partials, counter
  car::GradSource source;  // of car_grads_reduce_clip's second pass
  car::GradPlan plan;
};

namespace {

std::mutex g_mu;
std::unordered_set<const car_grads*> g_live;

car_status fail(cudaError_t e, const char* where) {
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
  car::set_last_error(msg);
  return CAR_ERR_CUDA;
}

car_status refuse(const char* msg, car_status st = CAR_ERR_ARG) {
  car::set_last_error(msg);
  return st;
}

car_status check(const car_grads* g) {
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g || g_live.count(g) == 0) return CAR_ERR_HANDLE;
  }
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(e, "cudaGetDevice");
  return dev == g->device ? CAR_OK : refuse("the gradient handle belongs to another device than the current one");
}

struct Range {
  uintptr_t lo, hi;
  int64_t tensor;
};

// Outputs must not overlap one another, nor an input other than the same
// tensor's at the same address: another CTA could read what this one writes.
car_status check_overlap(int W, int64_t n, const std::vector<int64_t>& bytes, const void* const* inputs,
                         void* const* outs) {
  std::vector<Range> r;
  for (int64_t t = 0; t < n; t++)
    if (bytes[t]) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(outs[t]);
      r.push_back(Range{lo, lo + (uintptr_t)bytes[t], t});
    }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  for (size_t i = 1; i < r.size(); i++)
    if (r[i].lo < r[i - 1].hi) return refuse("two outputs overlap");
  for (int64_t k = 0; k < W * n; k++) {
    const int64_t t = k % n;
    if (!bytes[t]) continue;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(inputs[k]), hi = lo + (uintptr_t)bytes[t];
    // the first output that ends after lo; outputs are disjoint, so ends are sorted too
    auto it = std::upper_bound(r.begin(), r.end(), lo, [](uintptr_t v, const Range& a) { return v < a.hi; });
    for (; it != r.end() && it->lo < hi; ++it)
      if (it->tensor != t || it->lo != lo) return refuse("an output overlaps another tensor's input, or its own at another address");
  }
  return CAR_OK;
}

car_status create(int W, int64_t n, const int64_t* numel, const car_dtype* dtypes, const void* const* inputs,
                  void* const* outs, car_grads** out) {
  if (W < 1 || W > car::kMaxRanks || n < 1 || !numel || !dtypes || !inputs || !outs) return CAR_ERR_ARG;
  if (n > INT32_MAX / car::kMaxRanks) return CAR_ERR_SIZE;
  std::vector<int64_t> bytes((size_t)n);
  int64_t vecs = 0;
  for (int64_t t = 0; t < n; t++) {
    if (dtypes[t] != CAR_BF16 && dtypes[t] != CAR_FP16 && dtypes[t] != CAR_FP32) return CAR_ERR_ARG;
    if (numel[t] < 0) return CAR_ERR_ARG;
    if (numel[t] > ((int64_t)1 << 48)) return CAR_ERR_SIZE;
    const int es = dtypes[t] == CAR_FP32 ? 4 : 2;
    bytes[t] = numel[t] * es;
    vecs += bytes[t] / 16 + 1;
    if (vecs / car::kGradThreads > ((int64_t)1 << 30)) return CAR_ERR_SIZE;  // here, before a sum of many wraps
    if (!bytes[t]) continue;
    if (!outs[t] || reinterpret_cast<uintptr_t>(outs[t]) % es) return outs[t] ? CAR_ERR_ALIGN : CAR_ERR_ARG;
    for (int r = 0; r < W; r++) {
      const void* p = inputs[r * n + t];
      if (!p || reinterpret_cast<uintptr_t>(p) % es) return p ? CAR_ERR_ALIGN : CAR_ERR_ARG;
    }
  }
  car_status st = check_overlap(W, n, bytes, inputs, outs);
  if (st != CAR_OK) return st;

  bool half = false, half_in_place = false, narrow = false, narrow_in_place = false;
  for (int64_t k = 0; k < W * n && W > 1; k++) {
    const int64_t t = k % n;
    if (!bytes[t]) continue;
    const bool is_half = dtypes[t] == CAR_FP16, replaced = inputs[k] == outs[t];
    half = half || is_half;
    narrow = narrow || dtypes[t] != CAR_FP32;
    half_in_place = half_in_place || (is_half && replaced);
    narrow_in_place = narrow_in_place || (dtypes[t] != CAR_FP32 && replaced);
  }
  // (Without fp16 the second pass need not look for infinities: W = 2, 64 M
  // values 89.7 against 91.0 us.)
  const car::GradSource source = W == 1 ? car::GradSource::kInput : half ? car::GradSource::kSums : car::GradSource::kOutput;

  int device = -1, num_sms = 0, l2 = 0, per_reduce = 0, per_sums = 0, per_once = 0, per_clip = 0, per_store = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, device);
  if (e == cudaSuccess) e = car::grads_occupancy(W, W > 1, &per_reduce);
  if (e == cudaSuccess) e = car::grads_occupancy(W, true, &per_store);
  if (e == cudaSuccess) e = car::grads_clip_occupancy(W, source, &per_sums);
  if (e == cudaSuccess && W > 1) e = car::grads_clip_occupancy(W, car::GradSource::kOnce, &per_once);
  if (e == cudaSuccess) e = car::grads_clip_occupancy(W, car::GradSource::kOutput, &per_clip);
  if (e != cudaSuccess) return fail(e, "gradient launch sizes");
  const int64_t reduce_cap = std::min<int64_t>((int64_t)std::max(1, per_reduce) * num_sms, car::kMaxGradCtas);
  const size_t stride = sizeof(car::GradChunk) + (size_t)W * sizeof(void*);
  std::vector<uint8_t> chunks;  // the reduce's list, then the clip's where that is another
  // Appends chunks of one length, so many to each CTA of a resident wave: as
  // long as `limit` vectors allow, and one pass of a CTA's threads at least.
  // (Stretching it until ragged tensor ends fit whole waves too measured no
  // better.)
  auto cut = [&](int64_t limit) {
    const int64_t each = std::max<int64_t>(1, (vecs + reduce_cap * limit - 1) / (reduce_cap * limit));
    const int64_t per_vecs = std::max<int64_t>(car::kGradThreads, (vecs + reduce_cap * each - 1) / (reduce_cap * each));
    const size_t from = chunks.size();
    for (int64_t t = 0; t < n; t++) {
      if (!bytes[t]) continue;
      const int es = dtypes[t] == CAR_FP32 ? 4 : 2, E = 16 / es;
      const uintptr_t off = reinterpret_cast<uintptr_t>(outs[t]) & 15u;
      bool shared = true;
      for (int r = 0; r < W; r++) shared = shared && (reinterpret_cast<uintptr_t>(inputs[r * n + t]) & 15u) == off;
      const int head = (int)((16 - off) & 15u) / es;
      // chunks start on a 16-byte boundary, but for the first, which takes the head too
      for (int64_t b = 0; b < numel[t];) {
        car::GradChunk c;
        c.out = static_cast<uint8_t*>(outs[t]) + b * es;
        c.count = (int32_t)std::min(numel[t] - b, per_vecs * E + (b == 0 && shared ? head : 0));
        c.dtype = (int16_t)dtypes[t];
        c.head = (int16_t)(!shared ? -1 : b == 0 ? head : 0);
        const size_t at = chunks.size();
        chunks.resize(at + stride);
        std::memcpy(chunks.data() + at, &c, sizeof(c));
        for (int r = 0; r < W; r++) {
          const void* p = static_cast<const uint8_t*>(inputs[r * n + t]) + b * es;
          std::memcpy(chunks.data() + at + sizeof(c) + r * sizeof(p), &p, sizeof(p));
        }
        b += c.count;
      }
    }
    return (int64_t)((chunks.size() - from) / stride);
  };
  const int64_t n_reduce = cut(W >= 8 ? car::kGradChunkVecsWide : car::kGradChunkVecs);
  const size_t clip_at = W >= 8 ? chunks.size() : 0;
  const int64_t n_clip = W >= 8 ? cut(car::kGradChunkVecs) : n_reduce;
  const int grid = (int)std::max<int64_t>(1, std::min(n_reduce, reduce_cap));
  const int store_grid = (int)std::min<int64_t>(grid, (int64_t)std::max(1, per_store) * num_sms);
  auto wave = [&](int64_t chunks, int per_sm) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(chunks, (int64_t)std::max(1, per_sm) * num_sms));
  };
  const size_t cb = chunks.size(), pb = (size_t)grid * sizeof(double);
  void* memory = nullptr;
  e = cudaMalloc(&memory, cb + pb + 8);
  if (e != cudaSuccess) return fail(e, "cudaMalloc gradient plan");
  uint8_t* m = static_cast<uint8_t*>(memory);
  if (cb) e = cudaMemcpy(m, chunks.data(), cb, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemset(m + cb, 0, pb + 8);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // the plan is in place for calls on any stream
  car_grads* g = e == cudaSuccess ? new (std::nothrow) car_grads() : nullptr;
  if (!g) {
    cudaFree(memory);
    return e == cudaSuccess ? refuse("out of host memory") : fail(e, "copy gradient plan");
  }
  g->device = device;
  g->grid = grid;
  g->sums_grid = wave(n_clip, per_sums);
  g->once_grid = wave(n_reduce, per_once);
  g->source = source;
  g->twice = narrow;
  g->clip_grid = wave(n_clip, per_clip);
  g->store_grid = store_grid;
  g->memory = memory;
  g->plan.reduce = car::GradList{m, (int)n_reduce};
  g->plan.clip = car::GradList{m + clip_at, (int)n_clip};
  g->plan.W = W;
  g->plan.evict_first = 16 * vecs < 2 * (int64_t)l2;
  g->plan.pass_on = 16 * vecs > (int64_t)l2 / 4;
  g->plan.half_in_place = half_in_place;
  g->plan.narrow_in_place = narrow_in_place;
  g->plan.partial = reinterpret_cast<double*>(m + cb);
  g->plan.arrived = reinterpret_cast<unsigned int*>(m + cb + pb);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    g_live.insert(g);
  }
  *out = g;
  return CAR_OK;
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

extern "C" {

car_status car_grads_create(int W, int64_t n, const int64_t* numel, const car_dtype* dtypes, const void* const* inputs,
                            void* const* outs, car_grads** out) {
  if (!out) return CAR_ERR_ARG;
  *out = nullptr;
  car::set_last_error("");
  try {
    return create(W, n, numel, dtypes, inputs, outs, out);
  } catch (...) {  // host allocation; nothing may leave a C entry point
    return refuse("out of host memory");
  }
}

car_status car_grads_destroy(car_grads* g) {
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g || g_live.erase(g) == 0) return CAR_ERR_HANDLE;
  }
  cudaError_t e = cudaFree(g->memory);
  delete g;
  return e == cudaSuccess ? CAR_OK : fail(e, "cudaFree");
}

car_status car_grads_reduce(car_grads* g, float scale, double* sumsq, void* stream) {
  car_status st = check(g);
  if (st != CAR_OK) return st;
  if (!sumsq || !std::isfinite(scale)) return CAR_ERR_ARG;
  if (!aligned(sumsq, 8)) return CAR_ERR_ALIGN;
  cudaError_t e = car::launch_grads_reduce(g->plan, scale, true, sumsq, false, g->store_grid, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : fail(e, "grads_reduce launch");
}

car_status car_grads_clip(car_grads* g, const double* sumsq, float max_norm, float* norm_out, void* stream) {
  car_status st = check(g);
  if (st != CAR_OK) return st;
  if (!sumsq || !(max_norm >= 0.f)) return CAR_ERR_ARG;
  if (!aligned(sumsq, 8) || !aligned(norm_out, 4)) return CAR_ERR_ALIGN;
  cudaError_t e = car::launch_grads_clip(g->plan, sumsq, 1, 1.f, car::GradSource::kOutput, max_norm, norm_out, g->clip_grid,
                                         static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : fail(e, "grads_clip launch");
}

static car_status reduce_clip(car_grads* g, float scale, float max_norm, float* norm_out, bool once, void* stream) {
  car_status st = check(g);
  if (st != CAR_OK) return st;
  if (!std::isfinite(scale) || !(max_norm >= 0.f)) return CAR_ERR_ARG;
  if (!aligned(norm_out, 4)) return CAR_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool one = g->plan.W == 1;  // the first pass then only reads (see grads.cu)
  once = once && g->twice;  // one rank's values are rounded once as it is, and fp32 sums not at all
  cudaError_t e = car::launch_grads_reduce(g->plan, scale, !one, nullptr, once, g->grid, s);
  if (e == cudaSuccess)
    e = car::launch_grads_clip(g->plan, g->plan.partial, g->grid, scale, once ? car::GradSource::kOnce : g->source, max_norm,
                               norm_out, once ? g->once_grid : g->sums_grid, s);
  return e == cudaSuccess ? CAR_OK : fail(e, "grads_reduce_clip launch");
}

car_status car_grads_reduce_clip(car_grads* g, float scale, float max_norm, float* norm_out, void* stream) {
  return reduce_clip(g, scale, max_norm, norm_out, false, stream);
}

car_status car_grads_reduce_clip_once(car_grads* g, float scale, float max_norm, float* norm_out, void* stream) {
  return reduce_clip(g, scale, max_norm, norm_out, true, stream);
}

}  // extern "C"
