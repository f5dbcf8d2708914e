// grads_api.cu -- the C ABI's gradient handles (include/car.h, car_grads_*):
// argument checks, the plan of chunks, launch sizes.  Everything is computed
// in the kernels of grads.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <unordered_set>
#include <vector>

#include "../../include/car.h"
#include "car_device.cuh"
#include "car_launch.h"

struct car_grads {
  int device;
  int reduce_grid, clip_grid;
  void* memory;  // one allocation: tensors, chunks, partials, sum, counter
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
  int64_t n_chunks = 0;
  for (int64_t t = 0; t < n; t++) {
    if (dtypes[t] != CAR_BF16 && dtypes[t] != CAR_FP16 && dtypes[t] != CAR_FP32) return CAR_ERR_ARG;
    if (numel[t] < 0) return CAR_ERR_ARG;
    if (numel[t] > ((int64_t)1 << 48)) return CAR_ERR_SIZE;
    const int es = dtypes[t] == CAR_FP32 ? 4 : 2;
    bytes[t] = numel[t] * es;
    n_chunks += bytes[t] / (16 * car::kGradChunkVecs) + 2;
    if (!bytes[t]) continue;
    if (!outs[t] || reinterpret_cast<uintptr_t>(outs[t]) % es) return outs[t] ? CAR_ERR_ALIGN : CAR_ERR_ARG;
    for (int r = 0; r < W; r++) {
      const void* p = inputs[r * n + t];
      if (!p || reinterpret_cast<uintptr_t>(p) % es) return p ? CAR_ERR_ALIGN : CAR_ERR_ARG;
    }
  }
  if (n_chunks > ((int64_t)1 << 31)) return CAR_ERR_SIZE;
  car_status st = check_overlap(W, n, bytes, inputs, outs);
  if (st != CAR_OK) return st;

  std::vector<car::GradTensor> tensors((size_t)n);
  std::vector<car::GradChunk> chunks;
  chunks.reserve((size_t)n_chunks);
  for (int64_t t = 0; t < n; t++) {
    car::GradTensor& g = tensors[t];
    std::memset(&g, 0, sizeof(g));
    if (!bytes[t]) continue;
    const int es = dtypes[t] == CAR_FP32 ? 4 : 2, E = 16 / es;
    const uintptr_t off = reinterpret_cast<uintptr_t>(outs[t]) & 15u;
    bool shared = true;
    for (int r = 0; r < W; r++) {
      g.in[r] = inputs[r * n + t];
      shared = shared && (reinterpret_cast<uintptr_t>(g.in[r]) & 15u) == off;
    }
    g.out = outs[t];
    g.dtype = (int32_t)dtypes[t];
    const int head = (int)((16 - off) & 15u) / es;
    g.head = shared ? head : -1;
    // chunks start on a 16-byte boundary, but for the first, which takes the head too
    const int64_t per = (int64_t)car::kGradChunkVecs * E;
    for (int64_t b = 0; b < numel[t];) {
      const int64_t count = std::min(numel[t] - b, per + (b == 0 && shared ? head : 0));
      chunks.push_back(car::GradChunk{b, (int32_t)count, (int32_t)t});
      b += count;
    }
  }

  car_grads* g = new car_grads();
  g->memory = nullptr;
  cudaError_t e = cudaGetDevice(&g->device);
  int num_sms = 0, per_reduce = 0, per_clip = 0;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, g->device);
  if (e == cudaSuccess) e = car::grads_occupancy(W, &per_reduce, &per_clip);
  if (e != cudaSuccess) {
    delete g;
    return fail(e, "gradient launch sizes");
  }
  const int64_t most = std::max<int64_t>(1, (int64_t)chunks.size());
  g->reduce_grid = (int)std::min<int64_t>(most, (int64_t)std::max(1, per_reduce) * num_sms);
  g->clip_grid = (int)std::min<int64_t>(most, (int64_t)std::max(1, per_clip) * num_sms);
  const size_t tb = tensors.size() * sizeof(car::GradTensor), cb = chunks.size() * sizeof(car::GradChunk);
  const size_t pb = (size_t)g->reduce_grid * sizeof(double);
  e = cudaMalloc(&g->memory, tb + cb + pb + 16);
  if (e != cudaSuccess) {
    delete g;
    return fail(e, "cudaMalloc gradient plan");
  }
  uint8_t* m = static_cast<uint8_t*>(g->memory);
  e = cudaMemcpy(m, tensors.data(), tb, cudaMemcpyHostToDevice);
  if (e == cudaSuccess && cb) e = cudaMemcpy(m + tb, chunks.data(), cb, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemset(m + tb + cb, 0, pb + 16);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // the plan is in place for calls on any stream
  if (e != cudaSuccess) {
    cudaFree(g->memory);
    delete g;
    return fail(e, "copy gradient plan");
  }
  g->plan.tensors = reinterpret_cast<const car::GradTensor*>(m);
  g->plan.chunks = reinterpret_cast<const car::GradChunk*>(m + tb);
  g->plan.n_chunks = (int64_t)chunks.size();
  g->plan.W = W;
  g->plan.partial = reinterpret_cast<double*>(m + tb + cb);
  g->plan.sumsq = reinterpret_cast<double*>(m + tb + cb + pb);
  g->plan.arrived = reinterpret_cast<unsigned int*>(m + tb + cb + pb + 8);
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
  cudaError_t e = car::launch_grads_reduce(g->plan, scale, sumsq, g->reduce_grid, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : fail(e, "grads_reduce launch");
}

car_status car_grads_clip(car_grads* g, const double* sumsq, float max_norm, float* norm_out, void* stream) {
  car_status st = check(g);
  if (st != CAR_OK) return st;
  if (!sumsq || !(max_norm >= 0.f)) return CAR_ERR_ARG;
  if (!aligned(sumsq, 8) || !aligned(norm_out, 4)) return CAR_ERR_ALIGN;
  cudaError_t e = car::launch_grads_clip(g->plan, sumsq, max_norm, norm_out, g->clip_grid, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : fail(e, "grads_clip launch");
}

car_status car_grads_reduce_clip(car_grads* g, float scale, float max_norm, float* norm_out, void* stream) {
  car_status st = check(g);
  if (st != CAR_OK) return st;
  if (!std::isfinite(scale) || !(max_norm >= 0.f)) return CAR_ERR_ARG;
  if (!aligned(norm_out, 4)) return CAR_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = car::launch_grads_reduce(g->plan, scale, g->plan.sumsq, g->reduce_grid, s);
  if (e == cudaSuccess) e = car::launch_grads_clip(g->plan, g->plan.sumsq, max_norm, norm_out, g->clip_grid, s);
  return e == cudaSuccess ? CAR_OK : fail(e, "grads_reduce_clip launch");
}

}  // extern "C"
