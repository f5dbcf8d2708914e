// grads.cu -- rank sum of many gradient tensors, their global norm, clipping.
//
//   G_t   = scale * sum_r g_{r,t}             (fp32, rank order)
//   norm  = sqrt(sum over all tensors of G^2)
//   out_t = rne_T(G_t) * min(1, max_norm / (norm + 1e-6)), rounded to T again
//
// Two passes: the first reads the W ranks, stores G in the tensors' own type
// and sums G^2 of the unrounded values; the second scales the stored values
// and does nothing when the norm is within the limit.  Keeping G in its type
// between the passes costs a clipped value one more rounding of half a step
// (what calling a reduce and then a clip would give) and keeps the second
// pass at one read and one write of the tensors, from L2 where they fit:
// chunks are taken in the opposite order, the last written first.
//
// Work is cut into chunks of one tensor each; a CTA takes a contiguous share
// of them.  Squares are summed in fp32 over a thread's part of one chunk
// (at most 64 vectors) and in 64 bits from there on; the CTAs' partials are
// added by the last CTA to arrive, in the order of their index, so the same
// call gives the same bits.  Roofline: HBM, (W + 1) * 16 bytes per vector.
#include "car_device.cuh"
#include "car_launch.h"

namespace car {
namespace {

template <int DT>
struct Scalar;
template <>
struct Scalar<kBF16> {
  using T = __nv_bfloat16;
  __device__ __forceinline__ static float up(T v) { return __bfloat162float(v); }
  __device__ __forceinline__ static T down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Scalar<kFP16> {
  using T = __half;
  __device__ __forceinline__ static float up(T v) { return __half2float(v); }
  __device__ __forceinline__ static T down(float v) { return __float2half_rn(v); }
};
template <>
struct Scalar<kFP32> {
  using T = float;
  __device__ __forceinline__ static float up(T v) { return v; }
  __device__ __forceinline__ static T down(float v) { return v; }
};

__device__ __forceinline__ double block_sum(double v, double* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kGradThreads / 32; w++) v += s_warp[w];
  return v;
}

// Parts of a chunk: `head` elements up to a 16-byte boundary, whole vectors,
// and a tail; or, where the pointers share no boundary, all of it as a tail.
struct Span {
  int head, vecs, tail;
};
template <int DT>
__device__ __forceinline__ Span span_of(const GradTensor& t, const GradChunk& c) {
  constexpr int E = Pack<DT>::kN;
  if (t.head < 0) return Span{0, 0, c.count};
  const int head = c.begin == 0 ? min(t.head, c.count) : 0;
  const int vecs = (c.count - head) / E;
  return Span{head, vecs, c.count - head - vecs * E};
}

template <int DT, int W>
__device__ __forceinline__ float sum_chunk(const GradTensor& t, const GradChunk& c, int n, float scale) {
  using S = Scalar<DT>;
  using T = typename S::T;
  constexpr int E = Pack<DT>::kN;
  constexpr int R = W > 0 ? W : kMaxRanks;
  const Span sp = span_of<DT>(t, c);
  float ss = 0.f;
  T* out = static_cast<T*>(t.out) + c.begin;
  const int64_t body = c.begin + sp.head;
  for (int v = threadIdx.x; v < sp.vecs; v += kGradThreads) {
    uint4 raw[R];
#pragma unroll
    for (int r = 0; r < R; r++)
      if (r < n) raw[r] = ld_stream(reinterpret_cast<const uint4*>(static_cast<const T*>(t.in[r]) + body) + v);
    float acc[E];
    rank_sum<DT, R>(raw, n, acc);
#pragma unroll
    for (int e = 0; e < E; e++) {
      acc[e] = __fmul_rn(acc[e], scale);
      ss = fmaf(acc[e], acc[e], ss);
    }
    st16(reinterpret_cast<uint4*>(out + sp.head) + v, Pack<DT>::narrow(acc));
  }
  // the ragged ends
  for (int i = threadIdx.x; i < sp.head + sp.tail; i += kGradThreads) {
    const int at = i < sp.head ? i : i + sp.vecs * E;
    float acc = S::up(static_cast<const T*>(t.in[0])[c.begin + at]);
    for (int r = 1; r < n; r++) acc = __fadd_rn(acc, S::up(static_cast<const T*>(t.in[r])[c.begin + at]));
    acc = __fmul_rn(acc, scale);
    ss = fmaf(acc, acc, ss);
    out[at] = S::down(acc);
  }
  return ss;
}

template <int DT>
__device__ __forceinline__ void clip_chunk(const GradTensor& t, const GradChunk& c, float coef) {
  using S = Scalar<DT>;
  using T = typename S::T;
  constexpr int E = Pack<DT>::kN;
  const Span sp = span_of<DT>(t, c);
  T* out = static_cast<T*>(t.out) + c.begin;
  uint4* body = reinterpret_cast<uint4*>(out + sp.head);
  for (int v = threadIdx.x; v < sp.vecs; v += kGradThreads) {
    float f[E];
    Pack<DT>::widen(body[v], f);
#pragma unroll
    for (int e = 0; e < E; e++) f[e] = __fmul_rn(f[e], coef);
    st16(body + v, Pack<DT>::narrow(f));
  }
  for (int i = threadIdx.x; i < sp.head + sp.tail; i += kGradThreads) {
    const int at = i < sp.head ? i : i + sp.vecs * E;
    out[at] = S::down(__fmul_rn(S::up(out[at]), coef));
  }
}

// This CTA's share [lo, hi) of the chunks.
__device__ __forceinline__ void chunk_share(int64_t n, int64_t* lo, int64_t* hi) {
  const int64_t share = n / gridDim.x, extra = n % gridDim.x;
  *lo = share * blockIdx.x + (blockIdx.x < extra ? blockIdx.x : extra);
  *hi = *lo + share + (blockIdx.x < extra ? 1 : 0);
}

template <int W>
__global__ void __launch_bounds__(kGradThreads)
    grads_reduce_kernel(const GradPlan p, const float scale, double* __restrict__ sumsq) {
  __shared__ double s_warp[kGradThreads / 32];
  __shared__ bool s_last;
  const int n = W > 0 ? W : p.W;
  int64_t lo, hi;
  chunk_share(p.n_chunks, &lo, &hi);
  pdl_wait_and_release();
  double total = 0.0;
  for (int64_t i = lo; i < hi; i++) {
    const GradChunk c = p.chunks[i];
    const GradTensor& t = p.tensors[c.tensor];
    float ss;
    switch (t.dtype) {
      case kBF16: ss = sum_chunk<kBF16, W>(t, c, n, scale); break;
      case kFP16: ss = sum_chunk<kFP16, W>(t, c, n, scale); break;
      default: ss = sum_chunk<kFP32, W>(t, c, n, scale); break;
    }
    total += (double)ss;
  }
  total = block_sum(total, s_warp);
  if (threadIdx.x == 0) {
    p.partial[blockIdx.x] = total;
    __threadfence();
    s_last = atomicAdd(p.arrived, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (s_last) {
    __threadfence();
    total = 0.0;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kGradThreads) total += __ldcg(p.partial + i);
    total = block_sum(total, s_warp);
    if (threadIdx.x == 0) {
      *sumsq = total;
      *p.arrived = 0u;  // for the next call, which waits for this grid
    }
  }
}

__global__ void __launch_bounds__(kGradThreads)
    grads_clip_kernel(const GradPlan p, const double* __restrict__ sumsq, const float max_norm, float* __restrict__ norm_out) {
  pdl_wait_and_release();
  const double norm = sqrt(*sumsq);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double ratio = (double)max_norm / (norm + 1e-6);
  // within the limit, or no limit (false for a NaN norm, which then reaches every value)
  if (ratio >= 1.0 || isinf(max_norm)) return;
  const float coef = (float)ratio;
  int64_t lo, hi;
  chunk_share(p.n_chunks, &lo, &hi);
  for (int64_t i = hi - 1; i >= lo; i--) {
    const GradChunk c = p.chunks[i];
    const GradTensor& t = p.tensors[c.tensor];
    switch (t.dtype) {
      case kBF16: clip_chunk<kBF16>(t, c, coef); break;
      case kFP16: clip_chunk<kFP16>(t, c, coef); break;
      default: clip_chunk<kFP32>(t, c, coef); break;
    }
  }
}

using GradsFn = void (*)(const GradPlan, const float, double*);
GradsFn pick_grads(int W) {
  switch (W) {
    case 1: return grads_reduce_kernel<1>;
    case 2: return grads_reduce_kernel<2>;
    case 4: return grads_reduce_kernel<4>;
    case 8: return grads_reduce_kernel<8>;
    case 16: return grads_reduce_kernel<16>;
    default: return grads_reduce_kernel<0>;
  }
}

}  // namespace

cudaError_t grads_occupancy(int W, int* reduce_blocks_per_sm, int* clip_blocks_per_sm) {
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
      reduce_blocks_per_sm, reinterpret_cast<const void*>(pick_grads(W)), kGradThreads, 0);
  if (e != cudaSuccess) return e;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(clip_blocks_per_sm,
                                                       reinterpret_cast<const void*>(grads_clip_kernel), kGradThreads, 0);
}

cudaError_t launch_grads_reduce(const GradPlan& plan, float scale, double* sumsq, int grid, cudaStream_t s) {
  return launch_pdl(pick_grads(plan.W), (unsigned)grid, kGradThreads, 0, s, 1, plan, scale, sumsq);
}

cudaError_t launch_grads_clip(const GradPlan& plan, const double* sumsq, float max_norm, float* norm_out, int grid,
                              cudaStream_t s) {
  return launch_pdl(grads_clip_kernel, (unsigned)grid, kGradThreads, 0, s, 1, plan, sumsq, max_norm, norm_out);
}

}  // namespace car
