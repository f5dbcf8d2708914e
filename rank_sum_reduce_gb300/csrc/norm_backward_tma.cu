// norm_backward_tma.cu -- backward of rank sum + residual add + RMSNorm for
// many rows, with the row slices streamed into shared memory by TMA bulk
// copies.  Same operation as norm_backward.cu, organised as the forward's
// pipeline kernel (fused_tma.cuh): one persistent CTA per SM takes rows
// blockIdx.x, blockIdx.x + grid, ...; a producer thread keeps a ring of about
// one row's slices in flight -- dy_0 .. dy_{W-1}, h, dres -- while the
// consumer warps fold them into fp32 accumulators in rank order.
//
// h stays in registers (packed) from the statistic to the gradient; the dres
// slice is only waited for after the statistic and is read from its slot
// there.  The weight row and the weight gradient of the CTA's rows stay in
// registers for the whole kernel.  Every mbarrier wait is bounded, as in the
// forward.
#include "ring.cuh"
#include "car_launch.h"

namespace car {
namespace {

struct BackwardTmaParams {
  RankPtrs dy;
  const uint8_t* h;
  const uint8_t* dres;  // may be null
  const uint4* weight;
  uint4* dx;
  float* partial;       // [grid, N], or null
  unsigned int* err;
  float eps;
  float cols;
  int64_t rows;
  int row_bytes;
  int vec_per_row;
  int slots;
  int slices;           // per row: W ranks, h, dres
  int consumers;        // consumer threads (multiple of 32)
  int nranks;
};

__device__ __forceinline__ const uint8_t* slice_source(const BackwardTmaParams& p, int q, int n) {
  return q < n ? static_cast<const uint8_t*>(p.dy.p[q]) : (q == n ? p.h : p.dres);
}

// As the forward's producer: keeps the ring full, then waits for every copy
// that it issued.
__device__ __forceinline__ void produce(const BackwardTmaParams& p, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                        volatile int* s_abort, int n) {
  const int S = p.slots;
  const uint32_t slice = (uint32_t)p.row_bytes;
  int slot = 0;
  uint32_t phase = 0;
  uint64_t issued = 0;
  bool ok = true;
  for (int64_t row = blockIdx.x; row < p.rows && ok; row += gridDim.x) {
    const int64_t off = row * (int64_t)p.row_bytes;
    for (int q = 0; q < p.slices; q++) {
      if (issued >= (uint64_t)S && !wait_bounded(&empty[slot], phase ^ 1u, s_abort)) {
        ok = false;
        break;
      }
      mbar_arrive_expect_tx(&full[slot], slice);
      bulk_load(ring + (size_t)slot * slice, slice_source(p, q, n) + off, slice, &full[slot]);
      issued++;
      if (++slot == S) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  if (!ok) {
    atomicOr(p.err, 1u);
    *s_abort = 1;
  }
  const int used = issued < (uint64_t)S ? (int)issued : S;
  for (int k = 0; k < used; k++) {  // copy number c is use c / S of slot c % S
    const uint64_t c = issued - 1 - (uint64_t)k;
    if (!wait_bounded_drain(&full[c % (uint64_t)S], (uint32_t)((c / (uint64_t)S) & 1u))) atomicOr(p.err, 1u);
  }
}

template <int DT, int VPT>
__device__ __forceinline__ void consume(const BackwardTmaParams& p, const uint8_t* ring, uint64_t* full, uint64_t* empty,
                                        uint64_t* rowbar, float2* s_warp, volatile int* s_abort, int n, int nwarps) {
  constexpr int E = Pack<DT>::kN;
  const int S = p.slots, slice = p.row_bytes, T = p.consumers;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint4 wv[VPT];
  float dw[VPT][E];
  bool ok[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const int v = threadIdx.x + k * T;
    ok[k] = v < p.vec_per_row;
    wv[k] = ok[k] ? __ldg(p.weight + v) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int e = 0; e < E; e++) dw[k][e] = 0.f;
  }
  int slot = 0;
  uint32_t phase = 0, it = 0;
  bool failed = false;
  auto release = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
  };
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, it++) {
    float g[VPT][E];
    uint4 hv[VPT];
    float ss = 0.f, c = 0.f;
    for (int q = 0; q < n; q++) {
      if (!wait_bounded(&full[slot], phase, s_abort)) {
        failed = true;
        break;
      }
      const uint8_t* sl = ring + (size_t)slot * slice;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        if (ok[k]) {
          float t[E];
          Pack<DT>::widen(lds16(sl + 16 * (threadIdx.x + k * T)), t);
#pragma unroll
          for (int e = 0; e < E; e++) g[k][e] = q == 0 ? t[e] : __fadd_rn(g[k][e], t[e]);
        }
      }
      release();
    }
    if (failed || !wait_bounded(&full[slot], phase, s_abort)) {
      failed = true;
      break;
    }
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        hv[k] = lds16(ring + (size_t)slot * slice + 16 * (threadIdx.x + k * T));
        float hf[E], wf[E];
        Pack<DT>::widen(hv[k], hf);
        Pack<DT>::widen(wv[k], wf);
#pragma unroll
        for (int e = 0; e < E; e++) {
          ss = fmaf(hf[e], hf[e], ss);
          c = fmaf(__fmul_rn(g[k][e], wf[e]), hf[e], c);
        }
      }
    }
    release();
    // row statistics: every warp adds the warp partials itself, in the same
    // order; they are double-buffered by row parity
    ss = warp_sum(ss);
    c = warp_sum(c);
    float2* sw = s_warp + 16 * (it & 1u);
    if (lane == 0) {
      sw[warp] = make_float2(ss, c);
      mbar_arrive(rowbar);
    }
    if (!wait_bounded(rowbar, it & 1u, s_abort)) {
      failed = true;
      break;
    }
    const float2 mine = lane < nwarps ? sw[lane] : make_float2(0.f, 0.f);
    const float rms = rsqrtf(__fdiv_rn(warp_sum(mine.x), p.cols) + p.eps);
    const float m = __fdiv_rn(__fmul_rn(warp_sum(mine.y), rms), p.cols);
    if (p.dres && !wait_bounded(&full[slot], phase, s_abort)) {
      failed = true;
      break;
    }
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
        const int v = threadIdx.x + k * T;
        float hf[E], wf[E], df[E], o[E];
        Pack<DT>::widen(hv[k], hf);
        Pack<DT>::widen(wv[k], wf);
        Pack<DT>::widen(p.dres ? lds16(ring + (size_t)slot * slice + 16 * v) : make_uint4(0u, 0u, 0u, 0u), df);
#pragma unroll
        for (int e = 0; e < E; e++) {
          const float u = __fmul_rn(hf[e], rms);
          dw[k][e] = fmaf(g[k][e], u, dw[k][e]);
          o[e] = fmaf(rms, fmaf(-u, m, __fmul_rn(g[k][e], wf[e])), df[e]);
        }
        st16(p.dx + row * (int64_t)p.vec_per_row + v, Pack<DT>::narrow(o));
      }
    }
    if (p.dres) release();
  }
  if (failed) {
    atomicOr(p.err, 1u);
    *s_abort = 1;
    return;
  }
  if (p.partial) {
    float* to = p.partial + blockIdx.x * (int64_t)p.vec_per_row * E;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      if (ok[k]) {
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *reinterpret_cast<float4*>(to + (threadIdx.x + k * T) * E + e) =
              make_float4(dw[k][e], dw[k][e + 1], dw[k][e + 2], dw[k][e + 3]);
      }
    }
  }
}

template <int DT, int W, int VPT>
__global__ void __launch_bounds__(544, 1) reduce_rmsnorm_backward_tma_kernel(const BackwardTmaParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int S = p.slots;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)S * p.row_bytes);
  uint64_t* empty = full + S;
  uint64_t* rowbar = empty + S;
  float2* s_warp = reinterpret_cast<float2*>(rowbar + 1);  // [2][16]
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_warp + 32);
  const int n = W > 0 ? W : p.nranks;
  const int nwarps = p.consumers >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], (uint32_t)nwarps);
    }
    mbar_init(rowbar, (uint32_t)nwarps);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the first row into L2 while the previous grid of the stream finishes
  if (warp == nwarps && lane < p.slices)
    prefetch_l2(slice_source(p, lane, n) + blockIdx.x * (int64_t)p.row_bytes, (uint32_t)p.row_bytes);
  __syncthreads();
  pdl_wait_and_release();
  if (warp == nwarps) {
    if (lane == 0) produce(p, smem, full, empty, s_abort, n);
  } else {
    consume<DT, VPT>(p, smem, full, empty, rowbar, s_warp, s_abort, n, nwarps);
  }
}

using BackwardTmaFn = void (*)(const BackwardTmaParams);

template <int DT, int VPT>
BackwardTmaFn pick_w(int W) {
  switch (W) {
    case 1: return reduce_rmsnorm_backward_tma_kernel<DT, 1, VPT>;
    case 2: return reduce_rmsnorm_backward_tma_kernel<DT, 2, VPT>;
    case 4: return reduce_rmsnorm_backward_tma_kernel<DT, 4, VPT>;
    case 8: return reduce_rmsnorm_backward_tma_kernel<DT, 8, VPT>;
    case 16: return reduce_rmsnorm_backward_tma_kernel<DT, 16, VPT>;
    default: return reduce_rmsnorm_backward_tma_kernel<DT, 0, VPT>;
  }
}
template <int DT>
BackwardTmaFn pick_vpt(int W, int vpt) {
  return vpt == 1 ? pick_w<DT, 1>(W) : vpt == 2 ? pick_w<DT, 2>(W) : nullptr;
}
BackwardTmaFn pick(int dtype, int W, int vpt) {
  switch (dtype) {
    case kBF16: return pick_vpt<kBF16>(W, vpt);
    case kFP16: return pick_vpt<kFP16>(W, vpt);
    default: return pick_vpt<kFP32>(W, vpt);
  }
}

constexpr int kRingBudget = 200 * 1024;

}  // namespace

bool backward_tma_shape(int64_t rows, int vec_per_row, int num_sms, int W, FusedTmaShape* out) {
  if (vec_per_row > 1024) return false;  // two vectors per thread at most: accumulators, h and dweight share 120 registers
  const int slice = vec_per_row * 16;
  out->cluster = 1;
  out->ls = 0;
  out->vpt = vec_per_row > 512 ? 2 : 1;
  const int per = (vec_per_row + out->vpt - 1) / out->vpt;
  out->consumers = (per + 31) / 32 * 32;
  int slots = W + 2 < 6 ? 6 : W + 2;
  if (slots > kRingBudget / slice) slots = kRingBudget / slice;
  out->slots = slots;
  out->grid = (int)(rows < num_sms ? rows : num_sms);
  out->smem = slots * slice + (2 * slots + 1) * 8 + 32 * 8 + 16;
  return slots >= 2;
}

cudaError_t backward_tma_prepare(int dtype, int W, const FusedTmaShape& sh) {
  BackwardTmaFn fn = pick(dtype, W, sh.vpt);
  if (!fn) return cudaErrorInvalidValue;
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, sh.smem);
}

cudaError_t launch_backward_tma(int dtype, int W, const RankPtrs& dy, const void* h, const void* weight, float eps,
                                const void* dres, void* dx, float* dweight, float* workspace, unsigned int* err,
                                int64_t rows, int64_t cols, int vec_per_row, const FusedTmaShape& sh, cudaStream_t s) {
  BackwardTmaFn fn = pick(dtype, W, sh.vpt);
  if (!fn) return cudaErrorInvalidValue;
  BackwardTmaParams p;
  p.dy = dy;
  p.h = static_cast<const uint8_t*>(h);
  p.dres = static_cast<const uint8_t*>(dres);
  p.weight = static_cast<const uint4*>(weight);
  p.dx = static_cast<uint4*>(dx);
  p.partial = dweight ? (sh.grid > 1 ? workspace : dweight) : nullptr;
  p.err = err;
  p.eps = eps;
  p.cols = (float)cols;
  p.rows = rows;
  p.row_bytes = vec_per_row * 16;
  p.vec_per_row = vec_per_row;
  p.slots = sh.slots;
  p.slices = W + 1 + (dres ? 1 : 0);
  p.consumers = sh.consumers;
  p.nranks = W;
  cudaError_t e = launch_pdl(fn, (unsigned)sh.grid, (unsigned)(sh.consumers + 32), (size_t)sh.smem, s, 1, p);
  if (e != cudaSuccess || !dweight || sh.grid == 1) return e;
  return launch_sum_partials(workspace, dweight, sh.grid, cols, s);
}

}  // namespace car
