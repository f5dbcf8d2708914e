// dropout.cu -- rank sum and dropout in one pass (an embedding that is split
// over the ranks); its backward is the same call on the gradient's ranks.
//
// Laid out as reduce.cu: every CTA takes one contiguous, equal share of the
// vectors, a thread keeps U x W independent 16-byte loads in flight.  The mask
// is computed where it is used (branch.cuh), from the vector's place in the
// [M, N] problem, so it costs no bytes.  Roofline: HBM, (W + 1) * 16 bytes per
// vector, next to the generator's 18 wide products.
#include "branch.cuh"
#include "car_launch.h"

namespace car {
namespace {

template <int DT, int W, int U>
__global__ void __launch_bounds__(kReduceThreads)
    rank_sum_dropout_kernel(const RankPtrs in, const int nranks, const DropParams drop, uint4* __restrict__ out,
                            const int64_t nvec) {
  constexpr int E = Pack<DT>::kN;
  constexpr int R = W > 0 ? W : kMaxRanks;
  const int n = W > 0 ? W : nranks;
  const int64_t share = nvec / gridDim.x, extra = nvec % gridDim.x;
  const int64_t lo = share * blockIdx.x + (blockIdx.x < extra ? blockIdx.x : extra);
  const int64_t hi = lo + share + (blockIdx.x < extra ? 1 : 0);
  pdl_wait_and_release();
  const DropState state = drop_state(drop);
  for (int64_t base = lo + threadIdx.x; base < hi; base += kReduceThreads * U) {
    uint4 raw[U][R];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t v = base + (int64_t)u * kReduceThreads;
      if (v < hi) {
#pragma unroll
        for (int r = 0; r < R; r++)
          if (r < n) raw[u][r] = ld_stream(static_cast<const uint4*>(in.p[r]) + v);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t v = base + (int64_t)u * kReduceThreads;
      if (v < hi) {
        float acc[E];
        rank_sum<DT, R>(raw[u], n, acc);
        float2 z[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[e] = make_float2(acc[2 * e], acc[2 * e + 1]);
        if (drop.active) {
          uint32_t bits[E / 2];
          drop_bits<E>(state, v, bits);
#pragma unroll
          for (int e = 0; e < E / 2; e++) z[e] = drop2(drop, bits[e], z[e]);
        }
        st16(out + v, narrow2<DT>(z));
      }
    }
  }
}

using DropoutFn = void (*)(const RankPtrs, const int, const DropParams, uint4*, const int64_t);

// As many vectors per thread as the plain rank sum takes.
constexpr int vectors_for(int W) { return W <= 4 ? 4 : (W == 16 ? 2 : 1); }

template <int DT>
DropoutFn pick_ranks(int W) {
  switch (W) {
    case 1: return rank_sum_dropout_kernel<DT, 1, vectors_for(1)>;
    case 2: return rank_sum_dropout_kernel<DT, 2, vectors_for(2)>;
    case 4: return rank_sum_dropout_kernel<DT, 4, vectors_for(4)>;
    case 8: return rank_sum_dropout_kernel<DT, 8, vectors_for(8)>;
    case 16: return rank_sum_dropout_kernel<DT, 16, vectors_for(16)>;
    default: return rank_sum_dropout_kernel<DT, 0, 1>;
  }
}
DropoutFn pick(int dtype, int W) {
  switch (dtype) {
    case kBF16: return pick_ranks<kBF16>(W);
    case kFP16: return pick_ranks<kFP16>(W);
    default: return pick_ranks<kFP32>(W);
  }
}

}  // namespace

int dropout_vectors_per_thread(int W) {
  return (W == 1 || W == 2 || W == 4 || W == 8 || W == 16) ? vectors_for(W) : 1;
}

cudaError_t dropout_occupancy(int dtype, int W, int* blocks_per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, reinterpret_cast<const void*>(pick(dtype, W)),
                                                       kReduceThreads, 0);
}

cudaError_t launch_dropout(int dtype, int W, const RankPtrs& in, const DropParams& drop, void* out, int64_t nvec, int grid,
                           cudaStream_t s) {
  return launch_pdl(pick(dtype, W), (unsigned)grid, kReduceThreads, 0, s, 1, in, W, drop, static_cast<uint4*>(out), nvec);
}

}  // namespace car
