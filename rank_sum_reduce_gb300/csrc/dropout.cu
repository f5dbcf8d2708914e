// dropout.cu -- rank sum and dropout in one pass (an embedding that is split
// over the ranks); its backward is the same call on the gradient's ranks.
//
// A thread keeps U x W independent 16-byte loads in flight.  The grid passes over the
// vectors in order, so that at any time it reads one region of each rank, and shares
// what is left for the last pass equally: with one contiguous share per CTA instead
// W = 8, M = 4099, N = 4096 bf16 took 48.2 us (46.0), W = 1, M = 16389 47.3 (43.4);
// without the equal last pass W = 8, M = 500 7.3 (7.0).  The mask
// is computed where it is used (branch.cuh), from the vector's place in the
// [M, N] problem, so it costs no bytes.  Roofline: HBM, (W + 1) * 16 bytes per
// vector, next to the generator's 18 wide products.
#include "branch.cuh"
#include "car_launch.h"

namespace car {
namespace {

template <int DT, int W, int U>
__global__ void __launch_bounds__(kReduceThreads)
    rank_sum_dropout_kernel(const RankPtrs in, const DropParams drop, uint4* __restrict__ out, const int64_t nvec) {
  constexpr int E = Pack<DT>::kN;
  constexpr int PASS = kReduceThreads * U;
  const int64_t wave = (int64_t)gridDim.x * PASS, waves = nvec / wave;
  const int64_t left = nvec - waves * wave, share = left / gridDim.x, extra = left % gridDim.x;
  pdl_wait_and_release();
  const DropState state = drop_state(drop);
  for (int64_t i = 0; i < waves + (left > 0 ? 1 : 0); i++) {
    int64_t lo = i * wave + (int64_t)blockIdx.x * PASS, hi = lo + PASS;
    if (i == waves) {
      lo = i * wave + share * blockIdx.x + (blockIdx.x < extra ? blockIdx.x : extra);
      hi = lo + share + (blockIdx.x < extra ? 1 : 0);
    }
    const int64_t base = lo + threadIdx.x;
    uint4 raw[U][W];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t v = base + (int64_t)u * kReduceThreads;
      if (v < hi) {
#pragma unroll
        for (int r = 0; r < W; r++) raw[u][r] = ld_stream(static_cast<const uint4*>(in.p[r]) + v);
      }
    }
    // the masks while the loads are on their way
    uint32_t bits[U][E / 2];
    if (drop.active) {
#pragma unroll
      for (int u = 0; u < U; u++) drop_bits_here<E>(state, base + (int64_t)u * kReduceThreads, bits[u]);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t v = base + (int64_t)u * kReduceThreads;
      if (v < hi) {
        float acc[E];
        rank_sum<DT, W>(raw[u], W, acc);
        float2 z[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; e++) z[e] = make_float2(acc[2 * e], acc[2 * e + 1]);
        if (drop.active) {
#pragma unroll
          for (int e = 0; e < E / 2; e++) z[e] = drop2(drop, bits[u][e], z[e]);
        }
        st16(out + v, narrow2<DT>(z));
      }
    }
  }
}

using DropoutFn = void (*)(const RankPtrs, const DropParams, uint4*, const int64_t);

// Vectors per thread and pass: 8 to 32 loads in flight.  W = 1, M = 16389, N = 4096
// bf16 46.7 us with four, 46.5 with two, M = 1000 4.1 and 4.8; W = 8, M = 500 7.1 us with
// two, 7.4 with one.
constexpr int vectors_for(int W) { return W <= 4 ? 4 : 2; }

// An instance for every rank count: one that holds registers for 16 ranks took 32.3 us
// for W = 3, M = 4000, N = 4096, with a floor of 19.3.
template <int DT, int W>
DropoutFn pick_ranks(int w) {
  if constexpr (W < kMaxRanks) {
    if (w > W) return pick_ranks<DT, W + 1>(w);
  }
  return rank_sum_dropout_kernel<DT, W, vectors_for(W)>;
}
DropoutFn pick(int dtype, int W) {
  switch (dtype) {
    case kBF16: return pick_ranks<kBF16, 1>(W);
    case kFP16: return pick_ranks<kFP16, 1>(W);
    default: return pick_ranks<kFP32, 1>(W);
  }
}

}  // namespace

int dropout_vectors_per_thread(int W) {
  return vectors_for(W);
}

cudaError_t dropout_occupancy(int dtype, int W, int* blocks_per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, reinterpret_cast<const void*>(pick(dtype, W)),
                                                       kReduceThreads, 0);
}

cudaError_t launch_dropout(int dtype, int W, const RankPtrs& in, const DropParams& drop, void* out, int64_t nvec, int grid,
                           cudaStream_t s) {
  return launch_pdl(pick(dtype, W), (unsigned)grid, kReduceThreads, 0, s, 1, in, drop, static_cast<uint4*>(out), nvec);
}

}  // namespace car
