// branch.h -- launch entry points of the kernels of a block's branch: the norm
// behind the block, gate, dropout and residual scale between rank sum and
// residual add (internal; arguments are checked in branch_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "car_launch.h"

namespace car {

struct DropParams {
  uint32_t key0, key1;
  uint64_t offset;
  const uint64_t* offset_dev;  // added to offset by the kernel; may be null
  bool active;                 // something is dropped
  uint32_t limit;              // 65536 t - 1, t of 65536 being dropped
  float scale;                 // of what is kept
};

// Pointers are device memory; what may be null is missing then.
struct BranchArgs {
  const void* norm_weight;  // may be null
  float norm_eps;
  const void* gate;         // may be null
  int64_t gate_span;        // rows that share a gate row; 0: each has its own
  float residual_scale;
  DropParams drop;
};
struct BranchGradArgs {
  const void* ar;           // may be null where nothing reads it
  const void* h;
  const void* dres;         // may be null
  void* dx;
  void* dresidual;          // may be null
  float* dweight;           // may be null
  float* dnorm_weight;      // may be null
  void* dgate;              // may be null
  float* workspace;
};

// ---- dropout of the rank sum (dropout.cu) ----
cudaError_t dropout_occupancy(int dtype, int W, int* blocks_per_sm);
int dropout_vectors_per_thread(int W);
cudaError_t launch_dropout(int dtype, int W, const RankPtrs& in, const DropParams& drop, void* out, int64_t nvec, int grid,
                           cudaStream_t s);

// ---- forward (branch_rows.cu) ----
constexpr int kBranchThreads = 512;
cudaError_t branch_resident_groups(int dtype, int W, const FusedShape& sh, int num_sms, int* groups);
cudaError_t launch_branch(int dtype, int W, const RankPtrs& in, const BranchArgs& br, const void* residual,
                          const void* weight, float eps, void* residual_out, void* norm_out, void* ar_out,
                          unsigned int* err, int64_t rows, int64_t cols, int vec_per_row, const FusedShape& sh,
                          const WaitHook& hook, cudaStream_t s);

struct BranchTeams : TeamShape {  // teams: rows of a tile; grid: CTAs
  int cluster;                    // CTAs that share a row, then with one team each
};
// ---- forward, many rows (branch_tma.cu, branch_tma.cuh) ----
void branch_tma_shape(int64_t rows, int vec_per_row, int num_sms, BranchTeams* out);
// Allows the instances their shared memory, and fits the grid to the clusters that can be resident.
cudaError_t branch_tma_prepare(int dtype, BranchTeams* sh);
cudaError_t launch_branch_tma(int dtype, int W, const RankPtrs& in, const BranchArgs& br, const void* residual,
                              const void* weight, float eps, void* residual_out, void* norm_out, void* ar_out,
                              unsigned int* err, int64_t rows, int64_t cols, int vec_per_row, const BranchTeams& sh,
                              const WaitHook& hook, cudaStream_t s);
// The ring of either pipeline (branch_ring.cuh).
constexpr int kMaxRingStages = 32;
struct RingPlan {
  int rows;
  int row_bytes;
  int vec_per_row;
  int cluster;          // CTAs that share a row
  int chunk;            // vectors of a row for each of them (the last one's may be fewer)
  int ranks;            // slices of a tile that are summed
  int held;             // slices that a row needs to its end
  int group;            // slices that a stage has room for
  int tile_stages;      // stages of a tile
  int stages;           // of the ring
  int teams;            // rows of a tile, each for a team of consumer warps
  int producers;        // threads, each in a warp of its own, that issue a stage's copies
  int team_threads;     // multiple of 32
  uint32_t gate_span;   // tiles end where a gate row's rows end; 0: they need not
};
// Chooses group, tile_stages and stages for `budget` bytes; false when the ring
// would be too small.
bool branch_ring_fit(int budget, RingPlan* p);
// Teams and grid for `cluster` CTAs a row and `vpt` vectors per thread.
void branch_teams(int64_t rows, int vec_per_row, int num_sms, int cluster, int vpt, BranchTeams* out);
// The clusters of `fn` that can be resident, at most *clusters.
cudaError_t branch_clusters(const void* fn, int cluster, int smem, int* clusters);

// ---- backward (branch_backward.cu) ----
// CTAs (or clusters) take contiguous spans of rows: the g-th of n starts here.
__host__ __device__ inline int64_t span_start(int64_t rows, int n, int g) {
  return (int64_t)((uint64_t)rows * (uint64_t)g / (uint64_t)n);
}
// Most CTAs (or clusters) that leave partial sums.
constexpr int kMaxBranchGroups = 304;
// Floats of the workspace for `groups` of them (0 for one): partials of dweight
// and dnorm_weight, and for a gate that rows share two partial rows of dgate
// (the gate rows that the span's ends may cut).
inline size_t branch_workspace_floats(int groups, int64_t cols, bool shared_gate) {
  return groups == 1 ? 0 : (size_t)groups * (size_t)cols * (shared_gate ? 4 : 2);
}
cudaError_t branch_backward_resident_groups(int dtype, int W, const FusedShape& sh, int num_sms, int* groups);
cudaError_t launch_branch_backward(int dtype, int W, const RankPtrs& dy, const BranchArgs& br, const BranchGradArgs& g,
                                   const void* weight, float eps, unsigned int* err, int64_t rows, int64_t cols,
                                   int vec_per_row, const FusedShape& sh, const WaitHook& hook, cudaStream_t s);
// Backward, many rows (branch_backward_tma.cu, branch_backward_tma.cuh): a launch, or
// several of a part of the rows each.
void branch_backward_tma_shape(int64_t rows, int vec_per_row, int num_sms, BranchTeams* out);
cudaError_t branch_backward_tma_prepare(int dtype, BranchTeams* sh);
cudaError_t launch_branch_backward_tma(int dtype, int W, const RankPtrs& dy, const BranchArgs& br, const BranchGradArgs& g,
                                       const void* weight, float eps, unsigned int* err, int64_t rows, int64_t cols,
                                       int vec_per_row, const BranchTeams& sh, const WaitHook& hook, cudaStream_t s);
// The sum of the groups' partials, behind either backward kernel; add, add_gate: to what
// dweight and dnorm_weight, or dgate, hold.
cudaError_t launch_branch_sums(const BranchArgs& br, const BranchGradArgs& g, int dtype, int groups, int64_t rows,
                               int64_t cols, bool add, bool add_gate, cudaStream_t s);

}  // namespace car
