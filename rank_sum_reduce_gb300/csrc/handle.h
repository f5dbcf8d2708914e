// handle.h -- the handle behind car_ctx, and what every call on one checks
// (internal; defined in api.cu).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "../../include/car.h"
#include "branch.h"
#include "car_device.cuh"
#include "car_launch.h"

struct car_ctx {
  int W;
  int64_t M, N;
  int dtype;
  int es;
  int64_t D;            // bytes per rank
  int64_t nvec;         // 16-byte vectors per rank
  int vec_per_row;      // 16-byte vectors per row
  int device;
  int num_sms;
  int reduce_grid;
  int two_shot_grid;
  bool fused_ok;        // row short enough for the fused kernel
  car::FusedShape fused_auto;
  car::FusedShape fused;
  bool tma_ok;          // row fits the shared-memory ring of the pipelined kernel
  car::FusedTmaShape tma_auto;
  car::FusedTmaShape tma;
  // The 8-bit output and the backward: found when first asked for, so that a
  // handle that does without them pays nothing for them (see prepare_quant).
  std::mutex shapes;
  std::atomic<bool> quant_ready{false}, backward_ready{false};
  car::FusedShape quant;     // row kernel with an 8-bit output: the automatic shape, its own resident count
  car::TeamShape quant_tma;
  bool quant_pipeline;       // the 8-bit output runs the pipeline kernel
  car::FusedShape backward;  // backward of the fused op: row kernel
  car::TeamShape backward_tma;
  bool backward_pipeline;
  int backward_groups;       // CTAs (or clusters) with a partial weight gradient each
  // The branch calls and dropout, the same way (branch_api.cu).
  std::atomic<bool> branch_ready{false}, branch_backward_ready{false}, dropout_ready{false};
  car::FusedShape branch, branch_backward;   // row kernels
  car::BranchTeams branch_tma, branch_backward_tma;
  bool branch_pipeline, branch_backward_pipeline;
  int dropout_grid;
  int fused_kernel_auto;  // CAR_FUSED_ROWS or CAR_FUSED_PIPELINE
  int fused_kernel;
  unsigned int* d_err;  // bounded-wait failures reported by kernels (device)
  car::WaitHook hook;   // the fused row kernel's partial-exchange wait limit and test delay
  int64_t ll128_lines;
  int ll128_encode_grid[2], ll128_decode_grid[2];  // [1]: the misaligned instances
  int64_t ll_lines;
  int ll_encode_grid, ll_decode_grid;
  bool lamport_ok;              // bf16 and a row the Lamport receive kernel takes
  car::FusedShape lamport;
  int lamport_grid;             // fill / push kernels
  car::StaleLog* log[3];       // [0] LL128, [1] LL, [2] Lamport (device)
  cudaStream_t last_stream[3];
  bool decoded[3];
  uint64_t calls[3];           // decode calls so far; call c counts in log->n[c & 1]
  int last_slot[3];
};

namespace car {

// Keeps the error's text for car_last_error; CAR_ERR_CUDA.
car_status cuda_fail(cudaError_t e, const char* where);
bool live(const car_ctx* h);
car_status check_handle(const car_ctx* h);
car_status check_table(const car_ctx* h, const void* const* ptrs, RankPtrs* out);
car_status check_dev(const void* p);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int round_up32(int64_t v) { return (int)((v + 31) / 32 * 32); }

// The handle's device as the current one while shapes are found for it.
struct OnDevice {
  int before = -1;
  bool moved = false;
  cudaError_t status;
  explicit OnDevice(int device) {
    status = cudaGetDevice(&before);
    if (status != cudaSuccess || before == device) return;
    status = cudaSetDevice(device);
    moved = true;
  }
  ~OnDevice() {
    if (moved) cudaSetDevice(before);
  }
};

// Automatic shape of a row-split kernel (the fused row kernel and the Lamport
// receive), given which (W, vectors per thread) instances are compiled and
// their thread limits.  A row is split over a cluster of c = 8 or 4 CTAs (the
// largest that qualifies) when
//  * each CTA keeps at least 128 16-byte vectors of the row,
//  * the c * M CTAs stay within 7/8 of the SMs (one wave of clusters), and
//  * there are at most 16 rows, or each row brings at least 48 KB of inputs;
// otherwise one CTA takes a row, with the fewest vectors per thread that the
// compiled instances allow.  A row too wide for one CTA's threads takes the
// smallest cluster whose CTAs cover it.
//
// Measured on GB300 for the fused row kernel, with the partials pushed by
// st.async (graph replay over cold inputs, bf16; us per call, rule's choice
// against one CTA per row): W = 8, N = 8192: M = 1 1.97 / 3.01, M = 32
// (c = 4) 2.70 / 3.19; W = 8, N = 4096, M = 1 (c = 4) 1.90 / 2.19; W = 2,
// N = 8192, M = 32 (c = 4) 2.26 / 2.45.  Where the rule keeps one CTA per row
// it was as fast or faster: W = 4, N = 4096, M = 32: 2.09 against 2.20 with
// four CTAs; W = 2, N = 2048, M = 1: 1.48 against 1.64 with two.
//
// With prefer_half_ctas, a shape that would need a 1024-thread CTA with one
// vector per thread takes 512 threads with two vectors instead when that
// instance exists.  Measured for the fused row kernel (one CTA per row, bf16,
// N = 8192, graph replay over cold inputs, us per call, 512 x 2 against
// 1024 x 1): W = 4, M = 128 3.51 / 3.61; W = 4, M = 64 2.74 / 2.85; W = 2,
// M = 128 2.89 / 3.05.
template <class HasVariant, class MaxThreads>
FusedShape row_split_shape(int W, int64_t M, int V, int num_sms, HasVariant has_variant, MaxThreads max_threads,
                           bool prefer_half_ctas) {
  auto fit = [&](int c, FusedShape* out) {
    const int chunk = (V + c - 1) / c;
    for (int vpt = 1; vpt <= 2; vpt++) {
      if (!has_variant(W, vpt)) continue;
      const int t = std::max(32, round_up32((chunk + vpt - 1) / vpt));
      if (vpt == 1 && prefer_half_ctas && t > 512 && has_variant(W, 2) &&
          std::max(32, round_up32((chunk + 1) / 2)) <= max_threads(W, 2))
        continue;
      if (t <= max_threads(W, vpt)) {
        *out = FusedShape{c, t, vpt, 1};
        return true;
      }
    }
    return false;
  };
  FusedShape sh;
  const int64_t row_in = (int64_t)(W + 1) * V * 16;
  for (int c = 8; c >= 4; c /= 2) {
    if (V / c < 128 || (int64_t)c * M > num_sms - num_sms / 8 || (M > 16 && row_in < 48 * 1024)) continue;
    if (fit(c, &sh)) return sh;
  }
  for (int c = 1; c <= 8; c *= 2)
    if (fit(c, &sh)) return sh;
  return FusedShape{8, std::max(32, round_up32((V + 7) / 8)), 1, 1};  // rows past CAR_MAX_ROW_BYTES only
}

}  // namespace car
