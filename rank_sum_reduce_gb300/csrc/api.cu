// api.cu -- the C ABI of libcar (include/car.h): argument checks, handles,
// launch shapes, stale-line reports.  Every operation runs in the kernels of
// reduce.cu, fused.cu, fused_tma.cu, fused_quant.cu, quant_tma.cu,
// norm_backward.cu, norm_backward_tma.cu, ll128.cu, ll.cu and lamport.cu;
// nothing here computes results.  (Gradient handles: grads_api.cu.)
//
// Argument rules follow the problem statement on the pages:
//   P1 "SGLang Custom AllReduce v1 线程模型和工作原理细节", section
//      "一次调用给 kernel 什么：参数与 grid" (message bytes a multiple of 16;
//      same size and type on every rank) and "线程模型：16 字节一个单位"
//      (16-byte aligned packed units);
//   P3 "0-custom-all-reduce", "调用" (up to 16 ranks) and "5. 写回"
//      (output may alias the input);
//   P2 "NCCL 专家课程 14：Simple、LL、LL128 的线格式、同步与真实性能边界",
//      "LL 如何发布和等待 flag" (waits are bounded: the page's loops check for
//      abort; here a poll count bounds them).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <unordered_set>

#include "../../include/car.h"
#include "car_device.cuh"
#include "car_launch.h"
#include "quant.cuh"

static_assert(car::kStaleCap == CAR_STALE_LIST_MAX, "stale list capacity mismatch");
static_assert((int)car::kScaleRow == CAR_SCALE_ROW && (int)car::kScaleGroup128 == CAR_SCALE_GROUP128 &&
                  (int)car::kScaleMx32 == CAR_SCALE_MX32 && (int)car::kScaleStatic == CAR_SCALE_STATIC,
              "scale kinds mismatch");

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

namespace {

std::mutex g_mu;
std::unordered_set<const car_ctx*> g_live;
thread_local char g_err[256] = "";

car_status cuda_fail(cudaError_t e, const char* where) {
  snprintf(g_err, sizeof(g_err), "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
  return CAR_ERR_CUDA;
}

bool live(const car_ctx* h) {
  if (!h) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  return g_live.count(h) != 0;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks shared by every call on a handle: the handle is live and its device
// is the current one.
car_status check_handle(const car_ctx* h) {
  if (!live(h)) return CAR_ERR_HANDLE;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != h->device) {
    snprintf(g_err, sizeof(g_err), "handle belongs to device %d, current device is %d", h->device, dev);
    return CAR_ERR_ARG;
  }
  return CAR_OK;
}

car_status check_table(const car_ctx* h, const void* const* ptrs, car::RankPtrs* out) {
  if (!ptrs) return CAR_ERR_ARG;
  std::memset(out, 0, sizeof(*out));
  for (int r = 0; r < h->W; r++) {
    if (!ptrs[r]) return CAR_ERR_ARG;
    if (!aligned16(ptrs[r])) return CAR_ERR_ALIGN;
    out->p[r] = ptrs[r];
  }
  return CAR_OK;
}

car_status check_dev(const void* p) {
  if (!p) return CAR_ERR_ARG;
  return aligned16(p) ? CAR_OK : CAR_ERR_ALIGN;
}

// Rank data of the LL128 calls needs only element alignment.
car_status check_dev_elem(const void* p, int es) {
  if (!p) return CAR_ERR_ARG;
  return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)es) == 0 ? CAR_OK : CAR_ERR_ALIGN;
}

int clamp_grid(int64_t needed, int per_sm, int num_sms) {
  const int64_t cap = (int64_t)std::max(per_sm, 1) * num_sms;
  return (int)std::max<int64_t>(1, std::min(needed, cap));
}

int round_up32(int64_t v) { return (int)((v + 31) / 32 * 32); }

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
car::FusedShape row_split_shape(int W, int64_t M, int V, int num_sms, HasVariant has_variant,
                                MaxThreads max_threads, bool prefer_half_ctas) {
  auto fit = [&](int c, car::FusedShape* out) {
    const int chunk = (V + c - 1) / c;
    for (int vpt = 1; vpt <= 2; vpt++) {
      if (!has_variant(W, vpt)) continue;
      const int t = std::max(32, round_up32((chunk + vpt - 1) / vpt));
      if (vpt == 1 && prefer_half_ctas && t > 512 && has_variant(W, 2) &&
          std::max(32, round_up32((chunk + 1) / 2)) <= max_threads(W, 2))
        continue;
      if (t <= max_threads(W, vpt)) {
        *out = car::FusedShape{c, t, vpt, 1};
        return true;
      }
    }
    return false;
  };
  car::FusedShape sh;
  const int64_t row_in = (int64_t)(W + 1) * V * 16;
  for (int c = 8; c >= 4; c /= 2) {
    if (V / c < 128 || (int64_t)c * M > num_sms - num_sms / 8 || (M > 16 && row_in < 48 * 1024)) continue;
    if (fit(c, &sh)) return sh;
  }
  for (int c = 1; c <= 8; c *= 2)
    if (fit(c, &sh)) return sh;
  return car::FusedShape{8, std::max(32, round_up32((V + 7) / 8)), 1, 1};  // rows past CAR_MAX_ROW_BYTES only
}

car::FusedShape auto_fused_shape(int W, int64_t M, int V, int num_sms) {
  return row_split_shape(W, M, V, num_sms, car::fused_has_variant, car::fused_max_threads, true);
}

bool shape_valid(int W, int V, const car::FusedShape& sh) {
  if (sh.cluster != 1 && sh.cluster != 2 && sh.cluster != 4 && sh.cluster != 8) return false;
  if (!car::fused_has_variant(W, sh.vpt)) return false;
  if (sh.threads < 32 || sh.threads % 32 != 0 || sh.threads > car::fused_max_threads(W, sh.vpt)) return false;
  const int64_t chunk = (V + sh.cluster - 1) / sh.cluster;
  return (int64_t)sh.threads * sh.vpt >= chunk;
}

// The pipelined kernel is faster once there are more rows than SMs and a row
// slice (N * s bytes, one bulk copy per rank) is larger than 8 KB.  Measured on
// GB300 against the row kernel (both fetching their first row into L2 before
// the PDL wait), N = 8192 bf16: at M = 152, W = 8 5.8 (rows) against 6.5 us
// (pipeline), W = 2 3.3 against 3.8; at M = 184, W = 8 8.2 against 7.5, W = 2
// 5.3 against 4.5; at M = 456, W = 8 15.4 against 13.4; at M = 1024 28.2
// (pipeline) against 32.3; 12 KB slices, W = 8, M = 1024, N = 6144 bf16: 21.7
// against 25.9.  With 8 KB
// slices and smaller the persistent CTA finishes its rows one after another
// (each behind the row statistic's barriers), and the row kernel, many CTAs
// per SM, keeps more rows in flight: W = 4,
// M = 1024, N = 4096 bf16 11.8 (rows) against 13.0 us; W = 8, M = 4096,
// N = 2048 29.2 against 46.1; W = 2, M = 4096, N = 1024 8.9 against 27.4; a
// deeper ring with several issuing lanes did not close the gap.
int auto_fused_kernel(const car_ctx* h) {
  const bool big_slices = h->N * (int64_t)h->es > 8192;
  return (h->tma_ok && big_slices && h->M > (int64_t)h->num_sms) ? CAR_FUSED_PIPELINE : CAR_FUSED_ROWS;
}

// Row-kernel shape for the Lamport receive step: the same rules as the fused
// row kernel, within the Lamport kernel's compiled instances.
car::FusedShape auto_lamport_shape(int W, int64_t M, int V, int num_sms) {
  return row_split_shape(W, M, V, num_sms, car::lamport_has_variant, car::lamport_max_threads, false);
}

// The rank counts that the row kernels of the 8-bit output and of the backward
// are compiled for; others run an instance that holds registers for 16 ranks.
bool rows_compiled(int W) { return W <= 2 || W == 4 || W == 8 || W == 16; }

// When the 8-bit output's pipeline kernel is faster than its row kernel.
// Measured on GB300 (graph replay over cold inputs, bf16 unless noted, scales
// of 128 columns, us per call, pipeline / rows).
//  * One or two ranks: once a tile keeps nearly every SM busy.  One scale per
//    row, W = 1, N = 4096, M = 304 3.4 / 2.5, M = 608 3.6 / 4.2, M = 1000 7.0 /
//    7.7; N = 5000, M = 304 3.9 / 3.6, M = 608 6.1 / 6.7; N = 2800, M = 1000 5.4
//    / 6.6.  Eight and more rows a tile only where the last tiles fill the SMs
//    too: W = 2, N = 2048, M = 1000 4.0 / 4.4, M = 1500 7.0 / 6.5, M = 3000 10.2
//    / 11.2.  Rows of at most 128 vectors (a warp each, no barrier) from half a
//    tile per SM: N = 1024, M = 1500, W = 1 3.3 / 4.4, W = 2 3.7 / 4.6.
//  * Three vectors per thread (rows that two do not fit, and which the row
//    kernel's threads do not fit either) from one and a half tiles per SM: N =
//    2800, M = 608, W = 4 4.9 / 4.8, W = 8 8.6 / 6.8, M = 1000 8.4 / 8.9 and 11.5
//    / 12.6; N = 5000, M = 304 4.5 / 4.9 and 9.1 / 6.9, M = 608 9.5 / 10.0 and
//    13.4 / 14.9, M = 1500 17.3 / 23.6 and 25.7 / 32.5.
//  * Four ranks: N = 8192, M = 304 7.5 / 6.8, M = 456 10.0 / 10.7; N = 4096, M =
//    912 9.8 / 9.4, M = 1216 12.2 / 12.0, M = 2000 17.8 / 18.9; N = 1024, M =
//    2432 7.3 / 6.9, M = 3648 9.7 / 11.3.
//    Where the row kernel's threads fit a row much better it stays ahead: N =
//    1248 (156 vectors; 5 teams of 96 threads), M = 5950 19.4 / 18.3.
//  * Eight ranks: N = 8192, M = 304 10.6 / 10.8, M = 456 14.2 / 15.2; rows of 4
//    and 8 KB stay with the row kernel (N = 4096, M = 1216 17.2 / 16.2, M = 6000
//    78.9 / 76.9), shorter ones do not (N = 1024, M = 3648 13.8 / 14.1).
//  * Sixteen: N = 2192, M = 2000 28 / 37; N = 4096, M = 1000 26.0 / 26.3; N =
//    2776, M = 531 11.2 / 10.9.
//  * Rows of more than 1024 vectors (N = 16384, one scale per row): W = 4, M =
//    2000 63.9 / 78.5; W = 1, M = 4000 76 / 108; W = 8, M = 300 18.7 / 20.3.
//    More than 2048, where the row kernel splits rows and waits for the parts:
//    fp32, N = 9000, M = 100, W = 1 4.0 / 5.6, W = 4 5.3 / 6.9, W = 8 9.0 / 9.0, M
//    = 600 15.8 / 30, 25.6 / 39 and 36 / 54; with seven vectors per thread N =
//    12800, M = 100, W = 1 5.0 / 6.0, W = 4 9.1 / 8.0, M = 304 18.9 / 22.9; bf16,
//    N = 27000, M = 100 7.8 / 7.0, M = 304 16.8 / 20.6.  With eight (3600, 3900
//    and 4096 vectors, fp32 and bf16, M from 152 to 2432) the quotient is 0.60
//    to 0.85 for W = 1, 0.64 to 0.87 for 2, 0.75 to 1.00 for 4, 0.83 to 1.11
//    (mean 0.97) for 8 and 0.80 to 0.96 for 16; at M = 100 0.92 to 1.26.
//  * Rank counts that the row kernel is not compiled for: W = 6, N = 4096, M =
//    4096 43 / 65; W = 3, N = 10000, M = 2000 40 / 118, N = 8192, M = 200 5.3 /
//    7.1, N = 2048, M = 200 3.0 / 2.4.
bool quant_pipeline_pays(const car_ctx* h, const car::TeamShape& sh) {
  const int64_t tiles = (h->M + sh.teams - 1) / sh.teams, sms = h->num_sms;
  if (!rows_compiled(h->W)) return 2 * tiles >= sms;
  if (sh.vpt > 4) return sh.vpt <= 6 ? 2 * tiles >= sms : tiles >= sms;
  if (h->vec_per_row > 1024) return 2 * tiles >= 3 * sms;
  if (h->W <= 2) {
    if (sh.teams >= 16) return 2 * tiles >= sms;
    return 5 * tiles >= 4 * sms && (sh.teams < 8 || tiles <= sms || tiles >= 2 * sms);
  }
  if (sh.vpt == 3) return 2 * tiles >= 3 * sms;
  if (h->vec_per_row > 512) return 2 * h->M >= 5 * sms;
  if (sh.use < 0.8) return false;
  if (h->W == 4) return tiles >= (sh.teams >= 8 ? 3 : 4) * sms;
  if (h->W == 8) return sh.teams >= 8 && tiles >= 3 * sms;
  return 2 * tiles >= 5 * sms;
}

// When the backward's pipeline kernel is faster than its row kernel.  Measured
// as above, with a weight gradient, pipeline / rows.
//  * One or two ranks, rows short enough for several teams: W = 1, N = 1024, M
//    = 640 5.6 / 6.2, M = 3648 10.3 / 11.0; N = 4096, M = 152 5.7 / 5.9, M = 912
//    10.2 / 10.9, M = 16389 82 / 104.  Three vectors per thread from five rows
//    per SM: N = 6144, M = 456 10.2 / 9.1, M = 1200 15.4 / 16.5; W = 2, N = 5000,
//    M = 608 11.3 / 10.7, M = 1500 18.2 / 20.2; fp32, N = 3000, M = 608 9.6 /
//    10.5.  With one team the row kernel, which holds two rows' loads in
//    registers there, keeps up for longer in 16 bits (N = 8192, M = 456 11.5 /
//    10.2, M = 912 15.6 / 15.7, M = 6000 64.9 / 65.4) than in fp32 (N = 4096, M
//    = 1000 14.3 / 16.6).
//  * More ranks pay the ring's start and its issuing threads until a CTA has two
//    tiles or three: N = 4096, W = 8, M = 400 12.2 / 10.7, M = 608 13.5 / 13.7,
//    M = 912 16.8 / 18.3; W = 4, M = 456 10.0 / 9.5, M = 608 10.6 / 11.3; N =
//    8192, W = 4, M = 304 11.4 / 10.7, M = 456 13.6 / 14.1, W = 8, M = 200 13.1 /
//    13.2, M = 304 14.3 / 16.6; W = 16, N = 2048, M = 1200 19.3 / 18.9.
//  * Rows of more than 1024 vectors, three per thread: W = 1, N = 11072, M = 304
//    12.1 / 10.8, M = 608 16.1 / 17.6, M = 1737 31 / 42; N = 10488, W = 4, M = 200
//    13.3 / 11.1, M = 304 13.9 / 14.6, M = 608 20 / 26.  Four: fp32 as three.  In
//    16 bits the accumulators leave little room, and from the 17th warp on one
//    of the SM's four schedulers has five: W = 1, M = 2432, 1740 vectors (16
//    warps) 61 / 63, 1800 vectors 72 / 63; W = 4 88 / 93 and 108 / 92.  Up to 16
//    warps (1540, 1640 and 1740 vectors) the quotient is 1.01 to 1.13 for W = 1
//    and 2 below M = 2432, 0.94 to 1.07 for W = 4 below M = 1216 and 0.91 to 1.00
//    from there, 0.80 to 0.97 for W = 8 and 0.85 to 0.95 for W = 16 from M = 152.
//    More, in fp32: N = 9000, M = 100, W = 2 6.9 / 7.6, W = 8 11.4 / 11.6, M =
//    600, W = 2 25.8 / 36.0, W = 8 44 / 53; N = 11000, M = 3000, W = 1 103 / 152,
//    W = 8 228 / 264.  Seven vectors per thread (3150, 3300 and 3400 vectors, M
//    from 152 to 2432): 0.80 to 0.91 for W = 1, 0.87 to 0.99 for 2, 0.91 to 1.06
//    for 4, 0.89 to 0.94 for 8, 0.68 to 1.01 for 16.  Eight (3600, 3900 and 4096,
//    M = 1216 and 2432): 0.90 to 1.02 for W = 1, whose tile fits the ring whole,
//    0.83 to 0.95 for W = 16, whose row kernel takes one vector per thread, 0.96
//    to 1.15 for the others; below M = 1216 0.90 to 1.33.
//  * Rank counts that the row kernel is not compiled for: W = 3, N = 10000, M =
//    2000 56 / 127; W = 6, N = 16384 fp32, M = 500 62 / 80; W = 3, N = 8192, M =
//    200 9.7 / 10.3.
bool backward_pipeline_pays(const car_ctx* h, const car::TeamShape& sh) {
  const int64_t tiles = (h->M + sh.teams - 1) / sh.teams, sms = h->num_sms;
  const int V = h->vec_per_row;
  const bool fp32 = h->dtype == CAR_FP32;
  if (!rows_compiled(h->W)) return 2 * tiles >= sms;
  if (sh.vpt == 8) return tiles >= 8 * sms && (sh.slots >= h->W + 2 || !car::backward_has_variant(h->W, 2));
  if (sh.vpt == 7) return tiles >= sms;
  if (sh.vpt > 4) return 3 * tiles >= 2 * sms;
  if (V > 1536 && fp32) return tiles >= 2 * sms;
  if (V > 1536) return sh.team_threads + 32 * sh.producers <= 512 && h->W >= 4 && tiles >= (h->W < 8 ? 6 : 1) * sms;
  if (V > 1024) return tiles >= (h->W <= 2 ? 3 : 2) * sms;
  if (h->W <= 2 && sh.teams == 1) return tiles >= (fp32 ? 4 : 6) * sms;
  if (h->W <= 2) return sh.vpt == 2 ? 2 * tiles >= sms : h->M >= 5 * sms;
  if (sh.teams == 1) return tiles >= (h->W < 8 ? 3 : 2) * sms;
  return 2 * tiles >= (h->W > 8 ? 5 : 4) * sms;
}

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

car_status prepare_quant(car_ctx* h) {
  if (h->quant_ready.load(std::memory_order_acquire)) return CAR_OK;
  std::lock_guard<std::mutex> lk(h->shapes);
  if (h->quant_ready.load(std::memory_order_relaxed)) return CAR_OK;
  const OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_fail(on.status, "device of the handle");
  int groups = 0;
  h->quant = auto_fused_shape(h->W, h->M, h->vec_per_row, h->num_sms);
  cudaError_t e = car::fused_quant_resident_groups(h->dtype, h->W, h->quant, h->num_sms, &groups);
  if (e != cudaSuccess) return cuda_fail(e, "8-bit output occupancy");
  h->quant.groups = (int)std::max<int64_t>(1, std::min<int64_t>(h->M, std::max(groups, 1)));
  h->quant_pipeline = car::quant_tma_shape(h->M, h->vec_per_row, h->num_sms, h->W, &h->quant_tma) &&
                      quant_pipeline_pays(h, h->quant_tma);
  if (h->quant_pipeline && (e = car::quant_tma_prepare(h->dtype, h->quant_tma)) != cudaSuccess)
    return cuda_fail(e, "8-bit output pipeline smem");
  h->quant_ready.store(true, std::memory_order_release);
  return CAR_OK;
}

car_status prepare_backward(car_ctx* h) {
  if (h->backward_ready.load(std::memory_order_acquire)) return CAR_OK;
  std::lock_guard<std::mutex> lk(h->shapes);
  if (h->backward_ready.load(std::memory_order_relaxed)) return CAR_OK;
  const OnDevice on(h->device);
  if (on.status != cudaSuccess) return cuda_fail(on.status, "device of the handle");
  int groups = 0;
  h->backward = row_split_shape(h->W, h->M, h->vec_per_row, h->num_sms, car::backward_has_variant, car::backward_max_threads, false);
  cudaError_t e = car::backward_resident_groups(h->dtype, h->W, h->backward, h->num_sms, &groups);
  if (e != cudaSuccess) return cuda_fail(e, "backward occupancy");
  const int64_t teams = car::backward_teams(h->backward);
  h->backward.groups = (int)std::max<int64_t>(1, std::min<int64_t>((h->M + teams - 1) / teams, std::max(groups, 1)));
  h->backward_pipeline = car::backward_tma_shape(h->dtype, h->M, h->vec_per_row, h->num_sms, h->W, &h->backward_tma) &&
                         backward_pipeline_pays(h, h->backward_tma);
  if (h->backward_pipeline && (e = car::backward_tma_prepare(h->dtype, h->backward_tma)) != cudaSuccess)
    return cuda_fail(e, "backward pipeline smem");
  h->backward_groups = h->backward_pipeline ? h->backward_tma.grid : h->backward.groups;
  h->backward_ready.store(true, std::memory_order_release);
  return CAR_OK;
}

car_status finish_fused_shape(car_ctx* h, car::FusedShape sh) {
  int groups = 0;
  cudaError_t e = car::fused_resident_groups(h->dtype, h->W, sh, h->num_sms, &groups);
  if (e != cudaSuccess) return cuda_fail(e, "fused occupancy");
  sh.groups = (int)std::max<int64_t>(1, std::min<int64_t>(h->M, std::max(groups, 1)));
  h->fused = sh;
  return CAR_OK;
}

// The log slot of the next decode of this kind (its kernel zeroes the other).
int next_log_slot(car_ctx* h, int which) {
  const int slot = (int)(h->calls[which] & 1u);
  h->calls[which]++;
  h->last_slot[which] = slot;
  return slot;
}

car_status decode_common(car_ctx* h, int which, const void* const* wires, int max_polls,
                         void* ar_out, cudaStream_t s, car::RankPtrs* tbl) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (max_polls < 1) return CAR_ERR_ARG;
  if ((st = check_table(h, wires, tbl)) != CAR_OK) return st;
  // LL128 output may sit at any element offset; LL output stays 16-byte aligned
  if ((st = which == 0 ? check_dev_elem(ar_out, h->es) : check_dev(ar_out)) != CAR_OK) return st;
  h->last_stream[which] = s;
  h->decoded[which] = true;
  return CAR_OK;
}

car_status report_common(car_ctx* h, int which, car_stale_report* out) {
  if (!live(h)) return CAR_ERR_HANDLE;
  if (!out || (out->cap > 0 && !out->entries)) return CAR_ERR_ARG;
  out->n_stale = 0;
  out->n_listed = 0;
  if (!h->decoded[which]) return CAR_OK;
  cudaError_t e = cudaStreamSynchronize(h->last_stream[which]);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  unsigned long long n = 0;
  e = cudaMemcpy(&n, &h->log[which]->n[h->last_slot[which]], sizeof(n), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "read stale count");
  const uint64_t listed = std::min<uint64_t>(n, std::min<uint64_t>(out->cap, car::kStaleCap));
  if (listed) {
    e = cudaMemcpy(out->entries, h->log[which]->entry, listed * 2 * sizeof(uint32_t),
                   cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "read stale list");
  }
  // Clear the count just read.  A decode zeroes only the other slot (for the
  // call after it), so a single decode captured in a CUDA graph would
  // otherwise add every replay's stale lines to the same count.
  if (n) {
    e = cudaMemsetAsync(&h->log[which]->n[h->last_slot[which]], 0, sizeof(n), h->last_stream[which]);
    if (e == cudaSuccess) e = cudaStreamSynchronize(h->last_stream[which]);
    if (e != cudaSuccess) return cuda_fail(e, "clear stale count");
  }
  out->n_stale = n;
  out->n_listed = (uint32_t)listed;
  return n ? CAR_ERR_STALE_FLAG : CAR_OK;
}

}  // namespace

namespace car {
void set_last_error(const char* msg) { snprintf(g_err, sizeof(g_err), "%s", msg); }
}  // namespace car

extern "C" {

const char* car_status_string(car_status s) {
  switch (s) {
    case CAR_OK: return "CAR_OK";
    case CAR_ERR_ARG: return "CAR_ERR_ARG: invalid argument";
    case CAR_ERR_ALIGN: return "CAR_ERR_ALIGN: device pointer not 16-byte aligned";
    case CAR_ERR_SIZE: return "CAR_ERR_SIZE: unsupported size";
    case CAR_ERR_CUDA: return "CAR_ERR_CUDA: CUDA runtime error";
    case CAR_ERR_STALE_FLAG: return "CAR_ERR_STALE_FLAG: stale lines found";
    case CAR_ERR_HANDLE: return "CAR_ERR_HANDLE: invalid handle";
    case CAR_ERR_TIMEOUT: return "CAR_ERR_TIMEOUT: a kernel gave up a bounded wait";
  }
  return "unknown car_status";
}

const char* car_last_error(void) { return g_err; }

car_status car_create(int W, int64_t M, int64_t N, car_dtype dtype, car_ctx** out) {
  if (!out) return CAR_ERR_ARG;
  *out = nullptr;
  g_err[0] = 0;
  if (W < 1 || W > car::kMaxRanks || M < 1 || N < 1) return CAR_ERR_ARG;
  if (dtype != CAR_BF16 && dtype != CAR_FP16 && dtype != CAR_FP32) return CAR_ERR_ARG;
  const int es = dtype == CAR_FP32 ? 4 : 2;
  if (N > (int64_t)INT32_MAX / es || (N * es) % 16 != 0) return CAR_ERR_SIZE;
  // whole message and both wire formats must stay far below int64 range
  if (M > ((int64_t)1 << 56) / (N * es)) return CAR_ERR_SIZE;
  const int64_t D = M * N * es;
  if ((D + 119) / 120 > (int64_t)UINT32_MAX || D / 8 > (int64_t)UINT32_MAX) return CAR_ERR_SIZE;

  car_ctx* h = new (std::nothrow) car_ctx();
  if (!h) return CAR_ERR_ARG;
  h->W = W;
  h->M = M;
  h->N = N;
  h->dtype = (int)dtype;
  h->es = es;
  h->D = D;
  h->nvec = D / 16;
  h->vec_per_row = (int)(N * es / 16);
  h->ll128_lines = (D + 119) / 120;
  h->ll_lines = D / 8;
  h->hook = car::WaitHook{car::kWaitLimitNs, 0, 0, -1};

  auto fail = [&](cudaError_t e, const char* where) {
    for (auto*& p : h->log)
      if (p) cudaFree(p);
    if (h->d_err) cudaFree(h->d_err);
    delete h;
    return cuda_fail(e, where);
  };
  cudaError_t e = cudaGetDevice(&h->device);
  if (e != cudaSuccess) return fail(e, "cudaGetDevice");
  e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) return fail(e, "SM count");

  int per_sm = 0, per_sm2 = 0;
  if ((e = car::reduce_occupancy(h->dtype, W, &per_sm)) != cudaSuccess) return fail(e, "reduce occupancy");
  const int64_t per_cta = (int64_t)car::kReduceThreads * car::reduce_vectors_per_thread(W);
  h->reduce_grid = clamp_grid((h->nvec + per_cta - 1) / per_cta, per_sm, h->num_sms);
  if ((e = car::two_shot_occupancy(h->dtype, W, &per_sm)) != cudaSuccess) return fail(e, "two-shot occupancy");
  h->two_shot_grid = clamp_grid((h->nvec + per_cta - 1) / per_cta, per_sm, h->num_sms);

  const int64_t pairs = (h->ll128_lines + 1) / 2;
  const int64_t warps_needed = (pairs + 1) / 2;
  const int64_t blocks_needed = (warps_needed + car::kWireThreads / 32 - 1) / (car::kWireThreads / 32);
  for (int mis = 0; mis < 2; mis++) {
    if ((e = car::ll128_occupancy(h->dtype, W, mis != 0, h->ll128_lines, &per_sm, &per_sm2)) != cudaSuccess)
      return fail(e, "ll128 occupancy");
    h->ll128_decode_grid[mis] = clamp_grid(blocks_needed, per_sm, h->num_sms);
    h->ll128_encode_grid[mis] = clamp_grid(blocks_needed, per_sm2, h->num_sms);
  }

  if ((e = car::ll_occupancy(h->dtype, W, &per_sm, &per_sm2)) != cudaSuccess) return fail(e, "ll occupancy");
  h->ll_decode_grid = clamp_grid((h->ll_lines + car::kWireThreads - 1) / car::kWireThreads, per_sm, h->num_sms);
  h->ll_encode_grid = clamp_grid((h->nvec + car::kWireThreads - 1) / car::kWireThreads, per_sm2, h->num_sms);

  h->fused_ok = N * es <= (int64_t)CAR_MAX_ROW_BYTES;
  // The pipelined kernel takes whole rows by default: splitting rows over CTA
  // pairs puts a cross-SM exchange on every row's critical path, which
  // measured slower on GB300 than the quantisation it removes.
  h->tma_ok = h->fused_ok && car::fused_tma_shape(M, h->vec_per_row, h->num_sms, 1, W, &h->tma);
  h->tma_auto = h->tma;
  if (h->tma_ok && (e = car::fused_tma_prepare(h->dtype, W, h->tma)) != cudaSuccess) return fail(e, "pipeline smem");
  h->fused_kernel_auto = auto_fused_kernel(h);
  h->fused_kernel = h->fused_kernel_auto;
  if (h->fused_ok) {
    h->fused_auto = auto_fused_shape(W, M, h->vec_per_row, h->num_sms);
    car_status st = finish_fused_shape(h, h->fused_auto);
    if (st != CAR_OK) {
      delete h;
      return st;
    }
    h->fused_auto = h->fused;
  }

  h->lamport_ok = h->fused_ok && dtype == CAR_BF16;
  if (h->lamport_ok) {
    car::FusedShape sh = auto_lamport_shape(W, M, h->vec_per_row, h->num_sms);
    int groups = 0;
    if ((e = car::lamport_resident_groups(W, sh, h->num_sms, &groups)) != cudaSuccess) return fail(e, "lamport occupancy");
    sh.groups = (int)std::max<int64_t>(1, std::min<int64_t>(M, std::max(groups, 1)));
    h->lamport = sh;
    h->lamport_grid = clamp_grid((h->nvec + car::kWireThreads - 1) / car::kWireThreads, 8, h->num_sms);
  }
  e = cudaMalloc(reinterpret_cast<void**>(&h->d_err), 16);
  if (e != cudaSuccess) return fail(e, "cudaMalloc error word");
  e = cudaMemset(h->d_err, 0, 16);
  if (e != cudaSuccess) return fail(e, "cudaMemset error word");
  for (int k = 0; k < 3; k++) {
    e = cudaMalloc(reinterpret_cast<void**>(&h->log[k]), sizeof(car::StaleLog));
    if (e != cudaSuccess) return fail(e, "cudaMalloc stale log");
    e = cudaMemset(h->log[k], 0, sizeof(unsigned long long) * 2);
    if (e != cudaSuccess) return fail(e, "cudaMemset stale log");
  }
  {
    std::lock_guard<std::mutex> lk(g_mu);
    g_live.insert(h);
  }
  *out = h;
  return CAR_OK;
}

car_status car_destroy(car_ctx* h) {
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!h || g_live.erase(h) == 0) return CAR_ERR_HANDLE;
  }
  car_status st = CAR_OK;
  for (auto* p : h->log) {
    cudaError_t e = cudaFree(p);
    if (e != cudaSuccess && st == CAR_OK) st = cuda_fail(e, "cudaFree");
  }
  cudaError_t e = cudaFree(h->d_err);
  if (e != cudaSuccess && st == CAR_OK) st = cuda_fail(e, "cudaFree");
  delete h;
  return st;
}

car_status car_tune_fused(car_ctx* h, int kernel, int cluster, int threads, int vpt) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (!h->fused_ok) return CAR_ERR_SIZE;
  if (kernel == CAR_FUSED_AUTO) {
    if (cluster || threads || vpt) return CAR_ERR_ARG;
    h->fused_kernel = h->fused_kernel_auto;
    h->tma = h->tma_auto;
    return finish_fused_shape(h, h->fused_auto);
  }
  if (kernel == CAR_FUSED_PIPELINE) {
    if (threads || vpt || (cluster != 0 && cluster != 1 && cluster != 2)) return CAR_ERR_ARG;
    if (!h->tma_ok) return CAR_ERR_SIZE;
    car::FusedTmaShape t;
    if (!car::fused_tma_shape(h->M, h->vec_per_row, h->num_sms, cluster ? cluster : 1, h->W, &t)) return CAR_ERR_SIZE;
    cudaError_t e = car::fused_tma_prepare(h->dtype, h->W, t);
    if (e != cudaSuccess) return cuda_fail(e, "pipeline smem");
    h->tma = t;
    h->fused_kernel = CAR_FUSED_PIPELINE;
    return CAR_OK;
  }
  if (kernel != CAR_FUSED_ROWS) return CAR_ERR_ARG;
  car::FusedShape sh = h->fused_auto;
  if (cluster) sh.cluster = cluster;
  if (threads) sh.threads = threads;
  if (vpt) sh.vpt = vpt;
  if (sh.cluster != 1 && sh.cluster != 2 && sh.cluster != 4 && sh.cluster != 8) return CAR_ERR_ARG;
  if (!car::fused_has_variant(h->W, sh.vpt)) return CAR_ERR_ARG;
  if (sh.threads < 32 || sh.threads % 32 || sh.threads > car::fused_max_threads(h->W, sh.vpt)) return CAR_ERR_ARG;
  if (!shape_valid(h->W, h->vec_per_row, sh)) return CAR_ERR_SIZE;
  st = finish_fused_shape(h, sh);
  if (st == CAR_OK) h->fused_kernel = CAR_FUSED_ROWS;
  return st;
}

car_status car_test_delay_partial(car_ctx* h, uint64_t wait_limit_ns, int cta, int64_t row, uint64_t delay_ns) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (cta < 0) {
    if (wait_limit_ns || row || delay_ns) return CAR_ERR_ARG;
    h->hook = car::WaitHook{car::kWaitLimitNs, 0, 0, -1};
    return CAR_OK;
  }
  if (cta > 7 || row < 0 || row >= h->M || wait_limit_ns < 1000 || wait_limit_ns > car::kWaitLimitNs ||
      delay_ns > CAR_TEST_MAX_DELAY_NS)
    return CAR_ERR_ARG;
  h->hook = car::WaitHook{wait_limit_ns, delay_ns, row, cta};
  return CAR_OK;
}

car_status car_sync(car_ctx* h, void* stream) {
  if (!live(h)) return CAR_ERR_HANDLE;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  unsigned int err = 0;
  e = cudaMemcpy(&err, h->d_err, sizeof(err), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "read error word");
  if (!err) return CAR_OK;
  e = cudaMemset(h->d_err, 0, sizeof(err));
  if (e != cudaSuccess) return cuda_fail(e, "clear error word");
  snprintf(g_err, sizeof(g_err), "a kernel gave up a bounded wait (code %u)", err);
  return CAR_ERR_TIMEOUT;
}

car_status car_reduce(car_ctx* h, const void* const* inputs, void* ar_out, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  car::RankPtrs tbl;
  if ((st = check_table(h, inputs, &tbl)) != CAR_OK) return st;
  if ((st = check_dev(ar_out)) != CAR_OK) return st;
  cudaError_t e = car::launch_reduce(h->dtype, h->W, tbl, ar_out, h->nvec, h->reduce_grid,
                                     static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "rank_sum_reduce launch");
}

car_status car_reduce_two_shot(car_ctx* h, const void* const* inputs, void* ar_out, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  car::RankPtrs tbl;
  if ((st = check_table(h, inputs, &tbl)) != CAR_OK) return st;
  if ((st = check_dev(ar_out)) != CAR_OK) return st;
  cudaError_t e = car::launch_two_shot(h->dtype, h->W, tbl, ar_out, h->nvec, h->two_shot_grid,
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "rank_sum_two_shot launch");
}

car_status car_reduce_residual_rmsnorm(car_ctx* h, const void* const* inputs, const void* residual,
                                       const void* weight, float eps, void* residual_out,
                                       void* norm_out, void* ar_out, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (!std::isfinite(eps) || eps < 0.f) return CAR_ERR_ARG;
  car::RankPtrs tbl;
  if ((st = check_table(h, inputs, &tbl)) != CAR_OK) return st;
  if ((st = check_dev(residual)) != CAR_OK) return st;
  if ((st = check_dev(weight)) != CAR_OK) return st;
  if ((st = check_dev(residual_out)) != CAR_OK) return st;
  if ((st = check_dev(norm_out)) != CAR_OK) return st;
  if (ar_out && !aligned16(ar_out)) return CAR_ERR_ALIGN;
  if (!h->fused_ok) return CAR_ERR_SIZE;
  cudaError_t e;
  if (h->fused_kernel == CAR_FUSED_PIPELINE)
    e = car::launch_fused_tma(h->dtype, h->W, tbl, residual, weight, eps, residual_out, norm_out, ar_out,
                              h->d_err, h->M, h->N, h->vec_per_row, h->tma, static_cast<cudaStream_t>(stream));
  else
    e = car::launch_fused(h->dtype, h->W, tbl, residual, weight, eps, residual_out, norm_out, ar_out, h->d_err,
                          h->M, h->N, h->vec_per_row, h->fused, h->hook, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "reduce_residual_rmsnorm launch");
}

static int scale_groups(const car_ctx* h, int kind) {
  return kind == CAR_SCALE_GROUP128 ? (int)((h->N + 127) / 128) : kind == CAR_SCALE_MX32 ? (int)((h->N + 31) / 32) : 1;
}

size_t car_quant_scale_bytes(car_ctx* h, car_scale_kind kind) {
  if (!live(h)) return 0;
  switch (kind) {
    case CAR_SCALE_ROW:
    case CAR_SCALE_GROUP128: return (size_t)h->M * (size_t)scale_groups(h, kind) * 4;
    case CAR_SCALE_MX32: return (size_t)h->M * (size_t)scale_groups(h, kind);
    case CAR_SCALE_STATIC: return 4;
  }
  return 0;
}

car_status car_reduce_residual_rmsnorm_quant(car_ctx* h, const void* const* inputs, const void* residual,
                                             const void* weight, float eps, car_scale_kind kind, void* residual_out,
                                             void* q_out, void* scales, void* norm_out, void* ar_out, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (!std::isfinite(eps) || eps < 0.f) return CAR_ERR_ARG;
  if (kind != CAR_SCALE_ROW && kind != CAR_SCALE_GROUP128 && kind != CAR_SCALE_MX32 && kind != CAR_SCALE_STATIC)
    return CAR_ERR_ARG;
  car::RankPtrs tbl;
  if ((st = check_table(h, inputs, &tbl)) != CAR_OK) return st;
  if ((st = check_dev(residual)) != CAR_OK) return st;
  if ((st = check_dev(weight)) != CAR_OK) return st;
  if ((st = check_dev(residual_out)) != CAR_OK) return st;
  if ((st = check_dev(q_out)) != CAR_OK) return st;
  if ((st = check_dev_elem(scales, kind == CAR_SCALE_MX32 ? 1 : 4)) != CAR_OK) return st;
  if ((norm_out && !aligned16(norm_out)) || (ar_out && !aligned16(ar_out))) return CAR_ERR_ALIGN;
  if (!h->fused_ok) return CAR_ERR_SIZE;
  if ((st = prepare_quant(h)) != CAR_OK) return st;
  car::QuantOut out;
  out.q = static_cast<uint8_t*>(q_out);
  out.scales = scales;
  out.kind = (int)kind;
  out.groups = scale_groups(h, kind);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (h->quant_pipeline)
    e = car::launch_quant_tma(h->dtype, h->W, tbl, residual, weight, eps, residual_out, out, norm_out, ar_out, h->d_err,
                              h->M, h->N, h->vec_per_row, h->quant_tma, s);
  else
    e = car::launch_fused_quant(h->dtype, h->W, tbl, residual, weight, eps, residual_out, out, norm_out, ar_out, h->d_err,
                                h->M, h->N, h->vec_per_row, h->quant, h->hook, s);
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "reduce_residual_rmsnorm_quant launch");
}

size_t car_backward_workspace_bytes(car_ctx* h) {
  if (!live(h) || !h->fused_ok || prepare_backward(h) != CAR_OK || h->backward_groups == 1) return 0;
  return (size_t)h->backward_groups * (size_t)h->N * sizeof(float);
}

car_status car_reduce_residual_rmsnorm_backward(car_ctx* h, const void* const* dnorm, const void* residual_out,
                                                const void* weight, float eps, const void* dresidual_out, void* dx,
                                                void* dweight, void* workspace, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (!std::isfinite(eps) || eps < 0.f) return CAR_ERR_ARG;
  car::RankPtrs tbl;
  if ((st = check_table(h, dnorm, &tbl)) != CAR_OK) return st;
  if ((st = check_dev(residual_out)) != CAR_OK) return st;
  if ((st = check_dev(weight)) != CAR_OK) return st;
  if ((st = check_dev(dx)) != CAR_OK) return st;
  if ((dresidual_out && !aligned16(dresidual_out)) || (dweight && !aligned16(dweight))) return CAR_ERR_ALIGN;
  if (!h->fused_ok) return CAR_ERR_SIZE;
  if ((st = prepare_backward(h)) != CAR_OK) return st;
  if (dweight && h->backward_groups > 1 && (st = check_dev(workspace)) != CAR_OK) return st;
  float *dw = static_cast<float*>(dweight), *ws = static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (h->backward_pipeline)
    e = car::launch_backward_tma(h->dtype, h->W, tbl, residual_out, weight, eps, dresidual_out, dx, dw, ws, h->d_err, h->M,
                                 h->N, h->vec_per_row, h->backward_tma, s);
  else
    e = car::launch_backward(h->dtype, h->W, tbl, residual_out, weight, eps, dresidual_out, dx, dw, ws, h->d_err, h->M,
                             h->N, h->vec_per_row, h->backward, h->hook, s);
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "reduce_residual_rmsnorm_backward launch");
}

size_t car_ll128_wire_bytes(car_ctx* h) { return live(h) ? (size_t)(128 * h->ll128_lines) : 0; }
size_t car_ll_wire_bytes(car_ctx* h) { return live(h) ? (size_t)(16 * h->ll_lines) : 0; }

car_status car_ll128_encode(car_ctx* h, const void* data, uint64_t flag, void* wire, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if ((st = check_dev_elem(data, h->es)) != CAR_OK) return st;
  if ((st = check_dev(wire)) != CAR_OK) return st;
  const int mis = aligned16(data) ? 0 : 1;
  cudaError_t e = car::launch_ll128_encode(data, h->D, h->ll128_lines, flag, wire, h->ll128_encode_grid[mis],
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "ll128_encode launch");
}

car_status car_ll128_decode_reduce(car_ctx* h, const void* const* wires, uint64_t expected_flag,
                                   int max_polls, void* ar_out, void* stream) {
  car::RankPtrs tbl;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  car_status st = decode_common(h, 0, wires, max_polls, ar_out, s, &tbl);
  if (st != CAR_OK) return st;
  cudaError_t e = car::launch_ll128_decode_reduce(h->dtype, h->W, tbl, h->D, h->ll128_lines, expected_flag,
                                                  max_polls, ar_out, h->log[0], next_log_slot(h, 0),
                                                  h->ll128_decode_grid[aligned16(ar_out) ? 0 : 1], s);
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "ll128_decode_reduce launch");
}

car_status car_ll128_report(car_ctx* h, car_stale_report* out) { return report_common(h, 0, out); }

car_status car_ll_encode(car_ctx* h, const void* data, uint32_t flag, void* wire, void* stream) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if ((st = check_dev(data)) != CAR_OK) return st;
  if ((st = check_dev(wire)) != CAR_OK) return st;
  cudaError_t e = car::launch_ll_encode(data, h->D, flag, wire, h->ll_encode_grid,
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "ll_encode launch");
}

car_status car_ll_decode_reduce(car_ctx* h, const void* const* wires, uint32_t expected_flag,
                                int max_polls, void* ar_out, void* stream) {
  car::RankPtrs tbl;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  car_status st = decode_common(h, 1, wires, max_polls, ar_out, s, &tbl);
  if (st != CAR_OK) return st;
  cudaError_t e = car::launch_ll_decode_reduce(h->dtype, h->W, tbl, h->D, expected_flag, max_polls,
                                               ar_out, h->log[1], next_log_slot(h, 1), h->ll_decode_grid, s);
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "ll_decode_reduce launch");
}

car_status car_ll_report(car_ctx* h, car_stale_report* out) { return report_common(h, 1, out); }

size_t car_lamport_buffer_bytes(car_ctx* h) {
  return (live(h) && h->dtype == CAR_BF16) ? (size_t)(3 * (int64_t)h->W * h->D) : 0;
}

static car_status lamport_checks(car_ctx* h, const void* comm) {
  car_status st = check_handle(h);
  if (st != CAR_OK) return st;
  if (h->dtype != CAR_BF16) {
    snprintf(g_err, sizeof(g_err), "the Lamport format packs bf16 pairs: the handle's dtype must be bf16");
    return CAR_ERR_ARG;
  }
  if (!h->lamport_ok) return CAR_ERR_SIZE;
  return check_dev(comm);
}

car_status car_lamport_init(car_ctx* h, void* comm, void* stream) {
  car_status st = lamport_checks(h, comm);
  if (st != CAR_OK) return st;
  cudaError_t e = car::launch_lamport_fill(comm, 3 * (int64_t)h->W * h->D, h->lamport_grid,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "lamport fill launch");
}

car_status car_lamport_push(car_ctx* h, const void* data, int rank, uint64_t round, void* comm, void* stream) {
  car_status st = lamport_checks(h, comm);
  if (st != CAR_OK) return st;
  if (rank < 0 || rank >= h->W) return CAR_ERR_ARG;
  if ((st = check_dev(data)) != CAR_OK) return st;
  uint8_t* slot = static_cast<uint8_t*>(comm) + ((int64_t)(round % 3) * h->W + rank) * h->D;
  cudaError_t e = car::launch_lamport_push(data, h->D, slot, h->lamport_grid, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "lamport push launch");
}

car_status car_lamport_reduce_residual_rmsnorm(car_ctx* h, void* comm, uint64_t round, int max_polls,
                                               const void* residual, const void* weight, float eps,
                                               void* residual_out, void* norm_out, void* ar_out, void* stream) {
  car_status st = lamport_checks(h, comm);
  if (st != CAR_OK) return st;
  if (max_polls < 1 || !std::isfinite(eps) || eps < 0.f) return CAR_ERR_ARG;
  if ((st = check_dev(residual)) != CAR_OK) return st;
  if ((st = check_dev(weight)) != CAR_OK) return st;
  if ((st = check_dev(residual_out)) != CAR_OK) return st;
  if ((st = check_dev(norm_out)) != CAR_OK) return st;
  if (ar_out && !aligned16(ar_out)) return CAR_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  h->last_stream[2] = s;
  h->decoded[2] = true;
  cudaError_t e;
  const int64_t region_bytes = (int64_t)h->W * h->D;
  uint8_t* base = static_cast<uint8_t*>(comm);
  e = car::launch_lamport_reduce(h->W, base + (int64_t)(round % 3) * region_bytes,
                                 base + (int64_t)((round + 2) % 3) * region_bytes, h->D, residual, weight, eps,
                                 residual_out, norm_out, ar_out, h->log[2], next_log_slot(h, 2), max_polls,
                                 h->d_err, h->M, h->N, h->vec_per_row, h->lamport, s);
  return e == cudaSuccess ? CAR_OK : cuda_fail(e, "lamport receive launch");
}

car_status car_lamport_report(car_ctx* h, car_stale_report* out) { return report_common(h, 2, out); }

}  // extern "C"
