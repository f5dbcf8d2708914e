// fused_tma.cu -- the pipeline kernel of fused_tma.cuh with the normalised row
// in the input type, its shape and launch.
#include "fused_tma.cuh"

namespace car {

// Largest dynamic shared memory the ring may use per CTA.
constexpr int kTmaSmemBudget = 200 * 1024;

cudaError_t fused_tma_prepare(int dtype, int W, const FusedTmaShape& sh) {
  TmaFn<false> fn = pick_tma<false>(dtype, W, sh.vpt, sh.ls);
  if (!fn) return cudaErrorInvalidValue;
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                              sh.smem);
}

bool fused_tma_shape(int64_t rows, int vec_per_row, int num_sms, int cluster, int W, FusedTmaShape* out) {
  if (cluster != 1 && cluster != 2) return false;
  if (vec_per_row % cluster != 0) return false;
  const int cols = vec_per_row / cluster;
  const int slice = cols * 16;
  if (slice > kTmaSmemBudget / 2) return false;
  int consumers = ((cols + 31) / 32) * 32;
  if (consumers > 512) consumers = 512;
  int vpt = (cols + consumers - 1) / consumers;
  if (vpt == 3) vpt = 4;
  if (vpt > 4 && vpt <= 8) vpt = 8;
  if (vpt > 8) return false;
  // The last kRegSlices slices of a row are loaded by the consumers at W = 8
  // when a thread holds at most two vectors (register room).  Measured on
  // GB300 (N = 8192 bf16 unless noted), it pays only there: W = 8 M = 512
  // 17.4 -> 17.0 us and M = 2048 57.5 -> 55.6 us, but W = 4 (M = 512 and
  // 2048, also N = 4096 fp32), W = 6 and W = 16 were 2-10 % slower.
  const int ls = (vpt <= 2 && W == 8) ? kRegSlices : 0;
  // Ring depth: about one row's bulk-copied slices (at least 6).  Deeper
  // rings keep more bulk copies outstanding and measured slower on GB300
  // (W=8, N=8192 bf16, M=512: 17.5 us with 9 slots, 17.9 us with 12 or 18).
  int slots = W + 1 - ls < 6 ? 6 : W + 1 - ls;
  if (slots > kTmaSmemBudget / slice) slots = kTmaSmemBudget / slice;
  if (slots < 2) return false;
  const int64_t groups = num_sms / cluster;
  out->cluster = cluster;
  out->ls = ls;
  out->consumers = consumers;
  out->vpt = vpt;
  out->slots = slots;
  out->grid = (int)((rows < groups ? rows : groups) * cluster);
  out->smem = slots * slice + (2 * slots + 4) * 8 + 192;
  return true;
}

cudaError_t launch_fused_tma(int dtype, int W, const RankPtrs& in, const void* residual, const void* weight,
                             float eps, void* residual_out, void* norm_out, void* ar_out, unsigned int* err,
                             int64_t rows, int64_t cols, int vec_per_row, const FusedTmaShape& sh,
                             cudaStream_t s) {
  TmaFn<false> fn = pick_tma<false>(dtype, W, sh.vpt, sh.ls);
  if (!fn) return cudaErrorInvalidValue;
  TmaParams p;
  fill_params(p, W, in, residual, weight, eps, residual_out, norm_out, ar_out, err, rows, cols, vec_per_row, sh);
  return launch_pdl(fn, (unsigned)sh.grid, (unsigned)(sh.consumers + 32), (size_t)sh.smem, s,
                    (unsigned)sh.cluster, p);
}

}  // namespace car
