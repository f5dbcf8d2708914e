// fused.cu -- the row kernel of fused_rows.cuh with the normalised row in the
// input type, and its launch.
#include "fused_rows.cuh"

namespace car {

int fused_max_threads(int W, int vpt) {
  // W outside {1, 2, 4, 8, 16} runs the runtime-W instance, compiled for 512.
  const bool compiled_w = W == 1 || W == 2 || W == 4;
  return (vpt == 1 && compiled_w) ? 1024 : 512;
}

bool fused_has_variant(int W, int vpt) {
  if (vpt == 1) return true;
  return vpt == 2 && (W == 1 || W == 2 || W == 4 || W == 8);
}

cudaError_t fused_resident_groups(int dtype, int W, const FusedShape& sh, int num_sms, int* groups) {
  return resident_groups<false>(dtype, W, sh, num_sms, groups);
}

cudaError_t launch_fused(int dtype, int W, const RankPtrs& in, const void* residual,
                         const void* weight, float eps, void* residual_out, void* norm_out,
                         void* ar_out, unsigned int* err, int64_t rows, int64_t cols, int vec_per_row,
                         const FusedShape& sh, const WaitHook& hook, cudaStream_t s) {
  FusedFn<false> fn = pick_fused<false>(dtype, W, sh.vpt, sh.cluster);
  if (!fn) return cudaErrorInvalidValue;
  FusedParams p;
  fill_params(p, W, in, residual, weight, eps, residual_out, norm_out, ar_out, err, rows, cols, vec_per_row, sh, hook);
  return launch_pdl(fn, (unsigned)(sh.groups * sh.cluster), (unsigned)sh.threads, 0, s, (unsigned)sh.cluster, p);
}

}  // namespace car
