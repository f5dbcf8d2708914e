// fused_quant.cu -- rank sum + residual add + RMSNorm with an 8-bit output and
// its scales: the row kernel of fused_rows.cuh (Q), and its launch.
#include "fused_rows.cuh"

namespace car {

cudaError_t fused_quant_resident_groups(int dtype, int W, const FusedShape& sh, int num_sms, int* groups) {
  return resident_groups<true>(dtype, W, sh, num_sms, groups);
}

cudaError_t launch_fused_quant(int dtype, int W, const RankPtrs& in, const void* residual, const void* weight,
                               float eps, void* residual_out, const QuantOut& out, void* norm_out, void* ar_out,
                               unsigned int* err, int64_t rows, int64_t cols, int vec_per_row, const FusedShape& sh,
                               const WaitHook& hook, cudaStream_t s) {
  FusedFn<true> fn = pick_fused<true>(dtype, W, sh.vpt, sh.cluster);
  if (!fn) return cudaErrorInvalidValue;
  FusedQuantParams p;
  fill_params(p, W, in, residual, weight, eps, residual_out, norm_out, ar_out, err, rows, cols, vec_per_row, sh, hook);
  // A group never straddles two CTAs: pieces are whole multiples of 32 vectors
  // (128 columns of the widest type); threads * vpt still cover a piece, both
  // being multiples of 32 already.
  if (sh.cluster > 1) p.chunk = (p.chunk + 31) / 32 * 32;
  p.out = out;
  return launch_pdl(fn, (unsigned)(sh.groups * sh.cluster), (unsigned)sh.threads, 0, s, (unsigned)sh.cluster, p);
}

}  // namespace car
