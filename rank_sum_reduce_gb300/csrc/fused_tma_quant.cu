// fused_tma_quant.cu -- rank sum + residual add + RMSNorm with an 8-bit output
// and its scales for many rows: the pipeline kernel of fused_tma.cuh (Q).
#include "fused_tma.cuh"

namespace car {

cudaError_t fused_tma_quant_prepare(int dtype, int W, FusedTmaShape* sh) {
  TmaFn<true> fn = pick_tma<true>(dtype, W, sh->vpt, sh->ls);
  if (!fn) return cudaErrorInvalidValue;
  sh->smem += 32 * (int)sizeof(uint32_t);  // the warps' max |t|
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, sh->smem);
}

cudaError_t launch_fused_tma_quant(int dtype, int W, const RankPtrs& in, const void* residual, const void* weight,
                                   float eps, void* residual_out, const QuantOut& out, void* norm_out, void* ar_out,
                                   unsigned int* err, int64_t rows, int64_t cols, int vec_per_row,
                                   const FusedTmaShape& sh, cudaStream_t s) {
  TmaFn<true> fn = pick_tma<true>(dtype, W, sh.vpt, sh.ls);
  if (!fn || sh.cluster != 1) return cudaErrorInvalidValue;
  TmaQuantParams p;
  fill_params(p, W, in, residual, weight, eps, residual_out, norm_out, ar_out, err, rows, cols, vec_per_row, sh);
  p.out = out;
  return launch_pdl(fn, (unsigned)sh.grid, (unsigned)(sh.consumers + 32), (size_t)sh.smem, s, 1, p);
}

}  // namespace car
