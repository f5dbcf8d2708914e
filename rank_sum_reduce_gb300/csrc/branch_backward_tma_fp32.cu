// branch_backward_tma_fp32.cu -- the fp32 instances of branch_backward_tma.cuh.
#include "branch_backward_tma.cuh"

namespace car {
BackwardTmaFn branch_backward_tma_fp32(int vpt, bool split, bool norm, int gate, bool drop) {
  return pick_instance<kFP32>(vpt, split, norm, gate, drop);
}
}  // namespace car
