// branch_backward_tma_bf16.cu -- the bf16 instances of branch_backward_tma.cuh.
#include "branch_backward_tma.cuh"

namespace car {
BackwardTmaFn branch_backward_tma_bf16(int vpt, bool split, bool norm, int gate, bool drop) {
  return pick_instance<kBF16>(vpt, split, norm, gate, drop);
}
}  // namespace car
