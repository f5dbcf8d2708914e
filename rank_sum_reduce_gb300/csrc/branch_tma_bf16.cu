// branch_tma_bf16.cu -- the bf16 instances of branch_tma.cuh.
#include "branch_tma.cuh"

namespace car {
BranchTmaFn branch_tma_bf16(int vpt, bool split, bool norm, int gate, bool drop) {
  return pick_instance<kBF16>(vpt, split, norm, gate, drop);
}
}  // namespace car
