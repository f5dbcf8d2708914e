// branch_tma_fp16.cu -- the fp16 instances of branch_tma.cuh.
#include "branch_tma.cuh"

namespace car {
BranchTmaFn branch_tma_fp16(int vpt, bool split, bool norm, int gate, bool drop) {
  return pick_instance<kFP16>(vpt, split, norm, gate, drop);
}
}  // namespace car
