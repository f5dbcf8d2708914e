// branch_backward_tma_bf16.cu -- instances of the backward pipeline of a block's branch: bf16.
#include "branch_backward_tma.cuh"

namespace car {

BackwardTmaFn branch_backward_tma_bf16(bool split, bool norm, int gate, bool drop) { return pick_norm<kBF16>(split, norm, gate, drop); }

}  // namespace car
