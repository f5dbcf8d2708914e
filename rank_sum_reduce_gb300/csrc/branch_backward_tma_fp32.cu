// branch_backward_tma_fp32.cu -- instances of the backward pipeline of a block's branch: fp32.
#include "branch_backward_tma.cuh"

namespace car {

BackwardTmaFn branch_backward_tma_fp32(bool split, bool norm, int gate, bool drop) { return pick_norm<kFP32>(split, norm, gate, drop); }

}  // namespace car
