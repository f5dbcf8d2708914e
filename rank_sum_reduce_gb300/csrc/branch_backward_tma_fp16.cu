// branch_backward_tma_fp16.cu -- instances of the backward pipeline of a block's branch: fp16.
#include "branch_backward_tma.cuh"

namespace car {

BackwardTmaFn branch_backward_tma_fp16(bool split, bool norm, int gate, bool drop) { return pick_norm<kFP16>(split, norm, gate, drop); }

}  // namespace car
