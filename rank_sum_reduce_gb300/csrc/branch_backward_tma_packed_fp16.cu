// branch_backward_tma_packed_fp16.cu -- instances of the backward pipeline of a block's branch: fp16, weights packed.
#include "branch_backward_tma.cuh"

namespace car {

BackwardTmaFn branch_backward_tma_packed_fp16(bool split, int gate, bool drop) { return pick_split<kFP16, true, true>(split, gate, drop); }

}  // namespace car
