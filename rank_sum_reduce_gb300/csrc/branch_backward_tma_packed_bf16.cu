// branch_backward_tma_packed_bf16.cu -- instances of the backward pipeline of a block's branch: bf16, weights packed.
#include "branch_backward_tma.cuh"

namespace car {

BackwardTmaFn branch_backward_tma_packed_bf16(bool split, int gate, bool drop) { return pick_split<kBF16, true, true>(split, gate, drop); }

}  // namespace car
