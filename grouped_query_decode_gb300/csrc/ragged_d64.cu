// Attention of packed batches, D = 64.
#include "gqa_ragged.cuh"

namespace gqa {

cudaError_t launch_ragged_d64(const RaggedLaunch& a, bool paged) {
    return paged ? launch_ragged<64, true>(a) : launch_ragged<64, false>(a);
}

}  // namespace gqa
