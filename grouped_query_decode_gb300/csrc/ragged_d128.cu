// Attention of packed batches, D = 128.
#include "gqa_ragged.cuh"

namespace gqa {

cudaError_t launch_ragged_d128(const RaggedLaunch& a, bool paged) {
    return paged ? launch_ragged<128, true>(a) : launch_ragged<128, false>(a);
}

}  // namespace gqa
