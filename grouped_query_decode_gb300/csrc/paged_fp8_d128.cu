// Paged e4m3 attention kernels for head dimension 128.
#include "gqa_paged_fp8.cuh"

namespace gqa {

cudaError_t launch_paged_fp8_d128(const PagedFp8Launch& a) { return launch_paged_fp8_rows<128>(a); }

}  // namespace gqa
