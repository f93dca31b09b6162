// Paged attention on the tcgen05 tensor cores, bfloat16 rows.
#include "paged_tc.cuh"

namespace specv {

cudaError_t launch_paged_tc_bf16(const PagedAttnParams &p, int grid, cudaStream_t st) {
    return launch_paged_tc_type<1>(p, grid, st);
}

}  // namespace specv
