// Paged attention on the tcgen05 tensor cores, half rows.
#include "paged_tc.cuh"

namespace specv {

cudaError_t launch_paged_tc_f16(const PagedAttnParams &p, int grid, cudaStream_t st) {
    return launch_paged_tc_type<2>(p, grid, st);
}

}  // namespace specv
