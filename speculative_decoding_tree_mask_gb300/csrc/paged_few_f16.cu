// Paged attention of few query rows, half rows.
#include "paged_few.cuh"

namespace specv {

cudaError_t launch_paged_few_f16(const PagedAttnParams &p, int mt, int grid, cudaStream_t st) {
    return launch_paged_few_type<2>(p, mt, grid, st);
}

}  // namespace specv
