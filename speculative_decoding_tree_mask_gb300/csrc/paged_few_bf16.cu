// Paged attention of few query rows, bfloat16 rows.
#include "paged_few.cuh"

namespace specv {

cudaError_t launch_paged_few_bf16(const PagedAttnParams &p, int mt, int grid, cudaStream_t st) {
    return launch_paged_few_type<1>(p, mt, grid, st);
}

}  // namespace specv
