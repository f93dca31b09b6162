// spec_kv_append by the type of the rows; bfloat16 rows here.
#include "kv_append.cuh"

namespace specv {

cudaError_t launch_kv_append_f32(const KvAppendParams &p, cudaStream_t st);
cudaError_t launch_kv_append_f16(const KvAppendParams &p, cudaStream_t st);

cudaError_t launch_kv_append(const KvAppendParams &p, cudaStream_t st) {
    if (p.T <= 0) return cudaSuccess;
    if (p.dtype == SPEC_F32) return launch_kv_append_f32(p, st);
    if (p.dtype == SPEC_F16) return launch_kv_append_f16(p, st);
    return launch_kv_append_type<1>(p, st);
}

}  // namespace specv
