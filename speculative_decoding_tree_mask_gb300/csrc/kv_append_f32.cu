// spec_kv_append for float32 rows.
#include "kv_append.cuh"

namespace specv {

cudaError_t launch_kv_append_f32(const KvAppendParams &p, cudaStream_t st) {
    return launch_kv_append_type<0>(p, st);
}

}  // namespace specv
