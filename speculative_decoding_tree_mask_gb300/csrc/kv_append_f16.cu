// spec_kv_append for half rows.
#include "kv_append.cuh"

namespace specv {

cudaError_t launch_kv_append_f16(const KvAppendParams &p, cudaStream_t st) {
    return launch_kv_append_type<2>(p, st);
}

}  // namespace specv
