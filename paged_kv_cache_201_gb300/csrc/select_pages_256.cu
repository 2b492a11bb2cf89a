// Page selection at head_dim 256; one translation unit per head dim, so that they compile side by side.
#include "select_pages.cuh"

namespace pa {

cudaError_t launch_select_pages_256(const SparseParams &sp, int dtype, int sms, cudaStream_t stream) {
    return launch_select_d<256>(sp, dtype, sms, stream);
}

}  // namespace pa
