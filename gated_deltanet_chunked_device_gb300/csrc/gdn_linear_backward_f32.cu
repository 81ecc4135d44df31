// gdn_linear_backward_f32.cu -- the gated linear recurrence's backward kernels for f32 inputs.
#include "gdn_linear_column_backward.cuh"

namespace gdn {

cudaError_t launch_linear_backward_f32(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream) {
    return linear::backward_typed<float, float>(p, s, vec, stream);
}

cudaError_t launch_linear_column_backward_f32(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream) {
    return linear::column_backward_typed<float, float>(p, s, width, stream);
}

}  // namespace gdn
