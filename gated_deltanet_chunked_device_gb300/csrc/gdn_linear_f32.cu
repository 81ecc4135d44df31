// gdn_linear_f32.cu -- the gated linear recurrence's scan kernels for f32 inputs.
#include "gdn_linear_column.cuh"

namespace gdn {

cudaError_t launch_linear_forward_f32(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream) {
    return linear::forward_typed<float, float>(p, s, vec, stream);
}

cudaError_t launch_linear_column_forward_f32(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream) {
    return linear::column_forward_typed<float, float>(p, s, width, stream);
}

}  // namespace gdn
