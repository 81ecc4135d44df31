// gdn_linear_f16.cu -- the gated linear recurrence's scan kernels for f16 inputs.
#include "gdn_linear_column.cuh"

namespace gdn {

cudaError_t launch_linear_forward_f16(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream) {
    return p.gate_dt == GDN_DTYPE_F32 ? linear::forward_typed<__half, float>(p, s, vec, stream)
                                      : linear::forward_typed<__half, __half>(p, s, vec, stream);
}

cudaError_t launch_linear_column_forward_f16(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream) {
    return p.gate_dt == GDN_DTYPE_F32 ? linear::column_forward_typed<__half, float>(p, s, width, stream)
                                      : linear::column_forward_typed<__half, __half>(p, s, width, stream);
}

}  // namespace gdn
