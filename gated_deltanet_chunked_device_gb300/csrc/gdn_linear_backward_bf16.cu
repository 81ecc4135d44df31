// gdn_linear_backward_bf16.cu -- the gated linear recurrence's backward kernels for bf16 inputs.
#include "gdn_linear_column_backward.cuh"

namespace gdn {

cudaError_t launch_linear_backward_bf16(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream) {
    return p.gate_dt == GDN_DTYPE_F32 ? linear::backward_typed<__nv_bfloat16, float>(p, s, vec, stream)
                                      : linear::backward_typed<__nv_bfloat16, __nv_bfloat16>(p, s, vec, stream);
}

cudaError_t launch_linear_column_backward_bf16(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream) {
    return p.gate_dt == GDN_DTYPE_F32 ? linear::column_backward_typed<__nv_bfloat16, float>(p, s, width, stream)
                                      : linear::column_backward_typed<__nv_bfloat16, __nv_bfloat16>(p, s, width, stream);
}

}  // namespace gdn
