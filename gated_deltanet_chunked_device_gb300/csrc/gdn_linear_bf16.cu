// gdn_linear_bf16.cu -- the gated linear recurrence's scan kernels for bf16 inputs.
#include "gdn_linear_column.cuh"

namespace gdn {

cudaError_t launch_linear_forward_bf16(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream) {
    return p.gate_dt == GDN_DTYPE_F32 ? linear::forward_typed<__nv_bfloat16, float>(p, s, vec, stream)
                                      : linear::forward_typed<__nv_bfloat16, __nv_bfloat16>(p, s, vec, stream);
}

cudaError_t launch_linear_column_forward_bf16(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream) {
    return p.gate_dt == GDN_DTYPE_F32 ? linear::column_forward_typed<__nv_bfloat16, float>(p, s, width, stream)
                                      : linear::column_forward_typed<__nv_bfloat16, __nv_bfloat16>(p, s, width, stream);
}

}  // namespace gdn
