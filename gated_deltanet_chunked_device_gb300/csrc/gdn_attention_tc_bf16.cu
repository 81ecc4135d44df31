// gdn_attention_tc_bf16.cu -- attention's tensor core kernels for bf16.
#include "gdn_attention_tc.cuh"

namespace gdn {

cudaError_t launch_attention_tc_bf16(const attn_tc::TcParams& p, const CUtensorMap* maps, int streams, int32_t blocks, cudaStream_t stream) {
    return attn_tc::launch_typed<__nv_bfloat16>(p, maps, streams, blocks, stream);
}

}  // namespace gdn
