// gdn_attention_tc_f16.cu -- attention's tensor core kernels for f16.
#include "gdn_attention_tc.cuh"

namespace gdn {

cudaError_t launch_attention_tc_f16(const attn_tc::TcParams& p, const CUtensorMap* maps, int streams, int32_t blocks, cudaStream_t stream) {
    return attn_tc::launch_typed<__half>(p, maps, streams, blocks, stream);
}

}  // namespace gdn
