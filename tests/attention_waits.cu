// attention_waits.cu -- attention over a paged cache on the tensor cores with a limit of a few cycles for its waits, or with keys and
// values that do not come: for a test of what the kernel does when a wait runs out.
#include "gdn_attention.cu"

extern "C" {

// gdn_attention_run with waits of `cycles`.  missing: half of each tile is never fetched, so that no tile is ever there (pages of
// 64 tokens or fewer; tiled copies).  Returns 0, a CUDA error, or -1 for arguments that do not go to the tensor cores.
int waits_attention(const gdn_kv_batch* batch, const gdn_kv_cache* cache, const gdn_attention_args* args, void* workspace,
                    size_t workspace_bytes, long long cycles, int missing, void* stream) {
    gdn::Route r;
    if (gdn::make_route(batch, cache, args, &r) != GDN_OK || r.streams == 0) return -1;
    if (workspace_bytes < gdn::attn_workspace(r.blocks, r.rows, r.p.c.head_dim)) return -1;
    if (missing && (r.tc.plain || r.tc.boxes < 2)) return -1;
    if (missing) r.tc.boxes /= 2;
    r.tc.wait_cycles = cycles;
    gdn::attn_place(&r.p, workspace, r.blocks, r.rows);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = gdn::launch_tc(r, s);
    return e == cudaSuccess ? gdn::launch_attention_join(r.p, r.blocks, s) : e;
}
}
