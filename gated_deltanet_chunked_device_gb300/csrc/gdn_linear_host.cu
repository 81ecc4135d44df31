// gdn_linear_host.cu -- host side of include/gdn_linear.h: plan validation,
// run-time argument checks and launches.  Nothing here synchronises, allocates
// device memory or reads it.
#include <new>

#include "gdn_linear.cuh"

struct gdn_linear_plan_s {
    gdn_linear_desc desc;
    size_t workspace;
};

namespace {

constexpr uint32_t kKnownFlags = GDN_LINEAR_HAS_B | GDN_LINEAR_GATES_PER_HEAD | GDN_LINEAR_HAS_INITIAL_STATE |
                                 GDN_LINEAR_OUTPUT_FINAL_STATE | GDN_LINEAR_HAS_STATE_INDICES |
                                 GDN_LINEAR_CU_SEQLENS_I64 | GDN_LINEAR_STATE_INDICES_I64;
constexpr int64_t kMaxChannels = 1 << 20;

bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool io_dtype(gdn_dtype t) { return t == GDN_DTYPE_F32 || t == GDN_DTYPE_BF16 || t == GDN_DTYPE_F16; }

bool storage_dtype(gdn_dtype t) { return io_dtype(t) || t == GDN_DTYPE_F8E4M3 || t == GDN_DTYPE_F8E5M2; }

// A required tensor: present, aligned to its element, its rows apart.
bool tensor_ok(const void* p, gdn_dtype t, int64_t& stride, int64_t row) {
    if (!p || !aligned(p, gdn::dtype_bytes(t))) return false;
    if (stride == 0) stride = row;
    return stride >= row;
}

bool workspace_ok(const void* p, size_t bytes, size_t needed) { return needed == 0 || (p && aligned(p, 16) && bytes >= needed); }

enum class Run { kForward, kBackward, kDecode };

// Checks the arguments that the runs share and fills the kernels' parameters.
gdn_status make_params(gdn_linear_plan_t plan, const gdn_linear_args* args, Run run, gdn::LinearParams* out) {
    if (!plan || !args) return GDN_ERR_INVALID_ARG;
    const gdn_linear_desc& d = plan->desc;
    gdn_linear_args a = *args;
    const uint32_t f = d.flags;
    const int64_t C = static_cast<int64_t>(d.num_heads) * d.head_dim;
    const int64_t gate_row = (f & GDN_LINEAR_GATES_PER_HEAD) ? d.num_heads : C;
    const bool has_b = (f & GDN_LINEAR_HAS_B) != 0;
    if (a.num_seqs < 0 || a.num_seqs > d.max_num_seqs || a.total_tokens < 0 || a.total_tokens > d.max_total_tokens)
        return GDN_ERR_INVALID_ARG;
    if (a.num_seqs == 0 && a.total_tokens != 0) return GDN_ERR_INVALID_ARG;
    if (run != Run::kDecode && !a.cu_seqlens && a.num_seqs > 1) return GDN_ERR_INVALID_ARG;
    if (a.cu_seqlens && !aligned(a.cu_seqlens, (f & GDN_LINEAR_CU_SEQLENS_I64) ? 8 : 4)) return GDN_ERR_INVALID_ARG;
    if (a.total_tokens > 0) {
        if (!tensor_ok(a.x, d.x_dtype, a.x_stride, C) || !tensor_ok(a.a, d.gate_dtype, a.a_stride, gate_row))
            return GDN_ERR_INVALID_ARG;
        if (has_b && !tensor_ok(a.b, d.gate_dtype, a.b_stride, gate_row)) return GDN_ERR_INVALID_ARG;
        if (run == Run::kBackward) {
            if (!tensor_ok(a.dy, d.x_dtype, a.dy_stride, C) || !tensor_ok(a.dx, d.x_dtype, a.dx_stride, C) ||
                !tensor_ok(a.da, d.gate_dtype, a.da_stride, gate_row))
                return GDN_ERR_INVALID_ARG;
            if (has_b && !tensor_ok(a.db, d.gate_dtype, a.db_stride, gate_row)) return GDN_ERR_INVALID_ARG;
            if (a.total_tokens > GDN_LINEAR_TILE && !a.tile_states) return GDN_ERR_INVALID_ARG;
        } else if (!tensor_ok(a.y, d.x_dtype, a.y_stride, C)) {
            return GDN_ERR_INVALID_ARG;
        }
    }
    if (!aligned(a.tile_states, 4) || !aligned(a.d_final_state, 4) || !aligned(a.d_initial_state, 4) ||
        !aligned(a.device_status, 4))
        return GDN_ERR_INVALID_ARG;
    gdn::LinearParams p{};
    if ((f & GDN_LINEAR_HAS_INITIAL_STATE) && a.num_seqs > 0) {
        if (!tensor_ok(a.initial_state, d.state_dtype, a.state_stride, C)) return GDN_ERR_INVALID_ARG;
        p.initial_state = a.initial_state;
    }
    if ((f & GDN_LINEAR_OUTPUT_FINAL_STATE) && run != Run::kBackward && a.num_seqs > 0) {
        if (!tensor_ok(a.output_state, d.state_dtype, a.state_stride, C)) return GDN_ERR_INVALID_ARG;
        p.output_state = a.output_state;
    }
    if (f & GDN_LINEAR_HAS_STATE_INDICES) {
        if (run == Run::kBackward) return GDN_ERR_UNSUPPORTED;
        if (a.num_seqs > 0 && (!a.state_indices || a.n_pool <= 0 ||
                               !aligned(a.state_indices, (f & GDN_LINEAR_STATE_INDICES_I64) ? 8 : 4)))
            return GDN_ERR_INVALID_ARG;
        p.state_indices = a.state_indices;
        p.idx_i64 = (f & GDN_LINEAR_STATE_INDICES_I64) ? 1 : 0;
        p.n_pool = a.n_pool;
    }
    p.x = a.x;
    p.a = a.a;
    p.b = has_b ? a.b : nullptr;
    p.x_stride = a.x_stride;
    p.a_stride = a.a_stride;
    p.b_stride = a.b_stride;
    p.H = d.num_heads;
    p.D = d.head_dim;
    p.C = static_cast<int32_t>(C);
    p.gate_div = (f & GDN_LINEAR_GATES_PER_HEAD) ? d.head_dim : 1;
    p.x_dt = d.x_dtype;
    p.gate_dt = d.gate_dtype;
    p.state_dt = d.state_dtype;
    p.cu_seqlens = a.cu_seqlens;
    p.cu_i64 = (f & GDN_LINEAR_CU_SEQLENS_I64) ? 1 : 0;
    p.N = a.num_seqs;
    p.T = a.total_tokens;
    p.state_stride = a.state_stride;
    p.status = a.device_status;
    p.y = a.y;
    p.y_stride = a.y_stride;
    p.tile_states = a.tile_states;
    p.dy = a.dy;
    p.dy_stride = a.dy_stride;
    p.d_final = a.d_final_state;
    p.d_initial = a.d_initial_state;
    p.dx = a.dx;
    p.da = a.da;
    p.db = has_b ? a.db : nullptr;
    p.dx_stride = a.dx_stride;
    p.da_stride = a.da_stride;
    p.db_stride = a.db_stride;
    *out = p;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_linear_plan(const gdn_linear_desc* desc, gdn_linear_plan_t* plan, size_t* workspace_bytes) {
    if (!desc || !plan || !workspace_bytes) return GDN_ERR_INVALID_ARG;
    *plan = nullptr;
    const gdn_linear_desc& d = *desc;
    if (d.flags & ~kKnownFlags) return GDN_ERR_INVALID_ARG;
    if (d.num_heads < 1 || d.head_dim < 1 || d.max_total_tokens < 0 || d.max_num_seqs < 0) return GDN_ERR_INVALID_ARG;
    if (static_cast<int64_t>(d.num_heads) * d.head_dim > kMaxChannels) return GDN_ERR_UNSUPPORTED;
    if (d.max_total_tokens > 0x7fffffffLL - GDN_LINEAR_TILE) return GDN_ERR_UNSUPPORTED;
    if (!io_dtype(d.x_dtype) || !storage_dtype(d.state_dtype)) return GDN_ERR_UNSUPPORTED;
    if (d.gate_dtype != d.x_dtype && d.gate_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
    const int64_t C = static_cast<int64_t>(d.num_heads) * d.head_dim;
    const int64_t head_dim = (d.flags & GDN_LINEAR_GATES_PER_HEAD) ? d.head_dim : 0;
    // tiles of one launch
    if (gdn::tiles_of(d.max_total_tokens) * gdn::backward_blocks(C, head_dim) > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    gdn_linear_plan_s* p = new (std::nothrow) gdn_linear_plan_s;
    if (!p) return GDN_ERR_INVALID_ARG;
    p->desc = d;
    p->workspace = gdn::workspace_bound(d.max_total_tokens, C, head_dim);
    *plan = p;
    *workspace_bytes = p->workspace;
    return GDN_OK;
}

void gdn_linear_plan_destroy(gdn_linear_plan_t plan) { delete plan; }

size_t gdn_linear_run_workspace(gdn_linear_plan_t plan, const gdn_linear_args* args, int32_t backward) {
    gdn::LinearParams p;
    if (make_params(plan, args, backward ? Run::kBackward : Run::kForward, &p) != GDN_OK || p.N == 0) return 0;
    return backward ? gdn::linear_backward_workspace(p) : gdn::linear_forward_workspace(p);
}

gdn_status gdn_linear_forward_run(gdn_linear_plan_t plan, const gdn_linear_args* args, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    gdn::LinearParams p;
    const gdn_status st = make_params(plan, args, Run::kForward, &p);
    if (st != GDN_OK) return st;
    if (p.N == 0) return GDN_OK;
    if (!workspace_ok(workspace, workspace_bytes, gdn::linear_forward_workspace(p))) return GDN_ERR_INVALID_ARG;
    return gdn::launch_linear_forward(p, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_linear_backward_run(gdn_linear_plan_t plan, const gdn_linear_args* args, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    gdn::LinearParams p;
    const gdn_status st = make_params(plan, args, Run::kBackward, &p);
    if (st != GDN_OK) return st;
    if (p.N == 0) return GDN_OK;
    if (!workspace_ok(workspace, workspace_bytes, gdn::linear_backward_workspace(p))) return GDN_ERR_INVALID_ARG;
    return gdn::launch_linear_backward(p, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_linear_decode_run(gdn_linear_plan_t plan, const gdn_linear_args* args, int32_t tokens_per_seq,
                                 void* stream) {
    gdn::LinearParams p;
    const gdn_status st = make_params(plan, args, Run::kDecode, &p);
    if (st != GDN_OK) return st;
    if (tokens_per_seq < 1 || p.T != static_cast<int64_t>(p.N) * tokens_per_seq) return GDN_ERR_INVALID_ARG;
    if (p.N == 0) return GDN_OK;
    p.m = tokens_per_seq;
    p.tile_states = nullptr;
    return gdn::launch_linear_decode(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
