// gdn_linear.cuh -- parameters shared by the host code and the kernels of the
// gated linear recurrence (include/gdn_linear.h).  Not part of the public C ABI.
#pragma once

#include "../../include/gdn_linear.h"
#include "gdn_internal.cuh"

namespace gdn {

struct LinearParams {
    const void* x;
    const void* a;
    const void* b;                 // nullptr = ones
    int64_t x_stride, a_stride, b_stride;
    int32_t D;
    int32_t C;                     // H * D channels
    int32_t H;
    int32_t gate_div;              // channels a gate serves: 1, or D with gates per head
    int32_t x_dt, gate_dt, state_dt;
    const void* cu_seqlens;        // nullptr: one sequence [0, T)
    int cu_i64;
    int32_t N;
    int64_t T;
    const void* initial_state;     // nullptr = zeros
    void* output_state;            // nullptr = not written
    int64_t state_stride;
    const void* state_indices;     // nullptr: row = sequence
    int idx_i64;
    int32_t n_pool;
    int32_t* status;               // nullptr: nothing is reported
    void* y;
    int64_t y_stride;
    float* tile_states;            // [ceil(T / 64)][C]
    const void* dy;
    int64_t dy_stride;
    const float* d_final;
    float* d_initial;
    void* dx;
    void* da;
    void* db;
    int64_t dx_stride, da_stride, db_stride;
    int32_t m;                     // decode: tokens per sequence
    float* scratch;                // backward, heads wider than a block: [T][H][pieces][2] sums
};

// One element of any of the types, at element offset `off`.
__device__ __forceinline__ float load1(const void* p, int64_t off, int32_t dt) {
    if (dt == GDN_DTYPE_F32) return static_cast<const float*>(p)[off];
    if (dt == GDN_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[off]);
    if (dt == GDN_DTYPE_F16) return __half2float(static_cast<const __half*>(p)[off]);
    float lo, hi;
    fp8x2_to_f32(static_cast<const uint8_t*>(p)[off], dt, lo, hi);
    return lo;
}

__device__ __forceinline__ void store1(void* p, int64_t off, int32_t dt, float v) {
    if (dt == GDN_DTYPE_F32)
        static_cast<float*>(p)[off] = v;
    else if (dt == GDN_DTYPE_BF16)
        static_cast<__nv_bfloat16*>(p)[off] = __float2bfloat16_rn(v);
    else if (dt == GDN_DTYPE_F16)
        static_cast<__half*>(p)[off] = __float2half_rn(v);
    else
        static_cast<uint8_t*>(p)[off] = static_cast<uint8_t>(f32_to_fp8x2(v, 0.f, dt));
}

// Blocks of channels of the backward pass: 128 wide, or with gates per head of head_dim channels (0: per channel) as
// many whole heads as fit into 128, or 128 of one head.
inline int64_t backward_blocks(int64_t C, int64_t head_dim) {
    if (head_dim == 0) return (C + 127) / 128;
    if (head_dim > 128) return C / head_dim * ((head_dim + 127) / 128);
    const int64_t width = 128 / head_dim * head_dim;
    return (C + width - 1) / width;
}

// Sums that the blocks of a head leave per token, where a head has more than one: a block has `width` channels.
inline size_t sums_bytes(int64_t T, int64_t C, int64_t head_dim, int64_t width) {
    if (head_dim <= width) return 0;
    return sizeof(float2) * static_cast<size_t>(T) * (C / head_dim) * ((head_dim + width - 1) / width);
}

// What `places` of a scan (tiles, or segments of columns) hand on: the ticket and the flags (zeroed before each run), the
// pairs, the known states and (segments) the exponents of the pairs' products.
struct ScanLayout {
    size_t zeroed, known, exponents, total;
};

inline ScanLayout scan_layout(int64_t places, int64_t flags, int64_t C, bool segments) {
    ScanLayout l{};
    if (places < 2) return l;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l.zeroed = 256 + up(sizeof(uint32_t) * static_cast<size_t>(places) * flags);
    l.known = l.zeroed + up(sizeof(float2) * static_cast<size_t>(places) * C);
    l.total = l.exponents = l.known + up(sizeof(float) * static_cast<size_t>(places) * C);
    if (segments) l.total += up(sizeof(int32_t) * static_cast<size_t>(places) * C);
    return l;
}

inline int64_t tiles_of(int64_t T) { return T > 0 ? (T + GDN_LINEAR_TILE - 1) / GDN_LINEAR_TILE : 1; }

// Any run's workspace with these bounds.  Columns have at most a quarter of the tiles as segments, with a flag for every 16
// channels; tiles have 4 flags for every 128 channels, or fewer.
inline size_t workspace_bound(int64_t T, int64_t C, int64_t head_dim) {
    return scan_layout(tiles_of(T), 4 * backward_blocks(C, head_dim) + (C + 15) / 16, C, false).total + sums_bytes(T, C, head_dim, 16) + 256;
}

// A map of T rows of C elements, `stride` elements apart, for boxes of `width` elements of `tokens` rows; what lies
// outside reads as zeros.
bool encode_rows(CUtensorMap* map, const void* base, int32_t dt, int64_t stride, int64_t C, int64_t T, int width, int tokens);

// A run's workspace in bytes (at most workspace_bound of the plan's bounds), and the runs themselves.
size_t linear_forward_workspace(const LinearParams& p);
size_t linear_backward_workspace(const LinearParams& p);
cudaError_t launch_linear_forward(const LinearParams& p, void* workspace, cudaStream_t stream);
cudaError_t launch_linear_backward(const LinearParams& p, void* workspace, cudaStream_t stream);
cudaError_t launch_linear_decode(const LinearParams& p, cudaStream_t stream);

}  // namespace gdn
