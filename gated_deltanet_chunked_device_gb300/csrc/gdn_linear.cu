// gdn_linear.cu -- kernels of the gated linear recurrence (include/gdn_linear.h):
//
//     h_t = a_t h_{t-1} + b_t x_t
//
// One block of 128 threads per (sequence, head); a thread owns every 128th
// channel of the head and walks the sequence's tokens.  Right for every case,
// and as slow as the longest sequence.
#include "gdn_linear.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void report(int32_t* status, int32_t bit) {
    if (status) atomicOr(status, bit);
}

// The sequence's tokens [s, e); false (and reported) when cu_seqlens is malformed.
__device__ __forceinline__ bool seq_range(const LinearParams& p, int64_t i, int64_t& s, int64_t& e) {
    if (p.m > 0) {
        s = i * p.m;
        e = s + p.m;
        return true;
    }
    if (!p.cu_seqlens) {
        s = 0;
        e = p.T;
        return true;
    }
    s = load_index(p.cu_seqlens, p.cu_i64, i);
    e = load_index(p.cu_seqlens, p.cu_i64, i + 1);
    const bool ok = s >= 0 && s <= e && e <= p.T && (i > 0 || s == 0) && (i + 1 < p.N || e == p.T);
    if (!ok) report(p.status, GDN_DEVICE_ERR_CU_SEQLENS);
    return ok;
}

__device__ __forceinline__ bool seq_row(const LinearParams& p, int64_t i, int64_t& row) {
    row = i;
    if (!p.state_indices) return true;
    row = load_index(p.state_indices, p.idx_i64, i);
    if (row >= 0 && row < p.n_pool) return true;
    report(p.status, GDN_DEVICE_ERR_STATE_INDEX_RANGE);
    return false;
}

__global__ void __launch_bounds__(kThreads) gdn_linear_forward_kernel(LinearParams p) {
    const int64_t i = blockIdx.x / p.H;
    const int32_t h = static_cast<int32_t>(blockIdx.x % p.H);
    int64_t s, e, row;
    if (!seq_range(p, i, s, e) || !seq_row(p, i, row)) return;
    for (int32_t d = threadIdx.x; d < p.D; d += kThreads) {
        const int64_t c = static_cast<int64_t>(h) * p.D + d;
        float st = p.initial_state ? load1(p.initial_state, row * p.state_stride + c, p.state_dt) : 0.f;
        for (int64_t t = s; t < e; ++t) {
            float u = load1(p.x, t * p.x_stride + c, p.x_dt);
            if (p.b) u *= load1(p.b, t * p.b_stride + c / p.gate_div, p.gate_dt);
            st = fmaf(load1(p.a, t * p.a_stride + c / p.gate_div, p.gate_dt), st, u);
            store1(p.y, t * p.y_stride + c, p.x_dt, st);
            if (p.tile_states && (t % GDN_LINEAR_TILE == GDN_LINEAR_TILE - 1 || t == p.T - 1))
                p.tile_states[t / GDN_LINEAR_TILE * p.C + c] = st;
        }
        if (p.output_state) store1(p.output_state, row * p.state_stride + c, p.state_dt, st);
    }
}

__global__ void __launch_bounds__(kThreads) gdn_linear_backward_kernel(LinearParams p) {
    __shared__ float sums[2][kThreads / 32];
    const int64_t i = blockIdx.x / p.H;
    const int32_t h = static_cast<int32_t>(blockIdx.x % p.H);
    int64_t s, e;
    if (!seq_range(p, i, s, e)) return;
    for (int32_t d0 = 0; d0 < p.D; d0 += kThreads) {
        const int32_t d = d0 + threadIdx.x;
        const bool on = d < p.D;
        const int64_t c = static_cast<int64_t>(h) * p.D + (on ? d : 0);
        float carry = on && p.d_final ? p.d_final[i * p.C + c] : 0.f;
        float before[GDN_LINEAR_TILE];  // the state before each token of a tile
        for (int64_t end = e; end > s;) {
            const int64_t f = (end - 1) / GDN_LINEAR_TILE;
            const int64_t from = f * GDN_LINEAR_TILE > s ? f * GDN_LINEAR_TILE : s;
            float st = 0.f;
            if (from > s)
                st = p.tile_states[(f - 1) * p.C + c];
            else if (p.initial_state)
                st = load1(p.initial_state, i * p.state_stride + c, p.state_dt);
            for (int64_t t = from; t < end; ++t) {
                before[t - from] = st;
                float u = load1(p.x, t * p.x_stride + c, p.x_dt);
                if (p.b) u *= load1(p.b, t * p.b_stride + c / p.gate_div, p.gate_dt);
                st = fmaf(load1(p.a, t * p.a_stride + c / p.gate_div, p.gate_dt), st, u);
            }
            for (int64_t t = end - 1; t >= from; --t) {
                const float g = load1(p.dy, t * p.dy_stride + c, p.x_dt) + carry;
                const float x = load1(p.x, t * p.x_stride + c, p.x_dt);
                const float b = p.b ? load1(p.b, t * p.b_stride + c / p.gate_div, p.gate_dt) : 1.f;
                carry = load1(p.a, t * p.a_stride + c / p.gate_div, p.gate_dt) * g;
                float da = on ? g * before[t - from] : 0.f, db = on ? g * x : 0.f;
                if (on) store1(p.dx, t * p.dx_stride + c, p.x_dt, b * g);
                if (p.gate_div == 1) {
                    if (on) store1(p.da, t * p.da_stride + c, p.gate_dt, da);
                    if (on && p.db) store1(p.db, t * p.db_stride + c, p.gate_dt, db);
                    continue;
                }
                for (int o = 16; o > 0; o >>= 1) {
                    da += __shfl_xor_sync(0xffffffffu, da, o);
                    db += __shfl_xor_sync(0xffffffffu, db, o);
                }
                if (threadIdx.x % 32 == 0) {
                    sums[0][threadIdx.x / 32] = da;
                    sums[1][threadIdx.x / 32] = db;
                }
                __syncthreads();
                if (threadIdx.x < 2) {
                    float v = 0.f;
                    for (int w = 0; w < kThreads / 32; ++w) v += sums[threadIdx.x][w];
                    float* acc = p.scratch + (t * p.H + h) * 2 + threadIdx.x;
                    if (d0 > 0) v += *acc;
                    if (d0 + kThreads < p.D)
                        *acc = v;
                    else if (threadIdx.x == 0)
                        store1(p.da, t * p.da_stride + h, p.gate_dt, v);
                    else if (p.db)
                        store1(p.db, t * p.db_stride + h, p.gate_dt, v);
                }
                __syncthreads();
            }
            end = from;
        }
        if (on && p.d_initial) p.d_initial[i * p.C + c] = carry;
    }
}

}  // namespace

cudaError_t launch_linear_forward(const LinearParams& p, cudaStream_t stream) {
    gdn_linear_forward_kernel<<<static_cast<unsigned>(static_cast<int64_t>(p.N) * p.H), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_linear_decode(const LinearParams& p, cudaStream_t stream) { return launch_linear_forward(p, stream); }

cudaError_t launch_linear_backward(const LinearParams& p, cudaStream_t stream) {
    gdn_linear_backward_kernel<<<static_cast<unsigned>(static_cast<int64_t>(p.N) * p.H), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
