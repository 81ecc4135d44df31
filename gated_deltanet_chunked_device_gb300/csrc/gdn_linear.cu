// gdn_linear.cu -- kernels of the gated linear recurrence (include/gdn_linear.h):
//
//     h_t = a_t h_{t-1} + b_t x_t
//
// One block of 128 threads per (sequence, head); a thread owns every 128th
// channel of the head and walks the sequence's tokens.  Right for every case,
// and as slow as the longest sequence.
#include <cudaTypedefs.h>

#include "gdn_linear_column.cuh"

namespace gdn {

cudaError_t launch_linear_forward_bf16(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream);
cudaError_t launch_linear_column_forward_bf16(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream);
cudaError_t launch_linear_forward_f16(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream);
cudaError_t launch_linear_column_forward_f16(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream);
cudaError_t launch_linear_forward_f32(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream);
cudaError_t launch_linear_column_forward_f32(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream);
cudaError_t launch_linear_backward_bf16(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream);
cudaError_t launch_linear_column_backward_bf16(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream);
cudaError_t launch_linear_backward_f16(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream);
cudaError_t launch_linear_column_backward_f16(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream);
cudaError_t launch_linear_backward_f32(const LinearParams& p, const linear::ScanSpace& s, bool vec, cudaStream_t stream);
cudaError_t launch_linear_column_backward_f32(const LinearParams& p, const linear::Segments& s, int width, cudaStream_t stream);

namespace {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ok ? f : nullptr);
    }();
    return fn;
}

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

__global__ void __launch_bounds__(kThreads) gdn_linear_decode_kernel(LinearParams p) {
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

// Whether rows of this tensor can be read 4 elements at a time.
bool vector_of_4(const void* p, int64_t stride, int32_t dt) {
    return reinterpret_cast<uintptr_t>(p) % (4 * dtype_bytes(dt)) == 0 && stride % 4 == 0;
}

// Loads of 4 channels: x, gates per channel and states allow them, and a head's channels do not share 4 with another's.
bool rows_vector(const LinearParams& p) {
    bool ok = p.C % 4 == 0 && vector_of_4(p.x, p.x_stride, p.x_dt) && vector_of_4(p.initial_state, p.state_stride, p.state_dt) &&
              vector_of_4(p.output_state, p.state_stride, p.state_dt);
    if (p.gate_div != 1) return ok && p.D % 4 == 0;
    return ok && vector_of_4(p.a, p.a_stride, p.gate_dt) && vector_of_4(p.b, p.b_stride, p.gate_dt);
}

// Whether rows can be copied 16 bytes at a time.
bool vector_of_16_bytes(const void* p, int64_t stride, int32_t dt, int64_t row) {
    const int64_t e = dtype_bytes(dt);
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * e % 16 == 0 && row * e % 16 == 0;
}

bool inputs_wide(const LinearParams& p) {
    const bool x = vector_of_16_bytes(p.x, p.x_stride, p.x_dt, p.C);
    if (p.gate_div != 1) return x;
    return x && vector_of_16_bytes(p.a, p.a_stride, p.gate_dt, p.C) && vector_of_16_bytes(p.b, p.b_stride, p.gate_dt, p.C);
}

// Width and time segments of the columns, with runs of `run` tokens.
linear::Segments segments(const LinearParams& p, int run, int* width) {
    const int64_t sms = multiprocessors(), blocks32 = (p.C + 31) / 32;
    int64_t segs = sms / blocks32;
    *width = 5 * blocks32 < 3 * sms && segs < 3 ? 16 : 32;
    linear::Segments s{};
    const int64_t tokens = 8 * (128 / *width) * run, n = p.T > 0 ? (p.T + tokens - 1) / tokens : 1;
    if (segs > n / 2) segs = n / 2;
    s.space.blocks = static_cast<uint32_t>((p.C + *width - 1) / *width);
    s.space.nt = 1;
    s.first = s.stages = static_cast<int32_t>(n);
    if (segs >= 3 && *width == 32) {
        // first + (segs - 1) stages = n, the first one six tenths of another
        s.stages = static_cast<int32_t>((10 * n + 10 * segs - 5) / (10 * segs - 4));
        s.first = static_cast<int32_t>((6 * s.stages + 9) / 10);
        s.space.nt = n <= s.first ? 1 : 1 + (n - s.first + s.stages - 1) / s.stages;
    }
    return s;
}

// The workspace as the kernels of columns take it.
cudaError_t segment_space(const LinearParams& p, void* workspace, cudaStream_t stream, linear::Segments* seg) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    linear::ScanSpace& s = seg->space;
    const size_t zeroed = 256 + sizeof(uint32_t) * s.nt * s.blocks, pairs = (zeroed + 255) / 256 * 256;
    s.ticket = reinterpret_cast<uint32_t*>(ws);
    s.flags = reinterpret_cast<uint32_t*>(ws + 256);
    s.pairs = reinterpret_cast<float2*>(ws + pairs);
    s.known = reinterpret_cast<float*>(ws + pairs + sizeof(float2) * s.nt * p.C);
    return s.nt > 1 ? cudaMemsetAsync(ws, 0, zeroed, stream) : cudaSuccess;
}

// The workspace as the kernels take it; what has to start from zero is zeroed, where there is more than one tile.
cudaError_t scan_space(const LinearParams& p, void* workspace, int64_t blocks, cudaStream_t stream, linear::ScanSpace* s) {
    const ScanLayout l = scan_layout(p.T, p.C, p.gate_div != 1 ? p.D : 0);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    s->nt = l.nt;
    s->blocks = static_cast<uint32_t>(blocks);
    s->ticket = reinterpret_cast<uint32_t*>(ws);
    s->flags = reinterpret_cast<uint32_t*>(ws + 256);
    s->pairs = reinterpret_cast<float2*>(ws + l.pairs);
    s->known = reinterpret_cast<float*>(ws + l.known);
    return l.nt > 1 ? cudaMemsetAsync(ws, 0, l.zeroed, stream) : cudaSuccess;
}

}  // namespace

bool encode_rows(CUtensorMap* map, const void* base, int32_t dt, int64_t stride, int64_t C, int64_t T, int width, int tokens) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const CUtensorMapDataType type = dt == GDN_DTYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dt == GDN_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(C), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride * dtype_bytes(dt))};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(tokens)}, es[2] = {1, 1};
    return enc(map, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int multiprocessors() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    return n > 0 ? n : 1;
}

cudaError_t launch_linear_forward(const LinearParams& p, void* workspace, cudaStream_t stream) {
    const bool vec = rows_vector(p) && vector_of_4(p.y, p.y_stride, p.x_dt) && vector_of_4(p.tile_states, 0, GDN_DTYPE_F32);
    if (vec && inputs_wide(p)) {
        int width;
        linear::Segments seg = segments(p, 8, &width);
        const cudaError_t e = segment_space(p, workspace, stream, &seg);
        if (e != cudaSuccess) return e;
        if (p.x_dt == GDN_DTYPE_BF16) return launch_linear_column_forward_bf16(p, seg, width, stream);
        if (p.x_dt == GDN_DTYPE_F16) return launch_linear_column_forward_f16(p, seg, width, stream);
        return launch_linear_column_forward_f32(p, seg, width, stream);
    }
    linear::ScanSpace s{};
    const cudaError_t e = scan_space(p, workspace, (p.C + linear::kCols - 1) / linear::kCols, stream, &s);
    if (e != cudaSuccess) return e;
    if (p.tile_states) s.known = p.tile_states;
    if (p.x_dt == GDN_DTYPE_BF16) return launch_linear_forward_bf16(p, s, vec, stream);
    if (p.x_dt == GDN_DTYPE_F16) return launch_linear_forward_f16(p, s, vec, stream);
    return launch_linear_forward_f32(p, s, vec, stream);
}

cudaError_t launch_linear_backward(const LinearParams& p, void* workspace, cudaStream_t stream) {
    LinearParams q = p;
    const int64_t head_dim = p.gate_div != 1 ? p.D : 0;
    q.scratch = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + scan_layout(p.T, p.C, head_dim).sums);
    bool vec = rows_vector(p) && vector_of_4(p.dy, p.dy_stride, p.x_dt) && vector_of_4(p.dx, p.dx_stride, p.x_dt) &&
               vector_of_4(p.d_final, 0, GDN_DTYPE_F32) && vector_of_4(p.d_initial, 0, GDN_DTYPE_F32);
    if (p.gate_div == 1) vec = vec && vector_of_4(p.da, p.da_stride, p.gate_dt) && vector_of_4(p.db, p.db_stride, p.gate_dt);
    if (vec && inputs_wide(p) && vector_of_16_bytes(p.dy, p.dy_stride, p.x_dt, p.C)) {
        int width;
        linear::Segments seg = segments(p, p.gate_div == 1 && p.gate_dt == GDN_DTYPE_F32 ? 4 : 8, &width);
        if (p.gate_div == 1 || linear::one_head(p, width)) {
            const cudaError_t e = segment_space(p, workspace, stream, &seg);
            if (e != cudaSuccess) return e;
            if (p.x_dt == GDN_DTYPE_BF16) return launch_linear_column_backward_bf16(q, seg, width, stream);
            if (p.x_dt == GDN_DTYPE_F16) return launch_linear_column_backward_f16(q, seg, width, stream);
            return launch_linear_column_backward_f32(q, seg, width, stream);
        }
    }
    linear::ScanSpace s{};
    const cudaError_t e = scan_space(p, workspace, backward_blocks(p.C, head_dim), stream, &s);
    if (e != cudaSuccess) return e;
    if (p.x_dt == GDN_DTYPE_BF16) return launch_linear_backward_bf16(q, s, vec, stream);
    if (p.x_dt == GDN_DTYPE_F16) return launch_linear_backward_f16(q, s, vec, stream);
    return launch_linear_backward_f32(q, s, vec, stream);
}

cudaError_t launch_linear_decode(const LinearParams& p, cudaStream_t stream) {
    gdn_linear_decode_kernel<<<static_cast<unsigned>(static_cast<int64_t>(p.N) * p.H), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
