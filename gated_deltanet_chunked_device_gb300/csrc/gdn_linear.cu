// gdn_linear.cu -- how runs of the gated linear recurrence go
// (include/gdn_linear.h): which kernels, their workspace and maps; and the
// decode step's kernel.
#include <atomic>
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

// One thread per sequence and V adjacent channels: its state stays in registers through the tokens, whose inputs are
// loaded kAhead tokens at a time.
template <class X, class G, int V, int kAhead, bool kHead, bool kHasB>
__global__ void __launch_bounds__(kThreads, kAhead == 1 ? 8 : 6) gdn_linear_decode_kernel(const LinearParams p) {
    const int per_seq = p.C / V;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t i = id <= 0xffffffffLL ? static_cast<uint32_t>(id) / static_cast<uint32_t>(per_seq) : id / per_seq;
    if (i >= p.N) return;
    const int c = static_cast<int>(id - i * per_seq) * V, gc = kHead ? c / p.D : c;
    const X* x = static_cast<const X*>(p.x) + i * p.m * p.x_stride + c;
    const G* a = static_cast<const G*>(p.a) + i * p.m * p.a_stride + gc;
    const G* b = static_cast<const G*>(p.b) + (kHasB ? i * p.m * p.b_stride + gc : 0);
    X* y = static_cast<X*>(p.y) + i * p.m * p.y_stride + c;
    constexpr int GV = kHead ? 1 : V;
    struct alignas(V * sizeof(X) < 16 ? V * sizeof(X) : 16) Values {
        X v[V];
    };
    struct alignas(GV * sizeof(G) < 16 ? GV * sizeof(G) : 16) GateValues {
        G v[GV];
    };
    Values px[kAhead];
    GateValues pa[kAhead], pb[kAhead];
    auto load = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (j0 + j >= p.m) continue;
            px[j] = *reinterpret_cast<const Values*>(x + (j0 + j) * p.x_stride);
            pa[j] = *reinterpret_cast<const GateValues*>(a + (j0 + j) * p.a_stride);
            if constexpr (kHasB) pb[j] = *reinterpret_cast<const GateValues*>(b + (j0 + j) * p.b_stride);
        }
    };
    load(0);
    const int64_t row = linear::state_row(p, i);
    if (row < 0) return;
    const int64_t off = row * p.state_stride + c;
    float h[V] = {};
    if (p.initial_state) {
        if constexpr (V == 1)
            h[0] = load1(p.initial_state, off, p.state_dt);
        else
#pragma unroll
            for (int k = 0; k < V; k += 4) {
                float v[4];
                state_load4(p.initial_state, off + k, p.state_dt, v);
                memcpy(h + k, v, sizeof(v));
            }
    }
    for (int j0 = 0; j0 < p.m; j0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (j0 + j >= p.m) break;
            Values out;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float u = linear::to_f32(px[j].v[k]);
                if constexpr (kHasB) u *= linear::to_f32(pb[j].v[GV == 1 ? 0 : k]);
                h[k] = fmaf(linear::to_f32(pa[j].v[GV == 1 ? 0 : k]), h[k], u);
                linear::from_f32(h[k], out.v[k]);
            }
            *reinterpret_cast<Values*>(y + (j0 + j) * p.y_stride) = out;
        }
        if (kAhead > 1) load(j0 + kAhead);
    }
    if (p.output_state) {
        if constexpr (V == 1)
            store1(p.output_state, off, p.state_dt, h[0]);
        else
#pragma unroll
            for (int k = 0; k < V; k += 4) {
                const float v[4] = {h[k], h[k + 1], h[k + 2], h[k + 3]};
                state_store4(p.output_state, off + k, p.state_dt, v);
            }
    }
}

template <class X, class G, int V, int kAhead>
void decode_gates(const LinearParams& p, unsigned blocks, cudaStream_t stream) {
    if (p.gate_div != 1) {
        if (p.b)
            gdn_linear_decode_kernel<X, G, V, kAhead, true, true><<<blocks, kThreads, 0, stream>>>(p);
        else
            gdn_linear_decode_kernel<X, G, V, kAhead, true, false><<<blocks, kThreads, 0, stream>>>(p);
    } else if (p.b) {
        gdn_linear_decode_kernel<X, G, V, kAhead, false, true><<<blocks, kThreads, 0, stream>>>(p);
    } else {
        gdn_linear_decode_kernel<X, G, V, kAhead, false, false><<<blocks, kThreads, 0, stream>>>(p);
    }
}

// channels: 8 (16-bit inputs), 4 or 1 of a thread.
template <class X, class G>
cudaError_t decode_typed(const LinearParams& p, int channels, cudaStream_t stream) {
    const int64_t threads = static_cast<int64_t>(p.N) * (p.C / channels), n = (threads + kThreads - 1) / kThreads;
    if (n > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned blocks = static_cast<unsigned>(n);
    constexpr int kMost = sizeof(X) == 2 ? 8 : 4;
    if (channels == 8 && p.m == 1)
        decode_gates<X, G, kMost, 1>(p, blocks, stream);
    else if (channels == 8)
        decode_gates<X, G, kMost, 2>(p, blocks, stream);
    else if (channels == 4 && p.m == 1)
        decode_gates<X, G, 4, 1>(p, blocks, stream);
    else if (channels == 4)
        decode_gates<X, G, 4, 2>(p, blocks, stream);
    else
        decode_gates<X, G, 1, 2>(p, blocks, stream);
    return cudaGetLastError();
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

// Width and time segments of the columns, for stages of `warps` warps with runs of `run` tokens.
//   - Columns of 32 channels, where they are blocks for three fifths of the SMs or more: 32768 x 4096 172 us, with columns of
//     16 212 us (rows of 32 bytes).
//   - Fewer columns, but too many for three segments each: columns of 16 (32768 x 2048 107 us, with columns of 32 134 us).
//   - Fewer still: as many time segments as the SMs hold (32768 x 1024 87 us, in one segment 134 us).  With two segments the
//     second pass over the later one would cost what the halves save.
// narrow: columns of 16 whatever the number (backward_route).
linear::Segments segments(const LinearParams& p, int warps, int run, bool narrow, int* width) {
    const int64_t sms = multiprocessors(), blocks32 = (p.C + 31) / 32;
    int64_t segs = sms / blocks32;
    *width = narrow || (5 * blocks32 < 3 * sms && segs < 3) ? 16 : 32;
    linear::Segments s{};
    const int64_t tokens = warps * (128 / *width) * run, n = p.T > 0 ? (p.T + tokens - 1) / tokens : 1;
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

// How a run goes: by columns, or (rows that cannot be copied 16 bytes at a time, heads that do not fit a column) by tiles.
struct Route {
    bool column, vec;
    int width;                 // of the columns
    linear::Segments seg;      // columns
    int64_t tiles, blocks;     // tiles
    ScanLayout layout;
    size_t sums;               // bytes of a head's sums, after the layout
};

void finish_route(const LinearParams& p, Route* r) {
    r->tiles = tiles_of(p.T);
    r->layout = r->column ? scan_layout(r->seg.space.nt, r->seg.space.blocks, p.C, true) : scan_layout(r->tiles, 4 * r->blocks, p.C, false);
}

Route forward_route(const LinearParams& p) {
    Route r{};
    r.vec = rows_vector(p) && vector_of_4(p.y, p.y_stride, p.x_dt) && vector_of_4(p.tile_states, 0, GDN_DTYPE_F32);
    r.column = r.vec && inputs_wide(p);
    if (r.column) r.seg = segments(p, linear::kForwardWarps, 8, false, &r.width);
    r.blocks = (p.C + linear::kCols - 1) / linear::kCols;
    finish_route(p, &r);
    return r;
}

Route backward_route(const LinearParams& p) {
    Route r{};
    const int64_t head_dim = p.gate_div != 1 ? p.D : 0;
    r.vec = rows_vector(p) && vector_of_4(p.dy, p.dy_stride, p.x_dt) && vector_of_4(p.dx, p.dx_stride, p.x_dt) &&
            vector_of_4(p.d_final, 0, GDN_DTYPE_F32) && vector_of_4(p.d_initial, 0, GDN_DTYPE_F32);
    if (p.gate_div == 1) r.vec = r.vec && vector_of_4(p.da, p.da_stride, p.gate_dt) && vector_of_4(p.db, p.db_stride, p.gate_dt);
    if (r.vec && inputs_wide(p) && vector_of_16_bytes(p.dy, p.dy_stride, p.x_dt, p.C)) {
        // Sums of heads of 16, 48, 80 channels fit columns of 16 alone, which have no time segments: taken where the columns
        // are blocks for two fifths of the SMs, or the batch is short (52 heads of 80, 32768 tokens: 329 us, tiles 1238;
        // 64 heads of 16, 4096 tokens: 28, tiles 30; 32 heads of 16, 512 tokens: 8, tiles 15; but 32768 tokens: 184, tiles 122).
        const bool narrow = p.gate_div != 1 && p.D % 32 != 0 && p.D % 16 == 0 &&
                            (5 * ((p.C + 31) / 32) >= multiprocessors() || p.T <= 2048);
        r.seg = segments(p, 8, p.gate_div == 1 && p.gate_dt == GDN_DTYPE_F32 ? 4 : 8, narrow, &r.width);  // backward_run
        r.column = p.gate_div == 1 || linear::one_head(p, r.width);
    }
    r.blocks = backward_blocks(p.C, head_dim);
    r.sums = sums_bytes(p.T, p.C, head_dim, r.column ? r.width : linear::kCols);
    finish_route(p, &r);
    return r;
}

// The workspace as the kernels take it; what has to start from zero is zeroed, where anything is handed on.
cudaError_t scan_space(const Route& r, void* workspace, cudaStream_t stream, linear::ScanSpace* s) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    s->wait_cycles = linear::kWaitCycles;
    if (!r.column) {
        s->nt = r.tiles;
        s->blocks = static_cast<uint32_t>(r.blocks);
    }
    if (r.layout.total == 0) return cudaSuccess;
    s->ticket = reinterpret_cast<uint32_t*>(ws);
    s->flags = reinterpret_cast<uint32_t*>(ws + 256);
    s->pairs = reinterpret_cast<float2*>(ws + r.layout.zeroed);
    s->known = reinterpret_cast<float*>(ws + r.layout.known);
    s->exponents = reinterpret_cast<int32_t*>(ws + r.layout.exponents);
    return cudaMemsetAsync(ws, 0, r.layout.zeroed, stream);
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
    static std::atomic<int> known[64];  // a device's count does not change
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

size_t linear_forward_workspace(const LinearParams& p) { return forward_route(p).layout.total; }

size_t linear_backward_workspace(const LinearParams& p) {
    const Route r = backward_route(p);
    return r.layout.total + r.sums;
}

cudaError_t launch_linear_forward(const LinearParams& p, void* workspace, cudaStream_t stream) {
    Route r = forward_route(p);
    linear::ScanSpace s{};
    const cudaError_t e = scan_space(r, workspace, stream, r.column ? &r.seg.space : &s);
    if (e != cudaSuccess) return e;
    if (r.column) {
        if (p.x_dt == GDN_DTYPE_BF16) return launch_linear_column_forward_bf16(p, r.seg, r.width, stream);
        if (p.x_dt == GDN_DTYPE_F16) return launch_linear_column_forward_f16(p, r.seg, r.width, stream);
        return launch_linear_column_forward_f32(p, r.seg, r.width, stream);
    }
    if (p.tile_states) s.known = p.tile_states;
    if (p.x_dt == GDN_DTYPE_BF16) return launch_linear_forward_bf16(p, s, r.vec, stream);
    if (p.x_dt == GDN_DTYPE_F16) return launch_linear_forward_f16(p, s, r.vec, stream);
    return launch_linear_forward_f32(p, s, r.vec, stream);
}

cudaError_t launch_linear_backward(const LinearParams& p, void* workspace, cudaStream_t stream) {
    Route r = backward_route(p);
    linear::ScanSpace s{};
    const cudaError_t e = scan_space(r, workspace, stream, r.column ? &r.seg.space : &s);
    if (e != cudaSuccess) return e;
    LinearParams q = p;
    if (r.sums > 0) q.scratch = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + r.layout.total);
    if (r.column) {
        if (p.x_dt == GDN_DTYPE_BF16) return launch_linear_column_backward_bf16(q, r.seg, r.width, stream);
        if (p.x_dt == GDN_DTYPE_F16) return launch_linear_column_backward_f16(q, r.seg, r.width, stream);
        return launch_linear_column_backward_f32(q, r.seg, r.width, stream);
    }
    if (p.x_dt == GDN_DTYPE_BF16) return launch_linear_backward_bf16(q, s, r.vec, stream);
    if (p.x_dt == GDN_DTYPE_F16) return launch_linear_backward_f16(q, s, r.vec, stream);
    return launch_linear_backward_f32(q, s, r.vec, stream);
}

cudaError_t launch_linear_decode(const LinearParams& p, cudaStream_t stream) {
    int channels = rows_vector(p) && vector_of_4(p.y, p.y_stride, p.x_dt) ? 4 : 1;
    // Loads of 16 bytes, where that leaves every SM some blocks: with few sequences, more threads with less each are faster
    // (2048 sequences of 4 tokens x 4096 channels: 60 us, 78 us with 4 channels a thread).
    if (channels == 4 && p.x_dt != GDN_DTYPE_F32 && p.C % 8 == 0 && (p.gate_div == 1 || p.D % 8 == 0) && inputs_wide(p) &&
        vector_of_16_bytes(p.y, p.y_stride, p.x_dt, p.C) && static_cast<int64_t>(p.N) * p.C >= 8LL * 4 * kThreads * multiprocessors())
        channels = 8;
    const bool wide_gates = p.gate_dt == GDN_DTYPE_F32;
    if (p.x_dt == GDN_DTYPE_F32) return decode_typed<float, float>(p, channels, stream);
    if (p.x_dt == GDN_DTYPE_BF16)
        return wide_gates ? decode_typed<__nv_bfloat16, float>(p, channels, stream)
                          : decode_typed<__nv_bfloat16, __nv_bfloat16>(p, channels, stream);
    return wide_gates ? decode_typed<__half, float>(p, channels, stream) : decode_typed<__half, __half>(p, channels, stream);
}

}  // namespace gdn
