// gdn_attention.cu -- attention over a paged cache (include/gdn_attention.h):
// host side, the kernel on CUDA cores, and the join of units that were cut.
#include <algorithm>
#include <cmath>
#include <cudaTypedefs.h>
#include <type_traits>

#include "gdn_attention_tc.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------------------------------------ CUDA cores
// Every type, head size and layout: 64 rows of a unit against tiles of 64 keys, all of it fp32, one pass with a running maximum
// and sum for each row.  256 threads as 16 x 16: a thread has 4 rows by 4 keys of the scores (keys tx + 16 c) and 4 rows by 4 x kCols
// channels of the result (channels 4 tx + 64 c).  Large calls in fp32 run at 26 TFLOP/s (2048 tokens over 6144, 16 heads on 2 of 128,
// 3250 us; of 112, two blocks an SM: 2445 us), half of what a library's fp32 product reaches; small ones are bound by the latency of a
// block's two or three tiles, single tokens by one warp of eight that works while nothing is fetched (64 sequences of 4096, 16 heads on 2
// of 128: 515 us, of which HBM needs 81).
constexpr int kRows = 64, kKeys = 64, kThreads = 256;

__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

template <class E, int V>
struct alignas(sizeof(E) * V) Vec {
    E e[V];
};

// The lowest n bits, n of any size and sign.
__device__ __forceinline__ uint64_t low_bits64(int64_t n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Floats from row to row in shared memory: an odd multiple of 4, so that 16-byte accesses of eight successive rows fall into different
// banks.
__host__ __device__ inline int row_floats(int D) { return 4 * ((D + 3) / 4 | 1); }

size_t simple_smem(int D) { return sizeof(float) * (3 * kRows * row_floats(D) + kRows * (kKeys + 4)) + kKeys * 2 * sizeof(int64_t); }

// Blocks an SM: two where the shared memory of both (and some 1.5 KB each beside it) fits, which is for heads of up to 124 channels.  A
// kernel is compiled for the number that it runs with.
int simple_resident(int D) { return 2 * (simple_smem(D) + 1536) <= 228 * 1024 ? 2 : 1; }

template <class E, int kVec, int kCols, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) attention_simple_kernel(const __grid_constant__ AttnParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ AttnScan<kThreads> scan;
    __shared__ uint32_t there_s[2];        // the keys of a tile that have a page, a bit a key
    const int D = p.c.head_dim, D4 = (D + 3) / 4 * 4, S = row_floats(D);
    float* q_s = reinterpret_cast<float*>(smem);
    float* k_s = q_s + kRows * S;
    float* v_s = k_s + kKeys * S;
    float* w_s = v_s + kKeys * S;                                          // [kRows][kKeys + 4]
    int64_t* off_s = reinterpret_cast<int64_t*>(w_s + kRows * (kKeys + 4)); // offset of a key's row of k and of v; -1: no page
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int32_t block = blockIdx.x;
    griddep_launch_dependents();  // the join's blocks, which wait for this kernel's end
    if (tid == 0) p.joins[2 * block] = make_int4(0, 0, 0, 0);
    AttnWalk walk;
    walk.begin(attn_start<kThreads>(p, block, gridDim.x, scan));
    AttnPart a;
    uint32_t err = 0;
    const int warp = tid >> 5, lane = tid & 31, pieces = D4 / kVec;  // with kVec = 4, D is a multiple of 4
    while (walk.next(p, a)) {
        const int rows = a.tokens * a.heads;
        __syncthreads();
        for (int r = warp; r < kRows; r += kThreads / 32) {
            const int t = r / a.heads, g = r - t * a.heads;
            const E* q = static_cast<const E*>(p.q) + (a.row0 + t) * p.q_stride + static_cast<int64_t>(a.head0 + g) * D;
            for (int d = lane; d < D4; d += 32) q_s[r * S + d] = r < rows && d < D ? wide(q[d]) : 0.f;
        }
        // each row's keys: [lo, hi)
        int32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t pos = static_cast<int64_t>(a.pos0) + (4 * ty + i) / a.heads;
            hi[i] = p.causal ? static_cast<int32_t>(min(max(pos + 1, int64_t{0}), static_cast<int64_t>(a.keys))) : a.keys;
            lo[i] = p.window ? static_cast<int32_t>(max(pos - p.window + 1, int64_t{0})) : 0;
        }
        float m[4], l[4], acc[4][4 * kCols];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < 4 * kCols; ++c) acc[i][c] = 0.f;
        }
        for (int32_t tile = a.tile0; tile < a.tile1; ++tile) {
            const int64_t key0 = static_cast<int64_t>(tile) * kKeys;
            if (tid < kKeys) {
                const int64_t key = key0 + tid;
                int64_t ko = -1, vo = -1;
                if (key < a.keys) {
                    const int32_t at = static_cast<int32_t>(key) / p.b.page_tokens, slot = static_cast<int32_t>(key) - at * p.b.page_tokens;
                    const int32_t page = p.b.table[static_cast<int64_t>(a.table_row) * p.b.max_pages + at];
                    if (page < 0 || page >= p.b.n_pages) {
                        err |= GDN_PAGES_ERR_PAGE;
                    } else {
                        ko = page * p.c.k_page_stride + slot * p.c.k_token_stride + a.kv_head * p.c.k_head_stride;
                        vo = page * p.c.v_page_stride + slot * p.c.v_token_stride + a.kv_head * p.c.v_head_stride;
                    }
                }
                off_s[2 * tid] = ko;
                off_s[2 * tid + 1] = vo;
                const unsigned there = __ballot_sync(~0u, ko >= 0);
                if (lane == 0) there_s[warp] = there;
            }
            __syncthreads();
            // Keys and values, a warp a row; rows that are not there are zero.
            if constexpr (kVec == 4 && sizeof(E) == 4) {
                for (int r = warp; r < kKeys; r += kThreads / 32) {
                    const int64_t ko = off_s[2 * r], vo = off_s[2 * r + 1];
                    for (int d = 4 * lane; d < D; d += 128) {
                        if (ko >= 0) {
                            cp_async16(k_s + r * S + d, static_cast<const E*>(p.c.k) + ko + d);
                            cp_async16(v_s + r * S + d, static_cast<const E*>(p.c.v) + vo + d);
                        } else {
                            *reinterpret_cast<float4*>(k_s + r * S + d) = *reinterpret_cast<float4*>(v_s + r * S + d) = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
                }
                cp_async_commit();
                cp_async_wait<0>();
            } else {
                for (int d0 = 0; d0 < pieces; d0 += 32) {
                    const int d = (d0 + lane) * kVec;
                    const bool in = d < D;
#pragma unroll 2
                    for (int r0 = warp; r0 < kKeys; r0 += 4 * (kThreads / 32)) {
                        Vec<E, kVec> k[4]{}, v[4]{};
                        bool ok[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int64_t ko = off_s[2 * (r0 + 8 * u)], vo = off_s[2 * (r0 + 8 * u) + 1];
                            ok[u] = in && ko >= 0;
                            if (ok[u]) {
                                k[u] = *reinterpret_cast<const Vec<E, kVec>*>(static_cast<const E*>(p.c.k) + ko + d);
                                v[u] = *reinterpret_cast<const Vec<E, kVec>*>(static_cast<const E*>(p.c.v) + vo + d);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u)
#pragma unroll
                            for (int j = 0; j < kVec; ++j)
                                if (d + j < D4) {
                                    k_s[(r0 + 8 * u) * S + d + j] = ok[u] ? wide(k[u].e[j]) : 0.f;
                                    v_s[(r0 + 8 * u) * S + d + j] = ok[u] ? wide(v[u].e[j]) : 0.f;
                                }
                    }
                }
            }
            __syncthreads();
            if (4 * (ty & ~1) < rows) {  // by whole warps: they shuffle
                float s[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[i][c] = 0.f;
#pragma unroll 2
                for (int d = 0; d < D4; d += 4) {
                    float4 x[4], y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(q_s + (4 * ty + i) * S + d);
#pragma unroll
                    for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const float4*>(k_s + (tx + 16 * c) * S + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            s[i][c] = fmaf(x[i].x, y[c].x, s[i][c]);
                            s[i][c] = fmaf(x[i].y, y[c].y, s[i][c]);
                            s[i][c] = fmaf(x[i].z, y[c].z, s[i][c]);
                            s[i][c] = fmaf(x[i].w, y[c].w, s[i][c]);
                        }
                }
                // The keys of the tile that each row sees, a bit a key; rows behind the unit's end see all that is there.
                const uint64_t there = there_s[0] | static_cast<uint64_t>(there_s[1]) << 32;
                uint64_t seen[4];
                bool cut = there != ~0ull;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    seen[i] = there;
                    if (4 * ty + i < rows) seen[i] &= low_bits64(hi[i] - key0) & ~low_bits64(lo[i] - key0);
                    cut |= seen[i] != ~0ull;
                }
                cut = __any_sync(~0u, cut);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[i][c] = !cut || seen[i] >> (tx + 16 * c) & 1 ? s[i][c] * p.scale_log2 : -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float top = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
                    for (int d = 8; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                    const float now = fmaxf(m[i], top), base = now == -INFINITY ? 0.f : now;
                    const float keep = exp2f(m[i] - base);
                    float sum = 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float w = exp2f(s[i][c] - base);
                        sum += w;
                        w_s[(4 * ty + i) * (kKeys + 4) + tx + 16 * c] = w;
                    }
                    m[i] = now;
                    l[i] = l[i] * keep + sum;  // of this thread's keys; the 16 threads of a row join at the unit's end
#pragma unroll
                    for (int c = 0; c < 4 * kCols; ++c) acc[i][c] *= keep;
                }
                __syncwarp();
                auto values = [&](auto some) {  // some: a hidden key's value is left out, not taken times zero: it may be infinite or NaN
#pragma unroll 2
                    for (int k = 0; k < kKeys; k += 4) {
                        float4 w[4];
                        uint32_t bits[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            w[i] = *reinterpret_cast<const float4*>(w_s + (4 * ty + i) * (kKeys + 4) + k);
                            bits[i] = static_cast<uint32_t>(seen[i] >> k);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int c = 0; c < kCols; ++c) {
                                if (4 * tx + 64 * c >= D4) break;
                                const float4 v = *reinterpret_cast<const float4*>(v_s + (k + j) * S + 4 * tx + 64 * c);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float u = j == 0 ? w[i].x : j == 1 ? w[i].y : j == 2 ? w[i].z : w[i].w;
                                    if (!some.value || bits[i] >> j & 1) {
                                        acc[i][4 * c] = fmaf(u, v.x, acc[i][4 * c]);
                                        acc[i][4 * c + 1] = fmaf(u, v.y, acc[i][4 * c + 1]);
                                        acc[i][4 * c + 2] = fmaf(u, v.z, acc[i][4 * c + 2]);
                                        acc[i][4 * c + 3] = fmaf(u, v.w, acc[i][4 * c + 3]);
                                    }
                                }
                            }
                    }
                };
                if (cut)
                    values(std::true_type());
                else
                    values(std::false_type());
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 8; d; d /= 2) l[i] += __shfl_xor_sync(~0u, l[i], d);
        const bool whole = a.tile0 == a.first && a.tile1 == a.last;
        const int32_t slot = attn_slot(a, block);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            if (r >= rows) continue;
            const int t = r / a.heads, g = r - t * a.heads;
            if (whole) {
                E* o = static_cast<E*>(p.o) + (a.row0 + t) * p.o_stride + static_cast<int64_t>(a.head0 + g) * D;
                const float by = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
                for (int c = 0; c < 4 * kCols; ++c) {
                    const int d = 4 * tx + 64 * (c / 4) + c % 4;
                    if (d < D) put(o + d, acc[i][c] * by);
                }
                if (p.lse && tx == 0)
                    p.lse[(a.row0 + t) * p.heads + a.head0 + g] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
            } else {
                const int64_t at = static_cast<int64_t>(slot) * (p.unit_tokens * p.group) + r;
#pragma unroll
                for (int c = 0; c < 4 * kCols; ++c) {
                    const int d = 4 * tx + 64 * (c / 4) + c % 4;
                    if (d < D) p.part_o[at * D + d] = acc[i][c];
                }
                if (tx == 0) p.part_ml[at] = make_float2(m[i], l[i]);
            }
        }
        if (tid == 0 && a.tile0 == a.first && a.tile1 < a.last) attn_note_join(p, a, block, walk.at.share);
    }
    kv_report(p.b.device_status, err);
}

template <class E, int kVec, int kCols, int kBlocks>
cudaError_t launch_simple(const AttnParams& p, int32_t blocks, cudaStream_t stream) {
    const size_t smem = simple_smem(p.c.head_dim);
    auto kernel = attention_simple_kernel<E, kVec, kCols, kBlocks>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    kernel<<<blocks, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <class E>
cudaError_t launch_simple_typed(const AttnParams& p, int32_t blocks, cudaStream_t stream) {
    const int64_t strides[] = {p.c.k_page_stride, p.c.k_token_stride, p.c.k_head_stride,
                               p.c.v_page_stride, p.c.v_token_stride, p.c.v_head_stride, p.c.head_dim};
    bool vec = reinterpret_cast<uintptr_t>(p.c.k) % (4 * sizeof(E)) == 0 && reinterpret_cast<uintptr_t>(p.c.v) % (4 * sizeof(E)) == 0;
    for (int64_t s : strides) vec = vec && s % 4 == 0;
    const int D = p.c.head_dim;
    if (D <= 64) return vec ? launch_simple<E, 4, 1, 2>(p, blocks, stream) : launch_simple<E, 1, 1, 2>(p, blocks, stream);
    if (simple_resident(D) == 2) return vec ? launch_simple<E, 4, 2, 2>(p, blocks, stream) : launch_simple<E, 1, 2, 2>(p, blocks, stream);
    if (D <= 128) return vec ? launch_simple<E, 4, 2, 1>(p, blocks, stream) : launch_simple<E, 1, 2, 1>(p, blocks, stream);
    return vec ? launch_simple<E, 4, 4, 1>(p, blocks, stream) : launch_simple<E, 1, 4, 1>(p, blocks, stream);
}

// ------------------------------------------------------------------------------------------------ the join
// A warp a row: the parts' results, each with its own maximum, weighted to the largest one, in the parts' order.
// Bound by latency: its blocks are launched ahead and wait, and those without a cut unit leave at once.
constexpr int kJoinWarps = 8;

template <class E>
__global__ void __launch_bounds__(32 * kJoinWarps) attention_join_kernel(const __grid_constant__ AttnParams p) {
    const int lane = threadIdx.x & 31, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), block = blockIdx.x;
    griddep_wait();
    const int4 head = p.joins[2 * block];
    if (head.x == 0 || r >= head.y * head.w) return;
    const int4 first = p.joins[2 * block + 1];
    const int64_t row0 = (static_cast<int64_t>(first.y) << 32) | static_cast<uint32_t>(first.x);
    const int parts = head.x, D = p.c.head_dim;
    const int64_t rows = p.unit_tokens * p.group;
    // the unit's first part is in this block's odd slot, the others in the even ones of the blocks after it
    auto place = [&](int k) { return (k == 0 ? 2 * static_cast<int64_t>(block) + 1 : 2 * (static_cast<int64_t>(block) + k)) * rows + r; };
    float top = -INFINITY;
    for (int k = lane; k < parts; k += 32) top = fmaxf(top, p.part_ml[place(k)].x);
    for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = 0.f;
    for (int k0 = 0; k0 < parts; k0 += 32) {
        // 32 parts' weights at a time, a lane each; their sums of values eight loads ahead
        const float2 ml = k0 + lane < parts ? p.part_ml[place(k0 + lane)] : make_float2(-INFINITY, 0.f);
        const float mine = exp2f(ml.x - base);
        float more = ml.y * mine;
        for (int d = 16; d; d /= 2) more += __shfl_xor_sync(~0u, more, d);
        sum += more;
        const int some = min(32, parts - k0);
        for (int k1 = 0; k1 < some; k1 += 4) {
            float x[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    x[k][c] = k1 + k < some && lane + 32 * c < D ? p.part_o[place(k0 + k1 + k) * D + lane + 32 * c] : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float by = __shfl_sync(~0u, mine, (k1 + k) & 31);
                if (k1 + k < some && by != 0.f)  // a part that sees nothing adds nothing
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc[c] = fmaf(x[k][c], by, acc[c]);
            }
        }
    }
    const int t = r / head.w, g = r - t * head.w;
    E* o = static_cast<E*>(p.o) + (row0 + t) * p.o_stride + static_cast<int64_t>(head.z + g) * D;
    const float by = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int d = lane + 32 * c;
        if (d < D) put(o + d, acc[c] * by);
    }
    if (p.lse && lane == 0)
        p.lse[(row0 + t) * p.heads + head.z + g] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------------------------------------ host side
constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Pages, tokens and heads of rows of D elements that do not overlap: from the smallest stride on, each has to pass the span of the
// smaller ones.
bool apart(int64_t pages, int64_t page_stride, int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride, int64_t D) {
    int64_t n[3] = {pages, tokens, heads}, s[3] = {page_stride, token_stride, head_stride};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                int64_t t = s[i];
                s[i] = s[j], s[j] = t;
                t = n[i];
                n[i] = n[j], n[j] = t;
            }
    int64_t span = D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < span) return false;
        int64_t more;
        if (__builtin_mul_overflow(n[i] - 1, s[i], &more) || __builtin_add_overflow(span, more, &span) || span > (1LL << 56)) return false;
    }
    return true;
}

struct Route {
    AttnParams p;
    attn_tc::TcParams tc;          // streams > 0
    int32_t blocks, rows;
    int32_t streams;               // row tiles of the tensor core kernel; 0: CUDA cores
};

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

// A map of 16-bit elements for boxes of 64 channels, swizzled in rows of 128 bytes; what lies outside reads as zeros.  strides:
// elements of all dimensions but the first.
bool encode(CUtensorMap* map, const void* base, gdn_dtype dtype, int rank, const int64_t* dims, const int64_t* strides, const int32_t* box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t n[4], s[3];
    cuuint32_t b[4], es[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        n[i] = static_cast<cuuint64_t>(dims[i]);
        b[i] = static_cast<cuuint32_t>(box[i]);
        // a dimension of one has no step, and its stride may be anything
        if (i > 0) s[i - 1] = static_cast<cuuint64_t>(dims[i] > 1 ? strides[i - 1] * 2 : (dims[0] + 7) / 8 * 16);
    }
    return enc(map, dtype == GDN_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), n,
               s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether tiled copies can fetch a call's rows: addresses and strides of 16 bytes, below 2^40, pages of boxes of at least 8 tokens
// (the swizzle's period).
bool tiles_fit(const AttnParams& p) {
    const gdn_kv_cache& c = p.c;
    if (p.b.page_tokens % 8 || !aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(p.q, 16))
        return false;
    auto fits = [](int64_t n, int64_t stride) { return n <= 1 || (stride % 8 == 0 && stride < (1LL << 39)); };
    return fits(p.b.n_pages, c.k_page_stride) && fits(p.b.page_tokens, c.k_token_stride) && fits(c.kv_heads, c.k_head_stride) &&
           fits(p.b.n_pages, c.v_page_stride) && fits(p.b.page_tokens, c.v_token_stride) && fits(c.kv_heads, c.v_head_stride) &&
           fits(p.b.total_tokens, p.q_stride) && fits(p.heads, c.head_dim);
}

// The widest piece of 16, 8, 4 or 2 bytes that divides every row, stride and address.
int widest_piece(const AttnParams& p) {
    const gdn_kv_cache& c = p.c;
    int64_t all = 16 | reinterpret_cast<intptr_t>(p.q) | reinterpret_cast<intptr_t>(c.k) | reinterpret_cast<intptr_t>(c.v) | 2 * c.head_dim;
    if (p.b.total_tokens > 1) all |= 2 * p.q_stride;
    if (p.b.n_pages > 1) all |= 2 * (c.k_page_stride | c.v_page_stride);
    if (p.b.page_tokens > 1) all |= 2 * (c.k_token_stride | c.v_token_stride);
    if (c.kv_heads > 1) all |= 2 * (c.k_head_stride | c.v_head_stride);
    return static_cast<int>(all & -all);
}

// Whether the tensor cores take a call.  fp32 would lose its last 13 bits there.  Rows that tiled copies cannot fetch are copied by two
// warps in such pieces, which bounds the kernel; whether that still pays (us, tensor cores and CUDA cores, 16 heads on 2, bf16):
//   64 sequences of 4096 tokens, one new: pieces of 16 bytes, heads of 128: 240 and 710; 104: 248 and 410
//                                                   8 bytes,          100: 377 and 401; 92: 314 and 390; 84: 314 and 383;  60: 248 and 237
//                                                   4 bytes,          202: 955 and 1264; 126: 555 and 742; 122: 554 and 458; 102: 505 and
//                                                                     440; 70: 397 and 368;  62: 342 and 209
//                                                   2 bytes,          101: 4879 and 436; 63: 2102 and 209
//   a prompt's 4096 tokens over as many: 16 bytes, 128: 847 and 8668; 8, 100: 1403 and 6148; 4, 102: 1986 and 6275; 2, 101: 9434 and 6272
// So pieces of 2 bytes, which no asynchronous copy has, are left to the CUDA cores; and of few rows those in pieces of 8 bytes up to 64
// channels, and those in pieces of 4 where two blocks fit an SM.
bool tensor_cores(const AttnParams& p) {
    if (p.c.dtype == GDN_DTYPE_F32 || p.b.n_pages < 1) return false;
    if (tiles_fit(p)) return true;
    const int piece = widest_piece(p);
    const bool many = p.b.total_tokens * p.per_kv > static_cast<int64_t>(p.b.num_seqs) * attn_tc::kRowTile;
    const bool small = piece == 8 ? p.c.head_dim <= 64 : simple_resident(p.c.head_dim) == 2;
    return piece == 16 || (piece >= 4 && (many || !small));
}

// The tensor cores' shape.  Two row tiles a unit pay where a sequence has, on the average, rows for more than one.
void tc_route(Route* r) {
    AttnParams& p = r->p;
    const int D = p.c.head_dim, rows = attn_tc::kRowTile;
    p.pieces = (p.per_kv + rows - 1) / rows;
    p.group = (p.per_kv + p.pieces - 1) / p.pieces;
    r->streams = D <= 128 && p.b.total_tokens * p.per_kv > static_cast<int64_t>(p.b.num_seqs) * rows ? 2 : 1;
    p.tile = 128;
    attn_tc::TcParams& t = r->tc;
    // Up to 32 rows a sequence, on the average: units of 32 rows, each in every quarter.
    t.quarters = r->streams == 1 && p.group <= 32 && p.b.total_tokens * p.per_kv <= 32LL * p.b.num_seqs;
    t.row_tokens = (t.quarters ? 32 : rows) / p.group;
    p.unit_tokens = r->streams * t.row_tokens;
    // What a unit's start and end take, in tiles.  One row tile (us with 1, 2, 3, 4 and 6): 300 sequences of 0 to 2093 tokens, one new, 16
    // heads on 2, heads of 256: 222, 175, 149, 142, 142; 128: 111, 90, 83, 84, 83; 64: 88, 75, 72, 73, 71.  1000 tokens over 2500 beside 63
    // single ones, heads of 256: 140, 132, 129, 128, 134.  Against it: 4 tokens of 64 sequences under a window of 1024: 69, 70, 72, 72, 73.
    p.unit_cost = r->streams == 2 ? 2 : 3;
    t.plain = tiles_fit(p) ? 0 : widest_piece(p);
    t.box_keys = p.tile;
    while (!t.plain && p.b.page_tokens % t.box_keys) t.box_keys /= 2;
    t.boxes = p.tile / t.box_keys;
    // Heads of more than 128 channels run as 256: what lies behind them reads as zeros.
    t.k_steps = D > 128 ? 8 : (D + 15) / 16;
    const bool f16 = p.c.dtype == GDN_DTYPE_F16;
    t.idesc_qk = idesc_16bit_f32(rows, p.tile, false, false, p.scale_log2 < 0.f, f16);
    t.idesc_pv = idesc_16bit_f32(rows, 16 * t.k_steps, false, true, false, f16);
    // Scores of keys that are not seen are -infinity, which has to survive the scaling: zero becomes fp32's smallest number, in which the
    // largest finite score, 2^128, becomes 2^-21.
    t.scale_log2 = fmaxf(fabsf(p.scale_log2), 0x1p-149f);
    t.out_vec = D % 8 == 0 && p.o_stride % 8 == 0 && aligned(p.o, 16);
    t.wait_cycles = attn_tc::kWaitCycles;
    r->blocks = multiprocessors();
    r->rows = p.unit_tokens * p.group;
    t.a = p;
}

cudaError_t launch_tc(const Route& r, cudaStream_t stream) {
    const AttnParams& p = r.p;
    const gdn_kv_cache& c = p.c;
    CUtensorMap maps[3]{};
    const int64_t q_dims[3] = {c.head_dim, p.heads, p.b.total_tokens}, q_strides[2] = {c.head_dim, p.q_stride};
    const int32_t q_box[3] = {64, p.group, r.tc.row_tokens}, kv_box[4] = {64, r.tc.box_keys, 1, 1};
    const int64_t kv_dims[4] = {c.head_dim, p.b.page_tokens, c.kv_heads, p.b.n_pages};
    const int64_t k_strides[3] = {c.k_token_stride, c.k_head_stride, c.k_page_stride}, v_strides[3] = {c.v_token_stride, c.v_head_stride, c.v_page_stride};
    if (!r.tc.plain &&
        (!encode(maps, p.q, c.dtype, 3, q_dims, q_strides, q_box) || !encode(maps + 1, c.k, c.dtype, 4, kv_dims, k_strides, kv_box) ||
         !encode(maps + 2, c.v, c.dtype, 4, kv_dims, v_strides, kv_box)))
        return cudaErrorInvalidValue;
    attn_tc::TcParams t = r.tc;
    t.a = p;
    return c.dtype == GDN_DTYPE_BF16 ? launch_attention_tc_bf16(t, maps, r.streams, r.blocks, stream)
                                     : launch_attention_tc_f16(t, maps, r.streams, r.blocks, stream);
}

gdn_status make_route(const gdn_kv_batch* batch, const gdn_kv_cache* cache, const gdn_attention_args* args, Route* out) {
    const gdn_status st = kv_check(batch, cache);
    if (st != GDN_OK) return st;
    if (!args) return GDN_ERR_INVALID_ARG;
    gdn_attention_args a = *args;
    const gdn_kv_cache& c = *cache;
    if (a.heads < 1 || a.heads % c.kv_heads || a.window < 0 || !std::isfinite(a.scale * kLog2e)) return GDN_ERR_INVALID_ARG;
    if (c.head_dim > GDN_ATTENTION_MAX_DIM || static_cast<int64_t>(a.heads) * c.head_dim > (1 << 20)) return GDN_ERR_UNSUPPORTED;
    const int64_t row = static_cast<int64_t>(a.heads) * c.head_dim;
    if (a.q_stride == 0) a.q_stride = row;
    if (a.output_stride == 0) a.output_stride = row;
    if (batch->total_tokens > 0 && (!a.q || !a.output || !aligned(a.q, dtype_bytes(c.dtype)) || !aligned(a.output, dtype_bytes(c.dtype)) ||
                                    a.q_stride < row || a.output_stride < row))
        return GDN_ERR_INVALID_ARG;
    const int64_t bytes = dtype_bytes(c.dtype);
    if (std::max(a.q_stride, a.output_stride) > (1LL << 56)) return GDN_ERR_INVALID_ARG;
    if (batch->total_tokens > 0 && !rows_apart(a.q, a.q_stride * bytes, row * bytes, a.output, a.output_stride * bytes, row * bytes, batch->total_tokens))
        return GDN_ERR_INVALID_ARG;  // a row may be read again after it is written
    if (!aligned(a.lse, 4)) return GDN_ERR_INVALID_ARG;
    if (a.lse && batch->total_tokens > 0) {
        const int64_t T = batch->total_tokens, lse_row = a.heads * int64_t{4};
        if (!rows_apart(a.lse, lse_row, lse_row, a.q, a.q_stride * bytes, row * bytes, T) ||
            !rows_apart(a.lse, lse_row, lse_row, a.output, a.output_stride * bytes, row * bytes, T))
            return GDN_ERR_INVALID_ARG;
    }
    Route r{};
    AttnParams& p = r.p;
    p.b = *batch;
    p.c = c;
    p.q = a.q;
    p.o = a.output;
    p.lse = a.lse;
    p.q_stride = a.q_stride;
    p.o_stride = a.output_stride;
    p.heads = a.heads;
    p.per_kv = a.heads / c.kv_heads;
    p.causal = a.causal != 0;
    p.window = a.window;
    p.scale_log2 = a.scale * kLog2e;
    p.pieces = (p.per_kv + kRows - 1) / kRows;
    p.group = (p.per_kv + p.pieces - 1) / p.pieces;
    p.unit_tokens = kRows / p.group;
    p.tile = kKeys;
    p.unit_cost = 1;
    p.min_steps = 2;
    r.rows = p.unit_tokens * p.group;
    r.blocks = multiprocessors() * simple_resident(c.head_dim);
    if (tensor_cores(p)) tc_route(&r);
    *out = r;
    return GDN_OK;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

gdn_status kv_check(const gdn_kv_batch* batch, const gdn_kv_cache* cache) {
    if (!batch || !cache) return GDN_ERR_INVALID_ARG;
    const gdn_kv_batch& b = *batch;
    const gdn_kv_cache& c = *cache;
    if (b.num_seqs < 0 || b.total_tokens < 0 || b.max_seqs < 0 || b.max_pages < 0 || b.n_pages < 0 || b.page_tokens < 1)
        return GDN_ERR_INVALID_ARG;
    if (b.total_tokens > GDN_ATTENTION_MAX_TOKENS) return GDN_ERR_UNSUPPORTED;
    if (c.kv_heads < 1 || c.head_dim < 1) return GDN_ERR_INVALID_ARG;
    if (c.dtype != GDN_DTYPE_F32 && c.dtype != GDN_DTYPE_BF16 && c.dtype != GDN_DTYPE_F16) return GDN_ERR_UNSUPPORTED;
    if (!b.cu_seqlens && (b.tokens_per_seq < 1 || static_cast<int64_t>(b.num_seqs) * b.tokens_per_seq != b.total_tokens))
        return GDN_ERR_INVALID_ARG;
    if (!b.seqs && b.num_seqs > b.max_seqs) return GDN_ERR_INVALID_ARG;
    if (b.num_seqs > 0) {
        if (!b.lengths || (!b.table && b.max_pages > 0) || (b.n_pages > 0 && (!c.k || !c.v))) return GDN_ERR_INVALID_ARG;
        if (!aligned(b.lengths, 4) || !aligned(b.table, 4) || !aligned(b.seqs, 4) || !aligned(b.cu_seqlens, b.cu_i64 ? 8 : 4) ||
            !aligned(b.device_status, 4) || !aligned(c.k, dtype_bytes(c.dtype)) || !aligned(c.v, dtype_bytes(c.dtype)))
            return GDN_ERR_INVALID_ARG;
    }
    if (!apart(b.n_pages, c.k_page_stride, b.page_tokens, c.k_token_stride, c.kv_heads, c.k_head_stride, c.head_dim) ||
        !apart(b.n_pages, c.v_page_stride, b.page_tokens, c.v_token_stride, c.kv_heads, c.v_head_stride, c.head_dim))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

size_t attn_workspace(int32_t blocks, int32_t rows, int32_t D) {
    const size_t slots = 2 * static_cast<size_t>(blocks);
    return up(slots * sizeof(int4)) + up(slots * rows * sizeof(float2)) + up(slots * rows * D * sizeof(float));
}

void attn_place(AttnParams* p, void* workspace, int32_t blocks, int32_t rows) {
    const size_t slots = 2 * static_cast<size_t>(blocks);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    p->joins = reinterpret_cast<int4*>(w);
    w += up(slots * sizeof(int4));
    p->part_ml = reinterpret_cast<float2*>(w);
    w += up(slots * rows * sizeof(float2));
    p->part_o = reinterpret_cast<float*>(w);
}

cudaError_t launch_attention_simple(const AttnParams& p, int32_t blocks, cudaStream_t stream) {
    if (p.c.dtype == GDN_DTYPE_F32) return launch_simple_typed<float>(p, blocks, stream);
    if (p.c.dtype == GDN_DTYPE_BF16) return launch_simple_typed<__nv_bfloat16>(p, blocks, stream);
    return launch_simple_typed<__half>(p, blocks, stream);
}

cudaError_t launch_attention_join(const AttnParams& p, int32_t blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks, (p.unit_tokens * p.group + kJoinWarps - 1) / kJoinWarps);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its blocks are there when the parts' kernel ends
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (p.c.dtype == GDN_DTYPE_F32) return cudaLaunchKernelEx(&cfg, attention_join_kernel<float>, p);
    if (p.c.dtype == GDN_DTYPE_BF16) return cudaLaunchKernelEx(&cfg, attention_join_kernel<__nv_bfloat16>, p);
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<__half>, p);
}

}  // namespace gdn

extern "C" {

size_t gdn_attention_workspace(const gdn_kv_batch* batch, const gdn_kv_cache* cache, const gdn_attention_args* args) {
    gdn::Route r;
    if (gdn::make_route(batch, cache, args, &r) != GDN_OK || batch->total_tokens == 0 || batch->num_seqs == 0) return 0;
    return gdn::attn_workspace(r.blocks, r.rows, r.p.c.head_dim);
}

gdn_status gdn_attention_run(const gdn_kv_batch* batch, const gdn_kv_cache* cache, const gdn_attention_args* args, void* workspace,
                             size_t workspace_bytes, void* stream) {
    gdn::Route r;
    const gdn_status st = gdn::make_route(batch, cache, args, &r);
    if (st != GDN_OK) return st;
    if (batch->total_tokens == 0 || batch->num_seqs == 0) return GDN_OK;
    if (!workspace || !gdn::aligned(workspace, 16) || workspace_bytes < gdn::attn_workspace(r.blocks, r.rows, r.p.c.head_dim))
        return GDN_ERR_INVALID_ARG;
    gdn::attn_place(&r.p, workspace, r.blocks, r.rows);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = r.streams ? gdn::launch_tc(r, s) : gdn::launch_attention_simple(r.p, r.blocks, s);
    if (e == cudaSuccess) e = gdn::launch_attention_join(r.p, r.blocks, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
