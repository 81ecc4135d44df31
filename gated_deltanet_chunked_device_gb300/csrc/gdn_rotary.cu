// gdn_rotary.cu -- rotary positions and the write of new keys and values into
// a paged cache (include/gdn_attention.h): one kernel, and its host side.
//
// A warp takes a token: it finds the token's sequence and position, computes
// the token's sines and cosines once for all heads into its own piece of shared
// memory, and turns (or copies) the heads in pieces of 16 bytes.  Where there
// are few tokens several warps share one.  Bound by HBM where there are many
// tokens, by a chain of dependent loads (bounds, sequence, length, page) else.
// 32768 tokens of 48 heads of 128, bf16: 131 us, 0.92 of a measured copy; 33720
// tokens into pages: 127 us, 0.81; 4096 tokens, two warps each (1.7 rounds of
// the warps that are resident): 23.0 us, of which HBM needs 15.  One width of pieces serves all of a call: turned channels
// that are no multiples of 16 bytes make narrow copies of the values, too.
#include <type_traits>

#include "gdn_attention.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// Blocks an SM: what counts is how many warps have their copies under way (48 heads of 32768 tokens, bf16: 151 us with 2 blocks, 133
// with 3, 131 with 4, which is 0.92 of a measured copy).
constexpr int kResident = 4;
constexpr int64_t kMaxRow = 1 << 20;  // elements of a token's heads

struct RotaryParams {
    const void *q, *k, *v;
    void *q_out, *k_out;           // k_out: not when appending
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    gdn_kv_batch b;                // appending: the whole; else cu_seqlens, num_seqs and total_tokens
    gdn_kv_cache c;
    const double* frequencies;
    const void* positions;
    int32_t positions_i64, append;
    int32_t heads, kv_heads, D, R;
    float sign, magnitude;
    int32_t splits;                // warps a token
    int32_t pair_items, rest_items, v_items;            // of a head: pieces that turn, that pass; pieces of v
    uint32_t pair_magic, rest_magic, v_magic;           // ceil(2^32 / items)
    int32_t q_same, k_same;        // in place: what passes is there already
};

// V elements as they are in memory: 16, 8, 4 or 2 bytes.
template <int kBytes>
struct Raw {
    uint32_t w[(kBytes + 3) / 4];
};
template <int kBytes>
__device__ __forceinline__ Raw<kBytes> load_raw(const void* p) {
    Raw<kBytes> r;
    if constexpr (kBytes == 16) {
        const uint4 v = *static_cast<const uint4*>(p);
        r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
    } else if constexpr (kBytes == 8) {
        const uint2 v = *static_cast<const uint2*>(p);
        r.w[0] = v.x, r.w[1] = v.y;
    } else if constexpr (kBytes == 4) {
        r.w[0] = *static_cast<const uint32_t*>(p);
    } else {
        r.w[0] = *static_cast<const uint16_t*>(p);
    }
    return r;
}
template <int kBytes>
__device__ __forceinline__ void store_raw(void* p, const Raw<kBytes>& r) {
    if constexpr (kBytes == 16)
        *static_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else if constexpr (kBytes == 8)
        *static_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    else if constexpr (kBytes == 4)
        *static_cast<uint32_t*>(p) = r.w[0];
    else
        *static_cast<uint16_t*>(p) = static_cast<uint16_t>(r.w[0]);
}

// Element i of a raw piece, widened; and the pair (lo, hi) or single element as 32 (16) bits.
template <class E>
__device__ __forceinline__ float element(const uint32_t* w, int i) {
    if constexpr (std::is_same<E, float>::value) return __uint_as_float(w[i]);
    const uint32_t x = i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
    if constexpr (std::is_same<E, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(x)));
    return __uint_as_float(x << 16);
}
template <class E>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same<E, __half>::value)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// V floats as V elements.
template <class E, int V>
__device__ __forceinline__ Raw<V * sizeof(E)> narrow(const float (&x)[V]) {
    Raw<V * sizeof(E)> r;
    if constexpr (std::is_same<E, float>::value) {
#pragma unroll
        for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(x[i]);
    } else if constexpr (V == 1) {
        r.w[0] = narrow2<E>(x[0], 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) r.w[i / 2] = narrow2<E>(x[i], x[i + 1]);
    }
    return r;
}

// n / d for n < 2^20 and d <= 1024, magic = ceil(2^32 / d): the error n (magic d - 2^32) / (2^32 d) stays below 1 / d.
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t magic) { return d == 1 ? n : __umulhi(n, magic); }

// The largest i < N with cu[i] <= t (N >= 1), by the whole warp: 32 candidates a step.
__device__ __forceinline__ int32_t find_sequence(const void* cu, int i64, int32_t N, int64_t t, int lane) {
    int32_t lo = 0, hi = N;
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 31) / 32;
        const int64_t at = lo + static_cast<int64_t>(lane + 1) * step;
        const unsigned vote = __ballot_sync(~0u, at < hi && load_index(cu, i64, at) <= t);
        lo += __popc(vote) * step;
        if (lo >= hi) lo = hi - 1;  // bounds out of order
        hi = min(hi, lo + step);
    }
    return lo;
}

// Turns the pieces of `heads` heads at src.  An item is V pairs: two pieces of V elements, side by side when interleaved, else half
// the turned channels apart.
template <class E, int V, bool kInterleaved>
__device__ __forceinline__ void turn_heads(const E* src, E* dst, int64_t dst_head, int32_t heads, const RotaryParams& p, const float2* cs,
                                           int first, int stride) {
    constexpr int kBytes = V * sizeof(E);
    const uint32_t items = p.pair_items, total = heads * items;
    const int apart = kInterleaved ? V : p.R / 2;
    for (uint32_t i0 = first; i0 < total; i0 += 2 * stride) {
        Raw<kBytes> a[2], b[2];
        uint32_t head[2], r[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t i = i0 + u * stride;
            head[u] = quotient(i, items, p.pair_magic);
            r[u] = (i - head[u] * items) * V;
            if (i < total) {
                const E* s = src + head[u] * p.D + (kInterleaved ? 2 * r[u] : r[u]);
                a[u] = load_raw<kBytes>(s);
                b[u] = load_raw<kBytes>(s + apart);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (i0 + u * stride >= total) continue;
            float x[V], y[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 t = cs[r[u] + j];
                if constexpr (kInterleaved) {
                    const int m = 2 * j;  // elements m and m + 1 of the 2 V
                    const float lo = m < V ? element<E>(a[u].w, m % V) : element<E>(b[u].w, m % V);
                    const float hi = m + 1 < V ? element<E>(a[u].w, (m + 1) % V) : element<E>(b[u].w, (m + 1) % V);
                    const float n0 = fmaf(lo, t.x, -hi * t.y), n1 = fmaf(hi, t.x, lo * t.y);
                    if (m < V) x[m % V] = n0; else y[m % V] = n0;
                    if (m + 1 < V) x[(m + 1) % V] = n1; else y[(m + 1) % V] = n1;
                } else {
                    const float lo = element<E>(a[u].w, j), hi = element<E>(b[u].w, j);
                    x[j] = fmaf(lo, t.x, -hi * t.y);
                    y[j] = fmaf(hi, t.x, lo * t.y);
                }
            }
            E* d = dst + head[u] * dst_head + (kInterleaved ? 2 * r[u] : r[u]);
            store_raw(d, narrow<E, V>(x));
            store_raw(d + apart, narrow<E, V>(y));
        }
    }
}

template <class E, int V>
__device__ __forceinline__ void copy_heads(const E* src, int32_t src_head, E* dst, int64_t dst_head, int32_t heads, uint32_t items,
                                           uint32_t magic, int first, int stride) {
    constexpr int kBytes = V * sizeof(E);
    const uint32_t total = heads * items;
    for (uint32_t i0 = first; i0 < total; i0 += 2 * stride) {
        Raw<kBytes> x[2];
        uint32_t head[2], r[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t i = i0 + u * stride;
            head[u] = quotient(i, items, magic);
            r[u] = (i - head[u] * items) * V;
            if (i < total) x[u] = load_raw<kBytes>(src + head[u] * src_head + r[u]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (i0 + u * stride < total) store_raw(dst + head[u] * dst_head + r[u], x[u]);
    }
}

// The fraction of a turn, in units of 2^-64, that `radians` make: the mantissa times 1 / (2 pi) to 128 bits, of which the exponent picks
// 64.  Off by less than a unit for |radians| < 2^63: 2^-33 of a turn at a position of 2^31.  (In doubles, a rounded 1 / (2 pi) was off
// by 2^-55 of the angle, and a second double for what it lacks took 1.5 us more for 4096 tokens: there are few units for doubles.)
__device__ __forceinline__ uint64_t turns_of(double radians) {
    constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;  // floor(2^128 / (2 pi))
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(radians));
    const int field = static_cast<int>(bits >> 52 & 0x7ff);
    const uint64_t m = (bits & ((1ull << 52) - 1)) | (field ? 1ull << 52 : 0ull);
    const int shift = 64 - ((field ? field : 1) - 1075);  // of the product, whose low 128 bits are a fraction: its bits from `shift` on
    const uint64_t p0 = m * kLow, p1 = __umul64hi(m, kLow) + m * kHigh, p2 = __umul64hi(m, kHigh) + (p1 < m * kHigh);
    uint64_t turn = 0;
    if (shift >= 128)
        turn = shift < 192 ? p2 >> (shift - 128) : 0;
    else if (shift > 64)
        turn = p1 >> (shift - 64) | p2 << (128 - shift);
    else if (shift > 0)
        turn = shift == 64 ? p1 : p0 >> shift | p1 << (64 - shift);
    return bits >> 63 ? 0 - turn : turn;
}

template <class E, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kResident) rotary_kernel(const __grid_constant__ RotaryParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = p.R / 2;
    // Frequencies as turns a token in units of 2^-64 of a turn: a position times that, modulo 2^64, is the angle's fraction of a turn.
    int64_t* turns = reinterpret_cast<int64_t*>(smem);
    float2* cs = reinterpret_cast<float2*>(turns + half) + warp * half;
    for (int i = tid; i < half; i += kThreads) turns[i] = static_cast<int64_t>(turns_of(p.frequencies[i]));
    __syncthreads();
    uint32_t err = 0;
    if (p.b.cu_seqlens && p.b.device_status && blockIdx.x == 0) {
        for (int32_t i = tid; i <= p.b.num_seqs; i += kThreads) {
            const int64_t here = load_index(p.b.cu_seqlens, p.b.cu_i64, i);
            const int64_t last = i ? load_index(p.b.cu_seqlens, p.b.cu_i64, i - 1) : 0;
            if (here < last || here > p.b.total_tokens || (i == 0 && here != 0)) err |= GDN_DEVICE_ERR_CU_SEQLENS;
        }
    }
    const int64_t tasks = p.b.total_tokens * p.splits;
    for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + warp; task < tasks; task += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = task / p.splits;
        const int first = static_cast<int>(task - t * p.splits) * 32 + lane, stride = 32 * p.splits;
        int64_t pos = t;
        E* k_dst = p.append ? nullptr : static_cast<E*>(p.k_out) + t * p.k_out_stride;
        E* v_dst = nullptr;
        if (p.append) {
            int32_t i;
            int64_t j;
            if (p.b.cu_seqlens) {
                i = find_sequence(p.b.cu_seqlens, p.b.cu_i64, p.b.num_seqs, t, lane);
                j = t - load_index(p.b.cu_seqlens, p.b.cu_i64, i);
            } else {
                i = static_cast<int32_t>(t / p.b.tokens_per_seq);
                j = t - static_cast<int64_t>(i) * p.b.tokens_per_seq;
            }
            const KvSpan s = kv_span(p.b, i, err);
            if (j < 0 || j >= s.n) continue;  // padding
            pos = static_cast<int64_t>(s.len) - s.n + j;
            if (s.row < 0) {
                pos = j;
            } else if (pos >= 0 && pos < s.keys) {
                const int32_t page = p.b.table[static_cast<int64_t>(s.row) * p.b.max_pages + pos / p.b.page_tokens];
                if (page < 0 || page >= p.b.n_pages) {
                    err |= GDN_PAGES_ERR_PAGE;
                } else {
                    const int64_t slot = pos % p.b.page_tokens;
                    k_dst = static_cast<E*>(p.c.k) + page * p.c.k_page_stride + slot * p.c.k_token_stride;
                    v_dst = static_cast<E*>(p.c.v) + page * p.c.v_page_stride + slot * p.c.v_token_stride;
                }
            } else {
                err |= GDN_PAGES_ERR_PAGE;
            }
        } else if (p.positions) {
            pos = load_index(p.positions, p.positions_i64, t);
        } else if (p.b.cu_seqlens) {
            const int32_t i = find_sequence(p.b.cu_seqlens, p.b.cu_i64, p.b.num_seqs, t, lane);
            pos = t - load_index(p.b.cu_seqlens, p.b.cu_i64, i);  // rows past the last bound go on counting
        }
        __syncwarp();
        for (int i = lane; i < half; i += 32) {
            // The nearest quarter turn is taken off as an integer, so that what is left (at most an eighth) keeps all bits.
            const uint64_t angle = static_cast<uint64_t>(pos) * static_cast<uint64_t>(turns[i]);
            const uint32_t quarter = static_cast<uint32_t>((angle + (1ull << 61)) >> 62);
            const int64_t left = static_cast<int64_t>(angle - (static_cast<uint64_t>(quarter) << 62));
            float s, c;
            sincospif(__ll2float_rn(left) * 0x1p-63f, &s, &c);
            const float u = quarter & 1 ? c : s, v = quarter & 1 ? s : c;
            const float sine = quarter & 2 ? -u : u;                   // 0: s, 1: c, 2: -s, 3: -c
            const float cosine = (quarter + 1) & 2 ? -v : v;           // 0: c, 1: -s, 2: -c, 3: s
            cs[i] = make_float2(cosine * p.magnitude, sine * p.sign * p.magnitude);
        }
        __syncwarp();
        // q, k, v one after the other through the same code: turned channels, then those that pass (all of v's).
#pragma unroll 1
        for (int part = 0; part < (p.append ? 3 : 2); ++part) {
            const int32_t heads = part == 0 ? p.heads : p.kv_heads;
            const E* src = part == 0   ? static_cast<const E*>(p.q) + t * p.q_stride
                           : part == 1 ? static_cast<const E*>(p.k) + t * p.k_stride
                                       : static_cast<const E*>(p.v) + t * p.v_stride;
            E* dst = part == 0 ? static_cast<E*>(p.q_out) + t * p.q_out_stride : k_dst;
            int64_t dst_head = p.D;
            if (p.append && part > 0) {
                dst = part == 1 ? k_dst : v_dst;
                dst_head = part == 1 ? p.c.k_head_stride : p.c.v_head_stride;
            }
            if (heads == 0 || !dst) continue;
            if (part < 2 && half > 0) turn_heads<E, V, kInterleaved>(src, dst, dst_head, heads, p, cs, first, stride);
            const int pass = part < 2 ? p.R : 0;
            if (part < 2 ? (part == 0 ? p.q_same : p.k_same) || pass == p.D : false) continue;
            copy_heads<E, V>(src + pass, p.D, dst + pass, dst_head, heads, part < 2 ? p.rest_items : p.v_items,
                             part < 2 ? p.rest_magic : p.v_magic, first, stride);
        }
    }
    kv_report(p.b.device_status, err);
}

template <class E, int V>
cudaError_t launch_vec(RotaryParams p, bool interleaved, cudaStream_t stream) {
    const int half = p.R / 2;
    auto magic = [](int32_t n) { return n > 1 ? static_cast<uint32_t>(((1ull << 32) + n - 1) / n) : 0u; };
    p.pair_items = half / V;
    p.rest_items = (p.D - p.R) / V;
    p.v_items = p.D / V;
    p.pair_magic = magic(p.pair_items);
    p.rest_magic = magic(p.rest_items);
    p.v_magic = magic(p.v_items);
    // Warps a token: enough to fill the SMs, no more than there are pieces for.
    const int64_t want = static_cast<int64_t>(kResident) * kWarps * multiprocessors(), most = (static_cast<int64_t>(p.heads + p.kv_heads) * p.v_items + 63) / 64;
    int64_t splits = (want + p.b.total_tokens - 1) / p.b.total_tokens;
    if (splits > most) splits = most;
    p.splits = splits < 1 ? 1 : static_cast<int32_t>(splits);
    const int64_t blocks = (p.b.total_tokens * p.splits + kWarps - 1) / kWarps, resident = static_cast<int64_t>(kResident) * multiprocessors();
    const size_t smem = half * (sizeof(int64_t) + kWarps * sizeof(float2));  // at most 36 KB
    const int grid = static_cast<int>(blocks < resident ? blocks : resident);
    if (interleaved)
        rotary_kernel<E, V, true><<<grid, kThreads, smem, stream>>>(p);
    else
        rotary_kernel<E, V, false><<<grid, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <class E>
cudaError_t launch_typed(const RotaryParams& p, bool interleaved, int vec, cudaStream_t stream) {
    if constexpr (sizeof(E) == 2)
        if (vec == 8) return launch_vec<E, 8>(p, interleaved, stream);
    if (vec >= 4) return launch_vec<E, 4>(p, interleaved, stream);
    if (vec == 2) return launch_vec<E, 2>(p, interleaved, stream);
    return launch_vec<E, 1>(p, interleaved, stream);
}

// The widest piece (elements, at most 16 bytes) that divides every address, stride and part of a head.
int widest(const RotaryParams& p, int size) {
    int vec = 16 / size;
    auto fits = [&](int64_t n) {
        while (n % vec) vec /= 2;
    };
    auto fits_address = [&](const void* a) {
        while (reinterpret_cast<uintptr_t>(a) % (static_cast<uintptr_t>(vec) * size)) vec /= 2;
    };
    fits(p.D);
    fits(p.R / 2);
    if (p.heads) {
        fits(p.q_stride), fits(p.q_out_stride);
        fits_address(p.q), fits_address(p.q_out);
    }
    if (p.kv_heads) {
        fits(p.k_stride), fits_address(p.k);
        if (p.append) {
            fits(p.v_stride), fits_address(p.v), fits_address(p.c.k), fits_address(p.c.v);
            for (int64_t s : {p.c.k_page_stride, p.c.k_token_stride, p.c.k_head_stride, p.c.v_page_stride, p.c.v_token_stride, p.c.v_head_stride})
                fits(s);
        } else {
            fits(p.k_out_stride), fits_address(p.k_out);
        }
    }
    return vec;
}

gdn_status launch(const RotaryParams& p, gdn_dtype dtype, bool interleaved, cudaStream_t stream) {
    if (p.b.total_tokens == 0 || p.heads + p.kv_heads == 0) return GDN_OK;
    const int vec = widest(p, static_cast<int>(dtype_bytes(dtype)));
    const cudaError_t e = dtype == GDN_DTYPE_F32    ? launch_typed<float>(p, interleaved, vec, stream)
                          : dtype == GDN_DTYPE_BF16 ? launch_typed<__nv_bfloat16>(p, interleaved, vec, stream)
                                                    : launch_typed<__half>(p, interleaved, vec, stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool tensor_ok(const void* p, gdn_dtype t, int64_t& stride, int64_t row) {
    if (!p || !aligned(p, dtype_bytes(t))) return false;
    if (stride == 0) stride = row;
    return stride >= row;
}

// Whether rows that are written are apart from others of the call's T tokens (`same`: or are these, in place).
struct Rows {
    const void* at;
    int64_t stride, row;           // elements
};
bool apart(const Rows& out, const Rows& other, bool same, int64_t T, int64_t size) {
    if (T == 0 || out.row == 0 || other.row == 0) return true;
    if (same && out.at == other.at && out.stride == other.stride) return true;
    if (out.stride > (1LL << 56) || other.stride > (1LL << 56)) return false;
    return rows_apart(out.at, out.stride * size, out.row * size, other.at, other.stride * size, other.row * size, T);
}

// What both calls check; fills the tensors and the turn.
gdn_status make_params(const gdn_rotary_args* args, int64_t T, bool append, RotaryParams* out) {
    if (!args) return GDN_ERR_INVALID_ARG;
    const gdn_rotary_args& a = *args;
    if (a.heads < 0 || a.kv_heads < 0 || a.head_dim < 1 || a.rotary_dim < 0 || a.rotary_dim > a.head_dim || a.rotary_dim % 2 || T < 0)
        return GDN_ERR_INVALID_ARG;
    if (a.dtype != GDN_DTYPE_F32 && a.dtype != GDN_DTYPE_BF16 && a.dtype != GDN_DTYPE_F16) return GDN_ERR_UNSUPPORTED;
    if (a.head_dim > GDN_ROTARY_MAX_DIM || static_cast<int64_t>(a.heads) * a.head_dim > kMaxRow ||
        static_cast<int64_t>(a.kv_heads) * a.head_dim > kMaxRow || T > 0x7fffffffLL)
        return GDN_ERR_UNSUPPORTED;
    if (a.rotary_dim && (!a.frequencies || !aligned(a.frequencies, 8))) return GDN_ERR_INVALID_ARG;
    RotaryParams p{};
    p.q = a.q, p.k = a.k, p.q_out = a.q_out, p.k_out = a.k_out;
    p.q_stride = a.q_stride, p.k_stride = a.k_stride, p.q_out_stride = a.q_out_stride, p.k_out_stride = a.k_out_stride;
    const int64_t q_row = static_cast<int64_t>(a.heads) * a.head_dim, k_row = static_cast<int64_t>(a.kv_heads) * a.head_dim;
    if (T > 0 && a.heads && (!tensor_ok(a.q, a.dtype, p.q_stride, q_row) || !tensor_ok(a.q_out, a.dtype, p.q_out_stride, q_row)))
        return GDN_ERR_INVALID_ARG;
    if (T > 0 && a.kv_heads &&
        (!tensor_ok(a.k, a.dtype, p.k_stride, k_row) || (!append && !tensor_ok(a.k_out, a.dtype, p.k_out_stride, k_row))))
        return GDN_ERR_INVALID_ARG;
    // Warps read and write their tokens, and parts of one token, in any order.
    const int64_t size = dtype_bytes(a.dtype);
    const Rows q{p.q, p.q_stride, q_row}, k{p.k, p.k_stride, k_row}, q_out{p.q_out, p.q_out_stride, q_row};
    if (!apart(q_out, q, true, T, size) || !apart(q_out, k, false, T, size)) return GDN_ERR_INVALID_ARG;
    if (!append) {
        const Rows k_out{p.k_out, p.k_out_stride, k_row};
        if (!apart(k_out, k, true, T, size) || !apart(k_out, q, false, T, size) || !apart(k_out, q_out, false, T, size)) return GDN_ERR_INVALID_ARG;
    }
    p.q_same = p.q == p.q_out;
    p.k_same = !append && p.k == p.k_out;
    p.frequencies = a.frequencies;
    p.append = append;
    p.heads = a.heads, p.kv_heads = a.kv_heads, p.D = a.head_dim, p.R = a.rotary_dim;
    p.sign = a.inverse ? -1.f : 1.f;
    p.magnitude = a.magnitude;
    *out = p;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_rotary_run(const gdn_rotary_args* args, const void* positions, int32_t positions_i64, const void* cu_seqlens,
                          int32_t cu_i64, int32_t num_seqs, int64_t total_tokens, void* stream) {
    gdn::RotaryParams p;
    const gdn_status st = gdn::make_params(args, total_tokens, false, &p);
    if (st != GDN_OK) return st;
    if (positions && (cu_seqlens || !gdn::aligned(positions, positions_i64 ? 8 : 4))) return GDN_ERR_INVALID_ARG;
    if (cu_seqlens && (num_seqs < 0 || !gdn::aligned(cu_seqlens, cu_i64 ? 8 : 4))) return GDN_ERR_INVALID_ARG;
    if (cu_seqlens && num_seqs == 0) cu_seqlens = nullptr;  // all rows are past the last bound
    p.positions = positions;
    p.positions_i64 = positions_i64;
    p.b.cu_seqlens = cu_seqlens;
    p.b.cu_i64 = cu_i64;
    p.b.num_seqs = num_seqs;
    p.b.total_tokens = total_tokens;
    return gdn::launch(p, args->dtype, args->interleaved != 0, static_cast<cudaStream_t>(stream));
}

gdn_status gdn_cache_append_run(const gdn_kv_batch* batch, const gdn_kv_cache* cache, const gdn_rotary_args* args, const void* v,
                                int64_t v_stride, void* stream) {
    gdn_status st = gdn::kv_check(batch, cache);
    if (st != GDN_OK) return st;
    gdn::RotaryParams p;
    st = gdn::make_params(args, batch->total_tokens, true, &p);
    if (st != GDN_OK) return st;
    if (args->kv_heads != cache->kv_heads || args->head_dim != cache->head_dim || args->dtype != cache->dtype) return GDN_ERR_INVALID_ARG;
    if (batch->total_tokens == 0 || batch->num_seqs == 0) return GDN_OK;
    if (!gdn::tensor_ok(v, args->dtype, v_stride, static_cast<int64_t>(args->kv_heads) * args->head_dim)) return GDN_ERR_INVALID_ARG;
    const int64_t q_row = static_cast<int64_t>(args->heads) * args->head_dim, v_row = static_cast<int64_t>(args->kv_heads) * args->head_dim;
    if (!gdn::apart(gdn::Rows{p.q_out, p.q_out_stride, q_row}, gdn::Rows{v, v_stride, v_row}, false, batch->total_tokens, gdn::dtype_bytes(args->dtype)))
        return GDN_ERR_INVALID_ARG;
    p.v = v;
    p.v_stride = v_stride;
    p.b = *batch;
    p.c = *cache;
    return gdn::launch(p, args->dtype, args->interleaved != 0, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
