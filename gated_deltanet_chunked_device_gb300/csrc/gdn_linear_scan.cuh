// gdn_linear_scan.cuh -- the gated linear recurrence over tiles that hand
// their states on (include/gdn_linear.h), both directions, for rows that allow
// no copies of 16 bytes and heads that do not fit a column
// (gdn_linear_column.cuh has the others); and pieces that all kernels share.
//
// What bounds it: a tile's life (loads of one or four elements, composing,
// looking back, storing) with two or three tiles an SM, not HBM: 8192 tokens of
// 13 x 100 bf16 channels take 72 us forward and 119 us backward (0.17, 0.18 of a
// measured copy), of 7 x 101 44 and 89 us.
//
// The packed tokens are cut into tiles of 64, whatever the sequences' bounds,
// and the channels into blocks of 128.  A block of 8 warps owns one tile: a
// warp has 8 successive tokens, a lane 4 channels of them, all in registers
// from one round of loads.
//
// Composition: over a stretch of tokens h_out = A h_in + B, with A the product
// of the gates and B the state that the stretch reaches from zero.  Warps
// compose their 8 tokens, 128 threads compose the 8 warps' pairs, and tiles
// hand (A, B) on to the tiles on their right: a tile publishes its pair, looks
// back to the nearest tile whose end state is known, and applies the pairs in
// between to it, in token order.  Its own end state is defined as
// fma(A, h_in, B), and so is each one that it may start from, so where it
// starts does not change a bit of the result.
//
// A sequence's first token resets the state: a stretch that holds one has an
// end state that depends on nothing before it (a selection, not a product with
// zero, so an infinite state never reaches another sequence).
#pragma once

#include "gdn_linear.cuh"

namespace gdn {
namespace linear {

constexpr int kTile = GDN_LINEAR_TILE;
constexpr int kCols = 128;             // channels of a block
constexpr int kWarps = 8;
constexpr int kSegTokens = kTile / kWarps;
constexpr int kThreads = 32 * kWarps;

// Limits of waits, in SM clocks.  For another block (a look-back) about two seconds; within a block, for copies half of that.
// Warps that wait for one that may itself wait for both, in turn, have the most patience: none gives up while what it waits for
// may still come.  What a wait should have brought is NaN once it has run out, for all that depends on it.
constexpr long long kWaitCycles = 4000000000LL;
__host__ __device__ constexpr long long copy_wait(long long wait) { return wait / 2; }
__host__ __device__ constexpr long long hand_wait(long long wait) { return 2 * wait; }
static_assert(hand_wait(kWaitCycles) > kWaitCycles + copy_wait(kWaitCycles), "a hand-over comes after a look-back and a copy");

template <class T>
struct alignas(4 * sizeof(T)) Pack {
    T v[4];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }

__device__ __forceinline__ Pack<float> load_stream(const Pack<float>* p) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
    return {v.x, v.y, v.z, v.w};
}
template <class T>
__device__ __forceinline__ Pack<T> load_stream(const Pack<T>* p) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
    Pack<T> r;
    memcpy(&r, &v, 8);
    return r;
}
__device__ __forceinline__ void store_stream(Pack<float>* p, const Pack<float>& v) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v.v[0], v.v[1], v.v[2], v.v[3]));
}
template <class T>
__device__ __forceinline__ void store_stream(Pack<T>* p, const Pack<T>& v) {
    uint2 r;
    memcpy(&r, &v, 8);
    __stcs(reinterpret_cast<uint2*>(p), r);
}

// A lane's 4 channels of a block: adjacent ones where the rows allow loads of
// 4 elements (kVec), else every 32nd.
template <bool kVec>
__device__ __forceinline__ int lane_col(int lane, int j) {
    return kVec ? lane * 4 + j : lane + 32 * j;
}

template <bool kVec, class T>
__device__ __forceinline__ Pack<T> load4(const T* row, int lane, int cols) {
    if constexpr (kVec) {
        return load_stream(reinterpret_cast<const Pack<T>*>(row) + lane);
    } else {
        Pack<T> r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r.v[j] = row[lane + 32 * j < cols ? lane + 32 * j : 0];
        return r;
    }
}

template <bool kVec, class T>
__device__ __forceinline__ void store4(T* row, int lane, int cols, const float (&v)[4]) {
    Pack<T> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) from_f32(v[j], r.v[j]);
    if constexpr (kVec) {
        store_stream(reinterpret_cast<Pack<T>*>(row) + lane, r);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (lane + 32 * j < cols) row[lane + 32 * j] = r.v[j];
    }
}

template <bool kVec>
__device__ __forceinline__ void put4(float* row, int lane, const float (&v)[4]) {
    if constexpr (kVec)
        *reinterpret_cast<float4*>(row + lane * 4) = make_float4(v[0], v[1], v[2], v[3]);
    else
#pragma unroll
        for (int j = 0; j < 4; ++j) row[lane + 32 * j] = v[j];
}

template <bool kVec>
__device__ __forceinline__ void get4(const float* row, int lane, float (&v)[4]) {
    if constexpr (kVec) {
        const float4 f = *reinterpret_cast<const float4*>(row + lane * 4);
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = row[lane + 32 * j];
    }
}

// 4 channels of a state row at element offset `off` of channel 0 of the block.
template <bool kVec>
__device__ __forceinline__ void state_load(const void* base, int64_t off, int32_t dt, int lane, int cols, float (&v)[4]) {
    if constexpr (kVec) {
        state_load4(base, off + lane * 4, dt, v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = load1(base, off + (lane + 32 * j < cols ? lane + 32 * j : 0), dt);
    }
}

template <bool kVec>
__device__ __forceinline__ void state_store(void* base, int64_t off, int32_t dt, int lane, int cols, const float (&v)[4]) {
    if constexpr (kVec) {
        state_store4(base, off + lane * 4, dt, v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (lane + 32 * j < cols) store1(base, off + lane + 32 * j, dt, v[j]);
    }
}

__device__ __forceinline__ void report(int32_t* status, int32_t bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ int64_t cu_at(const LinearParams& p, int64_t i) {
    return p.cu_seqlens ? load_index(p.cu_seqlens, p.cu_i64, i) : (i == 0 ? 0 : p.T);
}

// The state row of sequence i; -1 (and reported) when its index is out of range.
__device__ __forceinline__ int64_t state_row(const LinearParams& p, int64_t i) {
    if (!p.state_indices) return i;
    const int64_t row = load_index(p.state_indices, p.idx_i64, i);
    if (row >= 0 && row < p.n_pool) return row;
    report(p.status, GDN_DEVICE_ERR_STATE_INDEX_RANGE);
    return -1;
}

// Which of a tile's tokens are the first or the last of a sequence, and of which.
struct TileBounds {
    uint32_t starts[2], ends[2];
    int32_t start_seq[kTile], end_seq[kTile];
};

__device__ __forceinline__ uint32_t mask_byte(const uint32_t (&m)[2], int seg) { return (m[seg / 4] >> (8 * (seg % 4))) & 0xffu; }

// Fills a tile's bounds from cu_seqlens (one warp).  empty(i) is called, by the whole warp, for every empty sequence
// that lies in the tile.  Entries are taken as they are: a malformed cu_seqlens gives wrong bounds, none outside.
template <class Empty>
__device__ __forceinline__ void find_bounds(const LinearParams& p, int64_t t0, int64_t t1, bool last, int lane, TileBounds& b,
                                            Empty empty) {
    // first entry of [0, N] that is not below t0, by 32 probes at a time
    int64_t lo = 0, hi = static_cast<int64_t>(p.N) + 1;
    while (hi > lo) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
        const uint32_t below = __ballot_sync(0xffffffffu, at < hi && cu_at(p, at) < t0);
        if (below == 0) break;
        const int64_t k = 31 - __clz(below);
        const int64_t from = lo + k * step + 1;
        hi = lo + (k + 1) * step < hi ? lo + (k + 1) * step : hi;
        lo = from;
    }
    uint32_t starts[2] = {0, 0}, ends[2] = {0, 0};
    for (;; lo += 32) {
        const int64_t i = lo + lane;
        const int64_t c = i <= p.N ? cu_at(p, i) : t1 + 1;
        const bool in = c >= t0 && c <= t1;
        bool gap = false;
        if (in && i < p.N) {
            const int64_t next = cu_at(p, i + 1);
            if (next > c && c < t1) {
                b.start_seq[c - t0] = static_cast<int32_t>(i);
                starts[(c - t0) / 32] |= 1u << ((c - t0) % 32);
            }
            gap = next == c && (c < t1 || (last && c == t1));
        }
        if (in && i > 0 && c > t0 && cu_at(p, i - 1) < c) {
            b.end_seq[c - 1 - t0] = static_cast<int32_t>(i - 1);
            ends[(c - 1 - t0) / 32] |= 1u << ((c - 1 - t0) % 32);
        }
        for (uint32_t m = __ballot_sync(0xffffffffu, gap); m; m &= m - 1) empty(lo + __ffs(m) - 1);
        if (__any_sync(0xffffffffu, c > t1)) break;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint32_t s = __reduce_or_sync(0xffffffffu, starts[w]), e = __reduce_or_sync(0xffffffffu, ends[w]);
        if (lane == 0) {
            b.starts[w] = s;
            b.ends[w] = e;
        }
    }
}

// A tile's share of the check of cu_seqlens (one warp).
__device__ __forceinline__ void check_bounds(const LinearParams& p, int64_t f, int64_t nt, int lane) {
    if (!p.cu_seqlens) return;
    const int64_t n = static_cast<int64_t>(p.N) + 1, each = (n + nt - 1) / nt;
    const int64_t to = (f + 1) * each < n ? (f + 1) * each : n;
    bool bad = false;
    for (int64_t i = f * each + lane; i < to; i += 32) {
        const int64_t c = cu_at(p, i);
        bad |= i == 0 && c != 0;
        bad |= i < p.N ? cu_at(p, i + 1) < c : c != p.T;
    }
    if (bad) report(p.status, GDN_DEVICE_ERR_CU_SEQLENS);
}

// What tiles, or time segments of columns, hand on, in the workspace.
struct ScanSpace {
    uint32_t* ticket;              // next tile: tiles are taken in order, so whom one waits for has started
    uint32_t* flags;               // [blocks][4 channel quarters of a block][nt] (columns: [blocks][nt]): a pair, then kKnown
    float2* pairs;                 // [nt][C] (A, B)
    int32_t* exponents;            // [nt][C] columns: A is pairs' times 2^this
    float* known;                  // [nt][C] end states in the scan's direction
    int64_t nt;
    uint32_t blocks;
    long long wait_cycles;         // limit of a look-back; the others follow from it
};

constexpr uint32_t kPair = 1, kKnown = 2, kScaledPair = 3;  // a pair; an end state; a pair some of whose exponents are not 0

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Makes a warp's stores to pairs or known visible, and says so.
__device__ __forceinline__ void publish(uint32_t* flag, uint32_t what, int lane) {
    __threadfence();
    __syncwarp();
    if (lane == 0) store_release(flag, what);
}

// h through a tile's tokens.
__device__ __forceinline__ float pass_on(float a, float h, float b) { return h == 0.f ? b : fmaf(a, h, b); }

// A product of any number of gates, m 2^e with |m| in [1/2, 1) (or 0, or not finite): that of a whole time segment may leave
// fp32's range, or fall below it and come back, where no state does.
struct Product {
    float m;
    int e;
};

// (What is not finite has no exponent to speak of, and is not asked for it.)
__device__ __forceinline__ Product times(Product p, float a) {
    int e;
    const float f = frexpf(p.m * a, &e);
    return {f, p.e + e};
}
__device__ __forceinline__ Product times(Product p, Product q) {
    int e;
    const float f = frexpf(p.m * q.m, &e);
    return {f, p.e + q.e + e};
}

// The same product with an exponent of 0 where fp32 holds it without loss, as most do.
__device__ __forceinline__ Product folded(Product p) {
    return isfinite(p.m) && p.e >= -125 && p.e <= 127 ? Product{ldexpf(p.m, p.e), 0} : p;
}

// h through a time segment, fmaf(A, h, b) with one rounding whatever the exponent.
__device__ __forceinline__ float pass_on(Product a, float h, float b) {
    if (a.e == 0 || !isfinite(a.m) || !isfinite(h)) return pass_on(a.m, h, b);
    if (a.e < -300) return b;  // less than half of the least number, for any h
    // the exponents' sum is shared between two factors that both are in range, unless the product is far out of it
    int e;
    const float f = frexpf(h, &e);
    const int sum = min(max(a.e + e, -250), 252), half = sum / 2;
    return fmaf(ldexpf(a.m, half), ldexpf(f, sum - half), b);
}

// h through the pairs of `n` places, the last of which is f - 1, in token order.  kScaled: with their exponents.
template <bool kScaled, class At>
__device__ __forceinline__ float through_pairs(const ScanSpace& s, int64_t f, int n, float h, int C, int c, At at) {
    auto load = [&](int d, float2& ab, int& e) {
        const int64_t i = at(f - 1 - d) * C + c;
        ab = __ldcg(s.pairs + i);
        e = kScaled ? __ldcg(s.exponents + i) : 0;
    };
    auto pass = [&](float2 ab, int e) { h = kScaled ? pass_on(Product{ab.x, e}, h, ab.y) : pass_on(ab.x, h, ab.y); };
    int d = n - 1;
    for (; d >= 3; d -= 4) {
        float2 ab[4];
        int e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) load(d - j, ab[j], e[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) pass(ab[j], e[j]);
    }
    for (; d >= 0; --d) {
        float2 ab;
        int e;
        load(d, ab, e);
        pass(ab, e);
    }
    return h;
}

// The state that enters place `f` of the scan (f >= 1) for channel c, by one warp for 32 channels: from the nearest
// place whose end state is known, through the pairs of the places after it.  Places are numbered in the scan's
// direction; at(f) gives a place's row in pairs and known.  kSegments: places are time segments, with exponents.
// NaN when the wait runs out: handed on, it reaches whatever depends on it, and nobody after waits for long.
template <bool kSegments, class At>
__device__ __forceinline__ float look_back(const LinearParams& p, const ScanSpace& s, const uint32_t* flags, int64_t f, int c, int lane,
                                           At at) {
    const bool on = c < p.C;
    const long long t0 = clock64();
    int dist;
    uint32_t scaled;
    while (true) {
        const int64_t k = f - 1 - lane;
        const uint32_t flag = k >= 0 ? load_acquire(flags + k) : kKnown;
        const uint32_t known = __ballot_sync(0xffffffffu, flag == kKnown), any = __ballot_sync(0xffffffffu, flag != 0);
        scaled = __ballot_sync(0xffffffffu, flag == kScaledPair);
        dist = known ? __ffs(known) - 1 : 32;
        // all nearer places have their pairs
        if (dist < 32 && (~any & ((1u << dist) - 1)) == 0) break;
        if (__any_sync(0xffffffffu, clock64() - t0 > s.wait_cycles)) {
            if (lane == 0) report(p.status, GDN_DEVICE_ERR_TIMEOUT);
            return nanf("");
        }
    }
    __syncwarp();
    if (!on) return 0.f;
    float h = __ldcg(s.known + at(f - 1 - dist) * p.C + c);
    if (kSegments && scaled & ((1u << dist) - 1)) return through_pairs<true>(s, f, dist, h, p.C, c, at);
    return through_pairs<false>(s, f, dist, h, p.C, c, at);
}

struct ForwardSmem {
    TileBounds bounds;
    uint32_t ticket;
    alignas(16) float a[kWarps][kCols];
    alignas(16) float b[kWarps][kCols];
};

template <class X, class G, bool kVec, bool kHead, bool kHasB>
__global__ void __launch_bounds__(kThreads) gdn_linear_forward_kernel(const LinearParams p, const ScanSpace s) {
    __shared__ ForwardSmem sm;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool multi = s.nt > 1;
    uint32_t ticket = blockIdx.x;
    if (multi) {
        if (threadIdx.x == 0) sm.ticket = atomicAdd(s.ticket, 1u);
        __syncthreads();
        ticket = sm.ticket;
    }
    const int64_t f = ticket / s.blocks;
    const uint32_t blk = ticket % s.blocks;
    const int c0 = static_cast<int>(blk) * kCols, cols = min(kCols, p.C - c0);
    const int64_t t0 = f * kTile, t1 = t0 + kTile < p.T ? t0 + kTile : p.T;
    const bool last = f == s.nt - 1;
    const int64_t mine = t0 + warp * kSegTokens;
    const bool on = kVec ? lane * 4 < cols : true;

    // one round of loads
    const X* x = static_cast<const X*>(p.x) + c0;
    const G* ga = static_cast<const G*>(p.a);
    const G* gb = static_cast<const G*>(p.b);
    Pack<X> px[kSegTokens];
    Pack<G> pa[kSegTokens], pb[kSegTokens];
    int head[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = lane_col<kVec>(lane, j);
        head[j] = (c0 + (col < cols ? col : 0)) / p.D;
    }
#pragma unroll
    for (int k = 0; k < kSegTokens; ++k) {
        const int64_t t = mine + k;
        if (t >= t1 || !on) continue;
        px[k] = load4<kVec>(x + t * p.x_stride, lane, cols);
        if constexpr (kHead && kVec) {
            pa[k].v[0] = ga[t * p.a_stride + head[0]];
            if constexpr (kHasB) pb[k].v[0] = gb[t * p.b_stride + head[0]];
        } else if constexpr (kHead) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pa[k].v[j] = ga[t * p.a_stride + head[j]];
                if constexpr (kHasB) pb[k].v[j] = gb[t * p.b_stride + head[j]];
            }
        } else {
            pa[k] = load4<kVec>(ga + t * p.a_stride + c0, lane, cols);
            if constexpr (kHasB) pb[k] = load4<kVec>(gb + t * p.b_stride + c0, lane, cols);
        }
    }
    if (warp == 0) {
        find_bounds(p, t0, t1, last, lane, sm.bounds, [&](int64_t i) {
            // an empty sequence's final state is its initial one
            const int64_t row = state_row(p, i);  // looked at, and reported, whether or not there is anything to copy
            if (row < 0 || !p.output_state || p.output_state == p.initial_state || !on) return;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (p.initial_state) state_load<kVec>(p.initial_state, row * p.state_stride + c0, p.state_dt, lane, cols, v);
            state_store<kVec>(p.output_state, row * p.state_stride + c0, p.state_dt, lane, cols, v);
        });
    } else if (warp == 1 && blk == 0) {
        check_bounds(p, f, s.nt, lane);
    }
    __syncthreads();
    const uint32_t starts = mask_byte(sm.bounds.starts, warp), ends = mask_byte(sm.bounds.ends, warp);

    // compose the warp's tokens; u holds b x, with the initial state's share at a sequence's first token
    float u[kSegTokens][4], A[4] = {1.f, 1.f, 1.f, 1.f}, B[4] = {0.f, 0.f, 0.f, 0.f};
    auto gate = [&](int k, int j) { return to_f32(pa[k].v[kHead && kVec ? 0 : j]); };
#pragma unroll
    for (int k = 0; k < kSegTokens; ++k) {
        const int64_t t = mine + k;
        const bool in = t < t1 && on;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[k][j] = in ? to_f32(px[k].v[j]) : 0.f;
            if constexpr (kHasB)
                if (in) u[k][j] *= to_f32(pb[k].v[kHead && kVec ? 0 : j]);
        }
        if ((starts >> k) & 1) {
            if (p.initial_state && on) {
                const int64_t row = state_row(p, sm.bounds.start_seq[warp * kSegTokens + k]);
                if (row >= 0) {
                    float h0[4];
                    state_load<kVec>(p.initial_state, row * p.state_stride + c0, p.state_dt, lane, cols, h0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) u[k][j] = fmaf(gate(k, j), h0[j], u[k][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) B[j] = u[k][j];
        } else if (in) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                A[j] *= gate(k, j);
                B[j] = fmaf(gate(k, j), B[j], u[k][j]);
            }
        }
    }
    put4<kVec>(sm.a[warp], lane, A);
    put4<kVec>(sm.b[warp], lane, B);
    __syncthreads();

    // compose the warps, join the tiles: a thread a channel
    if (threadIdx.x < kCols) {
        const int col = threadIdx.x, c = c0 + col;
        const uint32_t reset_lo = sm.bounds.starts[0], reset_hi = sm.bounds.starts[1];
        const bool reset = (reset_lo | reset_hi) != 0;
        float h = 0.f;
        if (multi) {
            uint32_t* flags = s.flags + (static_cast<int64_t>(blk) * 4 + warp) * s.nt;
            float ta = 1.f, tb = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (mask_byte(sm.bounds.starts, w)) {
                    tb = sm.b[w][col];
                } else {
                    ta *= sm.a[w][col];
                    tb = fmaf(sm.a[w][col], tb, sm.b[w][col]);
                }
            }
            const bool known = reset || f == 0;
            if (c < p.C) {
                if (known)
                    s.known[f * p.C + c] = tb;
                else if (!last)
                    s.pairs[f * p.C + c] = make_float2(ta, tb);
            }
            if (!last) publish(flags + f, known ? kKnown : kPair, lane);
            if (f > 0 && !(reset_lo & 1)) {
                h = look_back<false>(p, s, flags, f, c, lane, [](int64_t k) { return k; });
                if (!known) {
                    if (c < p.C) s.known[f * p.C + c] = pass_on(ta, h, tb);
                    if (!last) publish(flags + f, kKnown, lane);
                }
            }
        }
        // the state that enters each warp's tokens
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float a = sm.a[w][col], b = sm.b[w][col];
            sm.a[w][col] = h;
            h = mask_byte(sm.bounds.starts, w) ? b : fmaf(a, h, b);
        }
        if (!multi && p.tile_states && c < p.C && p.T > 0) p.tile_states[c] = h;
    }
    __syncthreads();

    // the tokens once more, from their true state
    float h[4];
    get4<kVec>(sm.a[warp], lane, h);
    X* y = static_cast<X*>(p.y) + c0;
#pragma unroll
    for (int k = 0; k < kSegTokens; ++k) {
        const int64_t t = mine + k;
        if (t >= t1 || !on) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = (starts >> k) & 1 ? u[k][j] : fmaf(gate(k, j), h[j], u[k][j]);
        store4<kVec>(y + t * p.y_stride, lane, cols, h);
        if (((ends >> k) & 1) && p.output_state) {
            const int64_t row = state_row(p, sm.bounds.end_seq[warp * kSegTokens + k]);
            if (row >= 0) state_store<kVec>(p.output_state, row * p.state_stride + c0, p.state_dt, lane, cols, h);
        }
    }
}

// The channels of block `blk` of the backward pass.  With gates per head a block keeps to whole heads, or to a piece of
// one that is wider than a block, so that a head's sums are made in one place or in few.
__device__ __forceinline__ void backward_block(const LinearParams& p, bool head, uint32_t blk, int& c0, int& cols, int& piece) {
    piece = 0;
    if (!head) {
        c0 = static_cast<int>(blk) * kCols;
        cols = min(kCols, p.C - c0);
    } else if (p.D <= kCols) {
        const int width = kCols / p.D * p.D;
        c0 = static_cast<int>(blk) * width;
        cols = min(width, p.C - c0);
    } else {
        const int pieces = (p.D + kCols - 1) / kCols;
        piece = static_cast<int>(blk) % pieces;
        c0 = static_cast<int>(blk) / pieces * p.D + piece * kCols;
        cols = min(kCols, p.D - piece * kCols);
    }
}

template <bool kVec, bool kHead>
struct BackwardSmem {
    TileBounds bounds;
    uint32_t ticket;
    alignas(16) float a[kWarps][kCols];    // products of the gates
    alignas(16) float h[kWarps][kCols];    // state reached from zero, then the state that enters from the left
    alignas(16) float c[kWarps][kCols];    // carry reached from zero, then the carry that enters from the right
    // sums over a head's channels: a lane's shares of 8 tokens, or a token's 128 channels; da and db
    alignas(16) float red[kHead ? kWarps : 1][2][kHead ? (kVec ? kSegTokens * 33 : kCols) : 1];
};

// The carry goes from right to left: c_t = a_t (dy_t + c_{t+1}).  Tiles are taken from the right, and handed on as in
// the forward pass; the states come from the left, from what the forward pass saved at the tiles' ends.
// Two blocks an SM, although some variants then spill: 119 us for 8192 x 13 x 100 bf16, 134 us with one.
template <class X, class G, bool kVec, bool kHead, bool kHasB>
__global__ void __launch_bounds__(kThreads, 2) gdn_linear_backward_kernel(const LinearParams p, const ScanSpace s) {
    __shared__ BackwardSmem<kVec, kHead> sm;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool multi = s.nt > 1;
    uint32_t ticket = blockIdx.x;
    if (multi) {
        if (threadIdx.x == 0) sm.ticket = atomicAdd(s.ticket, 1u);
        __syncthreads();
        ticket = sm.ticket;
    }
    const int64_t r = ticket / s.blocks, f = s.nt - 1 - r;
    const uint32_t blk = ticket % s.blocks;
    int c0, cols, piece;
    backward_block(p, kHead, blk, c0, cols, piece);
    const int64_t t0 = f * kTile, t1 = t0 + kTile < p.T ? t0 + kTile : p.T;
    const bool last = f == s.nt - 1;
    const int64_t mine = t0 + warp * kSegTokens;
    const bool on = kVec ? lane * 4 < cols : true;

    const X* x = static_cast<const X*>(p.x) + c0;
    const X* dy = static_cast<const X*>(p.dy) + c0;
    const G* ga = static_cast<const G*>(p.a);
    const G* gb = static_cast<const G*>(p.b);
    Pack<X> px[kSegTokens], pdy[kSegTokens];
    Pack<G> pa[kSegTokens], pb[kSegTokens];
    int head[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = lane_col<kVec>(lane, j);
        head[j] = (c0 + (col < cols ? col : 0)) / p.D;
    }
#pragma unroll
    for (int k = 0; k < kSegTokens; ++k) {
        const int64_t t = mine + k;
        if (t >= t1 || !on) continue;
        px[k] = load4<kVec>(x + t * p.x_stride, lane, cols);
        pdy[k] = load4<kVec>(dy + t * p.dy_stride, lane, cols);
        if constexpr (kHead && kVec) {
            pa[k].v[0] = ga[t * p.a_stride + head[0]];
            if constexpr (kHasB) pb[k].v[0] = gb[t * p.b_stride + head[0]];
        } else if constexpr (kHead) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pa[k].v[j] = ga[t * p.a_stride + head[j]];
                if constexpr (kHasB) pb[k].v[j] = gb[t * p.b_stride + head[j]];
            }
        } else {
            pa[k] = load4<kVec>(ga + t * p.a_stride + c0, lane, cols);
            if constexpr (kHasB) pb[k] = load4<kVec>(gb + t * p.b_stride + c0, lane, cols);
        }
    }
    auto gate = [&](int k, int j) { return to_f32(pa[k].v[kHead && kVec ? 0 : j]); };
    auto scale = [&](int k, int j) {
        if constexpr (kHasB)
            return to_f32(pb[k].v[kHead && kVec ? 0 : j]);
        else
            return 1.f;
    };
    if (warp == 0) {
        find_bounds(p, t0, t1, last, lane, sm.bounds, [&](int64_t i) {
            // an empty sequence hands the gradient of its final state on
            if (!p.d_initial || !on) return;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (p.d_final) state_load<kVec>(p.d_final, i * p.C + c0, GDN_DTYPE_F32, lane, cols, v);
            state_store<kVec>(p.d_initial, i * p.C + c0, GDN_DTYPE_F32, lane, cols, v);
        });
    } else if (warp == 1 && blk == 0) {
        check_bounds(p, f, s.nt, lane);
    }
    __syncthreads();
    const uint32_t starts = mask_byte(sm.bounds.starts, warp), ends = mask_byte(sm.bounds.ends, warp);
    auto initial = [&](int k, float(&v)[4]) {
        v[0] = v[1] = v[2] = v[3] = 0.f;
        if (p.initial_state && on)
            state_load<kVec>(p.initial_state, sm.bounds.start_seq[warp * kSegTokens + k] * p.state_stride + c0, p.state_dt, lane, cols,
                             v);
    };
    auto final_gradient = [&](int k, float(&v)[4]) {
        v[0] = v[1] = v[2] = v[3] = 0.f;
        if (p.d_final && on)
            state_load<kVec>(p.d_final, static_cast<int64_t>(sm.bounds.end_seq[warp * kSegTokens + k]) * p.C + c0, GDN_DTYPE_F32, lane,
                             cols, v);
    };

    // compose the warp's tokens, in both directions
    {
        float A[4] = {1.f, 1.f, 1.f, 1.f}, B[4] = {0.f, 0.f, 0.f, 0.f}, E[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kSegTokens; ++k) {
            if (mine + k >= t1 || !on) continue;
            if ((starts >> k) & 1) initial(k, B);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = gate(k, j);
                A[j] *= a;
                B[j] = fmaf(a, B[j], to_f32(px[k].v[j]) * scale(k, j));
            }
        }
#pragma unroll
        for (int k = kSegTokens - 1; k >= 0; --k) {
            if (mine + k >= t1 || !on) continue;
            if ((ends >> k) & 1) final_gradient(k, E);
#pragma unroll
            for (int j = 0; j < 4; ++j) E[j] = gate(k, j) * (to_f32(pdy[k].v[j]) + E[j]);
        }
        put4<kVec>(sm.a[warp], lane, A);
        put4<kVec>(sm.h[warp], lane, B);
        put4<kVec>(sm.c[warp], lane, E);
    }
    __syncthreads();

    if (threadIdx.x < kCols) {
        // the carry, from the right: compose the warps, join the tiles
        const int col = threadIdx.x, c = c0 + col;
        const bool valid = col < cols;
        const bool reset = (sm.bounds.ends[0] | sm.bounds.ends[1]) != 0;
        float carry = 0.f;
        if (multi) {
            uint32_t* flags = s.flags + (static_cast<int64_t>(blk) * 4 + warp) * s.nt;
            float ta = 1.f, tc = 0.f;
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                if (mask_byte(sm.bounds.ends, w)) {
                    tc = sm.c[w][col];
                } else {
                    ta *= sm.a[w][col];
                    tc = fmaf(sm.a[w][col], tc, sm.c[w][col]);
                }
            }
            const bool known = reset || r == 0, first = r == s.nt - 1;
            if (valid && !first) {
                if (known)
                    s.known[f * p.C + c] = tc;
                else
                    s.pairs[f * p.C + c] = make_float2(ta, tc);
            }
            if (!first) publish(flags + r, known ? kKnown : kPair, lane);
            if (r > 0 && !(sm.bounds.ends[1] >> 31)) {
                carry = look_back<false>(p, s, flags, r, valid ? c : p.C, lane, [&](int64_t k) { return s.nt - 1 - k; });
                if (!known && !first) {
                    if (valid) s.known[f * p.C + c] = pass_on(ta, carry, tc);
                    publish(flags + r, kKnown, lane);
                }
            }
        }
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            const float b = sm.c[w][col];
            sm.c[w][col] = carry;
            carry = mask_byte(sm.bounds.ends, w) ? b : fmaf(sm.a[w][col], carry, b);
        }
    } else {
        // the states, from the left
        const int col = threadIdx.x - kCols;
        float h = 0.f;
        if (f > 0 && !(sm.bounds.starts[0] & 1) && col < cols) h = p.tile_states[(f - 1) * p.C + c0 + col];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float b = sm.h[w][col];
            sm.h[w][col] = h;
            h = mask_byte(sm.bounds.starts, w) ? b : fmaf(sm.a[w][col], h, b);
        }
    }
    __syncthreads();

    // the tokens once more: states from the left, then gradients from the right
    float before[kSegTokens][4];
    {
        float h[4];
        get4<kVec>(sm.h[warp], lane, h);
#pragma unroll
        for (int k = 0; k < kSegTokens; ++k) {
            if ((starts >> k) & 1) initial(k, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                before[k][j] = h[j];
                if (mine + k < t1 && on) h[j] = fmaf(gate(k, j), h[j], to_f32(px[k].v[j]) * scale(k, j));
            }
        }
    }
    float carry[4];
    get4<kVec>(sm.c[warp], lane, carry);
    X* dx = static_cast<X*>(p.dx) + c0;
    G* da = static_cast<G*>(p.da);
    G* db = static_cast<G*>(p.db);
    const int heads = kHead ? (cols + p.D - 1) / p.D : 0;      // heads of the block (one, when it has a piece of it)
    const int wide = kHead ? min(p.D, kCols) : 0;              // channels of a head in the block
    const int pieces = kHead ? (p.D + kCols - 1) / kCols : 0;
    // a head's sums over the block's channels, to their place (or to the pieces', summed by another kernel)
    auto store_sums = [&](int64_t t, int hd, float sa, float sb) {
        const int hh = c0 / p.D + hd;
        if (pieces == 1) {
            from_f32(sa, da[t * p.da_stride + hh]);
            if constexpr (kHasB) from_f32(sb, db[t * p.db_stride + hh]);
        } else {
            float* o = p.scratch + ((t * p.H + hh) * pieces + piece) * 2;
            o[0] = sa;
            o[1] = sb;
        }
    };
#pragma unroll
    for (int k = kSegTokens - 1; k >= 0; --k) {
        const int64_t t = mine + k;
        const bool in = t < t1 && on;
        if (((ends >> k) & 1)) final_gradient(k, carry);
        float va[4], vb[4], vx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            va[j] = vb[j] = vx[j] = 0.f;
            if (!in) continue;
            const float g = to_f32(pdy[k].v[j]) + carry[j];
            va[j] = g * before[k][j];
            vb[j] = g * to_f32(px[k].v[j]);
            vx[j] = g * scale(k, j);
            carry[j] = gate(k, j) * g;
        }
        if (in) {
            store4<kVec>(dx + t * p.dx_stride, lane, cols, vx);
            if constexpr (!kHead) {
                store4<kVec>(da + t * p.da_stride + c0, lane, cols, va);
                if constexpr (kHasB) store4<kVec>(db + t * p.db_stride + c0, lane, cols, vb);
            }
            if (((starts >> k) & 1) && p.d_initial)
                state_store<kVec>(p.d_initial, static_cast<int64_t>(sm.bounds.start_seq[warp * kSegTokens + k]) * p.C + c0,
                                  GDN_DTYPE_F32, lane, cols, carry);
        }
        if constexpr (kHead && kVec) {
            sm.red[warp][0][k * 33 + lane] = (va[0] + va[1]) + (va[2] + va[3]);
            sm.red[warp][1][k * 33 + lane] = (vb[0] + vb[1]) + (vb[2] + vb[3]);
        } else if constexpr (kHead) {
            if (heads <= 4) {  // a sum over the warp for each of them
                for (int hd = 0; hd < heads; ++hd) {
                    float sa = 0.f, sb = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int col = lane + 32 * j;
                        const bool of = col < cols && col / wide == hd;
                        sa += of ? va[j] : 0.f;
                        sb += of ? vb[j] : 0.f;
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        sa += __shfl_xor_sync(0xffffffffu, sa, o);
                        sb += __shfl_xor_sync(0xffffffffu, sb, o);
                    }
                    if (lane == 0 && t < t1) store_sums(t, hd, sa, sb);
                }
                continue;
            }
            put4<kVec>(sm.red[warp][0], lane, va);
            put4<kVec>(sm.red[warp][1], lane, vb);
            __syncwarp();
            if (t < t1)
                for (int hd = lane; hd < heads; hd += 32) {
                    float sa = 0.f, sb = 0.f;
                    for (int i = hd * wide; i < min((hd + 1) * wide, cols); ++i) {
                        sa += sm.red[warp][0][i];
                        sb += sm.red[warp][1][i];
                    }
                    store_sums(t, hd, sa, sb);
                }
            __syncwarp();
        }
    }
    if constexpr (kHead && kVec) {
        __syncwarp();
        const int lanes = wide / 4;
        for (int i = lane; i < kSegTokens * heads; i += 32) {
            const int k = i % kSegTokens, hd = i / kSegTokens;
            if (mine + k >= t1) continue;
            float sa = 0.f, sb = 0.f;
            for (int l = hd * lanes; l < min((hd + 1) * lanes, cols / 4); ++l) {
                sa += sm.red[warp][0][k * 33 + l];
                sb += sm.red[warp][1][k * 33 + l];
            }
            store_sums(mine + k, hd, sa, sb);
        }
    }
}

// Joins the pieces' sums of heads wider than a block.
template <class G>
__global__ void gdn_linear_join_kernel(const LinearParams p, int pieces) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= p.T * p.H) return;
    float sa = 0.f, sb = 0.f;
    for (int k = 0; k < pieces; ++k) {
        const float2 v = reinterpret_cast<const float2*>(p.scratch)[i * pieces + k];
        sa += v.x;
        sb += v.y;
    }
    const int64_t t = i / p.H, h = i % p.H;
    from_f32(sa, static_cast<G*>(p.da)[t * p.da_stride + h]);
    if (p.db) from_f32(sb, static_cast<G*>(p.db)[t * p.db_stride + h]);
}

template <class X, class G, bool kVec, bool kHead>
cudaError_t backward_gates(const LinearParams& p, const ScanSpace& s, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(s.nt * s.blocks);
    if (p.b)
        gdn_linear_backward_kernel<X, G, kVec, kHead, true><<<grid, kThreads, 0, stream>>>(p, s);
    else
        gdn_linear_backward_kernel<X, G, kVec, kHead, false><<<grid, kThreads, 0, stream>>>(p, s);
    if (kHead && p.D > kCols && p.T > 0)
        gdn_linear_join_kernel<G><<<static_cast<unsigned>((p.T * p.H + 255) / 256), 256, 0, stream>>>(p, (p.D + kCols - 1) / kCols);
    return cudaGetLastError();
}

template <class X, class G>
cudaError_t backward_typed(const LinearParams& p, const ScanSpace& s, bool vec, cudaStream_t stream) {
    const bool head = p.gate_div != 1;
    if (vec) return head ? backward_gates<X, G, true, true>(p, s, stream) : backward_gates<X, G, true, false>(p, s, stream);
    return head ? backward_gates<X, G, false, true>(p, s, stream) : backward_gates<X, G, false, false>(p, s, stream);
}

template <class X, class G, bool kVec, bool kHead>
cudaError_t forward_gates(const LinearParams& p, const ScanSpace& s, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(s.nt * s.blocks);
    if (p.b)
        gdn_linear_forward_kernel<X, G, kVec, kHead, true><<<grid, kThreads, 0, stream>>>(p, s);
    else
        gdn_linear_forward_kernel<X, G, kVec, kHead, false><<<grid, kThreads, 0, stream>>>(p, s);
    return cudaGetLastError();
}

template <class X, class G>
cudaError_t forward_typed(const LinearParams& p, const ScanSpace& s, bool vec, cudaStream_t stream) {
    const bool head = p.gate_div != 1;
    if (vec) return head ? forward_gates<X, G, true, true>(p, s, stream) : forward_gates<X, G, true, false>(p, s, stream);
    return head ? forward_gates<X, G, false, true>(p, s, stream) : forward_gates<X, G, false, false>(p, s, stream);
}

}  // namespace linear
}  // namespace gdn
