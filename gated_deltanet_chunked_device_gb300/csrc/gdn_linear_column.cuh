// gdn_linear_column.cuh -- the gated linear recurrence with columns of
// channels streamed along the tokens (include/gdn_linear.h), for rows that can
// be copied 4 elements at a time.  Included by one .cu file for each type of x.
//
// A block owns 32 channels and walks the packed tokens, a stage of some 100
// tokens after the other, with the next stages on their way into a ring in
// shared memory.  The state (forward) or the carry (backward) stays in the
// block from stage to stage, so nothing is handed from block to block, and the
// loads never wait for the recurrence.
//
// In a stage a thread composes S successive tokens of 4 channels (h_out = A
// h_in + B, see gdn_linear_scan.cuh), 4 such runs are composed over a warp's
// lanes, the 8 warps through shared memory; then every thread goes over its
// tokens once more from their true state.
#pragma once

#include "gdn_linear_scan.cuh"
#include "sm103_ptx.cuh"

namespace gdn {
namespace linear {

constexpr int kColWidth = 32;                    // channels of a block
constexpr int kLanesRow = kColWidth / 4;         // lanes that hold one token's channels
constexpr int kRuns = 32 / kLanesRow;            // runs of tokens of a warp
constexpr int kColWarps = 8;                     // and one more, which finds the sequences' bounds
constexpr int kColThreads = 32 * (kColWarps + 1);
constexpr int kRingBytes = 220 * 1024;           // shared memory of the ring, at most

// Tokens of a thread's run: 8, or 4 where an element of a token takes more than 6 bytes of the inputs, so that the
// ring holds four stages or more of either.
__host__ __device__ constexpr int forward_run(int x_bytes, int gate_bytes, bool head, bool has_b) {
    return x_bytes + (head ? 0 : has_b ? 2 * gate_bytes : gate_bytes) > 6 ? 4 : 8;
}

// Two fp32 at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    float2 r;
    memcpy(&r, &d, 8);
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t x, y, z, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    memcpy(&z, &c, 8);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    float2 r;
    memcpy(&r, &d, 8);
    return r;
}

// Four channels.
struct Quad {
    float2 lo, hi;
};
__device__ __forceinline__ Quad mul(Quad a, Quad b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ Quad fma(Quad a, Quad b, Quad c) { return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)}; }
__device__ __forceinline__ Quad all4(float v) { return {{v, v}, {v, v}}; }
__device__ __forceinline__ Quad quad(float4 v) { return {{v.x, v.y}, {v.z, v.w}}; }
__device__ __forceinline__ float4 flat(Quad v) { return make_float4(v.lo.x, v.lo.y, v.hi.x, v.hi.y); }
__device__ __forceinline__ Quad pick(bool c, Quad a, Quad b) {
    return {{c ? a.lo.x : b.lo.x, c ? a.lo.y : b.lo.y}, {c ? a.hi.x : b.hi.x, c ? a.hi.y : b.hi.y}};
}
__device__ __forceinline__ Quad shift_up(Quad v, int lanes) {
    return {{__shfl_up_sync(0xffffffffu, v.lo.x, lanes), __shfl_up_sync(0xffffffffu, v.lo.y, lanes)},
            {__shfl_up_sync(0xffffffffu, v.hi.x, lanes), __shfl_up_sync(0xffffffffu, v.hi.y, lanes)}};
}
template <class T>
__device__ __forceinline__ Quad widen(const Pack<T>& p) {
    return {{to_f32(p.v[0]), to_f32(p.v[1])}, {to_f32(p.v[2]), to_f32(p.v[3])}};
}
__device__ __forceinline__ Quad widen(const Pack<__nv_bfloat16>& p) {
    uint2 w;
    memcpy(&w, &p, 8);
    return {{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u)},
            {__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)}};
}
__device__ __forceinline__ Pack<float> narrow(Quad q, float) { return {q.lo.x, q.lo.y, q.hi.x, q.hi.y}; }
__device__ __forceinline__ Pack<__nv_bfloat16> narrow(Quad q, __nv_bfloat16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(q.lo.x, q.lo.y), b = __floats2bfloat162_rn(q.hi.x, q.hi.y);
    return {a.x, a.y, b.x, b.y};
}
__device__ __forceinline__ Pack<__half> narrow(Quad q, __half) {
    const __half2 a = __floats2half2_rn(q.lo.x, q.lo.y), b = __floats2half2_rn(q.hi.x, q.hi.y);
    return {a.x, a.y, b.x, b.y};
}

// States are read and written where sequences start and end: out of line, to keep them out of the instruction cache.
static __device__ __noinline__ float4 state_quad_load(const void* base, int64_t off, int32_t dt) {
    float v[4];
    state_load4(base, off, dt, v);
    return make_float4(v[0], v[1], v[2], v[3]);
}
static __device__ __noinline__ void state_quad_store(void* base, int64_t off, int32_t dt, float4 q) {
    const float v[4] = {q.x, q.y, q.z, q.w};
    state_store4(base, off, dt, v);
}

template <int kBytes>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A stage of one array in shared memory: rows of 32 channels, S rows a run; runs are padded so that the runs of a warp
// lie in different banks.
template <class T, int S>
struct StageArray {
    static constexpr int kRow = kColWidth * static_cast<int>(sizeof(T));
    static constexpr int kRunBytes = S * kRow + (kRow < 128 ? kRow : 0);
    static constexpr int kBytes = kColWarps * kRuns * kRunBytes;

    // This thread's share of the copy of tokens [t0, t1) (at most a stage); kWide: 16 bytes at a time, else 4 elements.
    template <bool kWide>
    static __device__ __forceinline__ void fetch(uint8_t* stage, const T* base, int64_t stride, int64_t t0, int64_t t1, int cols,
                                                 int tid) {
        constexpr int kChunk = kWide ? 16 : 4 * static_cast<int>(sizeof(T));
        constexpr int kPerRow = kRow / kChunk, kElems = kChunk / static_cast<int>(sizeof(T));
        constexpr int kStep = 32 * kColWarps / kPerRow;  // tokens between a thread's chunks
        const int part = tid % kPerRow;
        if (part * kElems >= cols) return;
        const int tok = tid / kPerRow, n = static_cast<int>(t1 - t0);
        const T* src = base + (t0 + tok) * stride + part * kElems;
        uint8_t* dst = stage + tok / S * kRunBytes + tok % S * kRow + part * kChunk;
        static_assert(kStep % S == 0, "a thread's chunks lie whole runs apart");
        constexpr int kTimes = kColWarps * kRuns * S / kStep;
        if (n == kColWarps * kRuns * S) {
#pragma unroll
            for (int i = 0; i < kTimes; ++i) {
                cp_async<kChunk>(dst + i * (kStep / S) * kRunBytes, src);
                src += kStep * stride;
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kTimes; ++i) {
                if (tok + i * kStep < n) cp_async<kChunk>(dst + i * (kStep / S) * kRunBytes, src);
                src += kStep * stride;
            }
        }
    }

    static __device__ __forceinline__ Pack<T> get(const uint8_t* stage, int run, int k, int l) {
        return *reinterpret_cast<const Pack<T>*>(stage + run * kRunBytes + k * kRow + l * 4 * static_cast<int>(sizeof(T)));
    }
};

// The bounds of a stage's tokens.
template <int kTokens>
struct StageBounds {
    uint32_t starts[kTokens / 32], ends[kTokens / 32];
    uint32_t warps;                // which warps' tokens hold a start
    uint32_t plain;                // which warps' tokens are all there, with neither a start nor an end
    int32_t start_seq[kTokens], end_seq[kTokens];
};

// Fills the bounds of tokens [t0, t1) (one warp); `lo`: an entry of cu_seqlens such that none before it is at or past
// t0.  Returns such an entry for tokens from t1 on.  empty(i) is called by the whole warp for every empty sequence.
template <int kTokens, class Empty>
__device__ __forceinline__ int64_t stage_bounds(const LinearParams& p, int64_t lo, int64_t t0, int64_t t1, bool last, int lane,
                                                StageBounds<kTokens>& b, Empty empty) {
#pragma unroll
    for (int w = 0; w < kTokens / 32; ++w)
        if (lane == 0) b.starts[w] = b.ends[w] = 0;
    __syncwarp();
    int64_t next_lo = lo;
    for (;; lo += 32) {
        const int64_t i = lo + lane;
        const int64_t c = i <= p.N ? cu_at(p, i) : t1 + 1;
        const int64_t next = i < p.N ? cu_at(p, i + 1) : c, prev = i > 0 && i <= p.N ? cu_at(p, i - 1) : c;
        const bool in = c >= t0 && c <= t1 && i <= p.N;
        const bool start = in && c < t1 && next > c, end = in && c > t0 && prev < c;
        const bool gap = in && i < p.N && next == c && (c < t1 || (last && c == t1));
        if (start) {
            b.start_seq[c - t0] = static_cast<int32_t>(i);
            atomicOr(&b.starts[(c - t0) / 32], 1u << ((c - t0) % 32));
        }
        if (end) {
            b.end_seq[c - 1 - t0] = static_cast<int32_t>(i - 1);
            atomicOr(&b.ends[(c - 1 - t0) / 32], 1u << ((c - 1 - t0) % 32));
        }
        next_lo += __popc(__ballot_sync(0xffffffffu, i <= p.N && c < t1));
        for (uint32_t m = __ballot_sync(0xffffffffu, gap); m; m &= m - 1) empty(lo + __ffs(m) - 1);
        if (__any_sync(0xffffffffu, c > t1)) break;
    }
    __syncwarp();
    constexpr int kWarpTokens = kTokens / kColWarps;
    uint32_t s = 0, e = 0;
    if (lane < kColWarps) {
        constexpr uint32_t kMask = kWarpTokens == 32 ? 0xffffffffu : (1u << (kWarpTokens % 32)) - 1u;
        s = (b.starts[lane * kWarpTokens / 32] >> (lane * kWarpTokens % 32)) & kMask;
        e = (b.ends[lane * kWarpTokens / 32] >> (lane * kWarpTokens % 32)) & kMask;
    }
    const uint32_t warps = __ballot_sync(0xffffffffu, s != 0);
    const uint32_t plain = __ballot_sync(0xffffffffu, (s | e) == 0 && t0 + (lane + 1) * kWarpTokens <= t1);
    if (lane == 0) {
        b.warps = warps;
        b.plain = plain;
    }
    return next_lo;
}

// First entry of cu_seqlens[0 .. n) that is not below t0 (n: none), by 32 probes at a time (one warp).
__device__ __forceinline__ int64_t first_entry(const LinearParams& p, int64_t n, int64_t t0, int lane) {
    int64_t lo = 0, hi = n;
    while (hi > lo) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
        const uint32_t below = __ballot_sync(0xffffffffu, at < hi && cu_at(p, at) < t0);
        if (below == 0) break;
        const int64_t k = 31 - __clz(below);
        hi = lo + (k + 1) * step < hi ? lo + (k + 1) * step : hi;
        lo = lo + k * step + 1;
    }
    return lo;
}

// Whether a run (8 bits or fewer of a word) holds one of the bounds.
template <int S>
__device__ __forceinline__ uint32_t run_bits(const uint32_t* words, int run) {
    return (words[run * S / 32] >> (run * S % 32)) & ((S == 32 ? 0u : (1u << S)) - 1u);
}

// Of a warp's runs, which hold a bound: one bit each.
template <int S>
__device__ __forceinline__ uint32_t runs_with(const uint32_t* words, int warp) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) r |= (run_bits<S>(words, warp * kRuns + i) ? 1u : 0u) << i;
    return r;
}

// Whether no bit is set after bit `at`.
template <int kTokens>
__device__ __forceinline__ bool is_last_bit(const uint32_t* words, int at) {
    uint32_t after = at % 32 == 31 ? 0u : words[at / 32] >> (at % 32 + 1);
    for (int w = at / 32 + 1; w < kTokens / 32; ++w) after |= words[w];
    return after == 0;
}

// Time segments of a column, where there are too few columns for the GPU's SMs.  The first one is twice as long as the
// others, which go over their tokens twice: once to learn what they do to a state, and, when the state that enters is
// known, once more (from L2, mostly).
struct Segments {
    ScanSpace space;               // nt = segments; flags [blocks][nt]
    int32_t stages;                // stages of a segment but the first
};

template <class X, class G, bool kHead, bool kHasB>
struct ForwardShape {
    static constexpr int kArrays = kHead ? 0 : (kHasB ? 2 : 1);
    static constexpr int S = forward_run(sizeof(X), sizeof(G), kHead, kHasB);
    static constexpr int kTokens = kColWarps * kRuns * S;
    static constexpr int kStageBytes = StageArray<X, S>::kBytes + kArrays * StageArray<G, S>::kBytes;
    static constexpr int kDepth = kRingBytes / kStageBytes < 4 ? kRingBytes / kStageBytes : 4;
    struct Tables {
        StageBounds<kTokens> bounds[2];
        float2 pairs[kColWarps][kColWidth];
        float enter[kColWidth];
        alignas(16) float kept[kColWidth];  // initial state of the last sequence that starts in the segment
        int64_t kept_at;                    // its first token
        uint32_t ticket;
    };
    static constexpr int kSmem = kDepth * kStageBytes + static_cast<int>(sizeof(Tables));
};

template <class X, class G, bool kWide, bool kHead, bool kHasB>
__global__ void __launch_bounds__(kColThreads, 1) gdn_linear_column_forward_kernel(const LinearParams p, const Segments seg) {
    using Shape = ForwardShape<X, G, kHead, kHasB>;
    using AX = StageArray<X, Shape::S>;
    using AG = StageArray<G, Shape::S>;
    constexpr int S = Shape::S, kTokens = Shape::kTokens, kDepth = Shape::kDepth;
    extern __shared__ __align__(128) uint8_t ring[];
    typename Shape::Tables& sm = *reinterpret_cast<typename Shape::Tables*>(ring + kDepth * Shape::kStageBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / kLanesRow, l = lane % kLanesRow, run = warp * kRuns + sub;
    const ScanSpace& sp = seg.space;
    uint32_t ticket = blockIdx.x;
    if (sp.nt > 1) {
        if (threadIdx.x == 0) sm.ticket = atomicAdd(sp.ticket, 1u);
        __syncthreads();
        ticket = sm.ticket;
    }
    const int64_t part = ticket / sp.blocks;
    const uint32_t blk = ticket % sp.blocks;
    const int c0 = static_cast<int>(blk) * kColWidth, cols = min(kColWidth, p.C - c0);
    const int64_t each = seg.stages * static_cast<int64_t>(kTokens);
    const int64_t from = part == 0 ? 0 : (part + 1) * each, end = part == sp.nt - 1 ? p.T : (part + 2) * each;
    const int stages = static_cast<int>(max(static_cast<int64_t>(1), (end - from + kTokens - 1) / kTokens));
    // A later segment learns what it does to a state in steps 0 .. stages - 1.
    const bool twice = part > 0;
    const int steps = twice ? 2 * stages : stages;
    const bool on = l * 4 < cols;

    const X* x = static_cast<const X*>(p.x) + c0;
    const G* ga = static_cast<const G*>(p.a) + (kHead ? (c0 + (on ? l * 4 : 0)) / p.D : c0);
    const G* gb = kHasB ? static_cast<const G*>(p.b) + (kHead ? (c0 + (on ? l * 4 : 0)) / p.D : c0) : nullptr;
    auto stage_start = [&](int q) { return from + static_cast<int64_t>(q < stages ? q : q - stages) * kTokens; };
    auto fetch = [&](int q) {
        if (q < steps) {
            uint8_t* stage = ring + q % kDepth * Shape::kStageBytes;
            const int64_t t0 = stage_start(q), t1 = min(t0 + kTokens, end);
            AX::template fetch<kWide>(stage, x, p.x_stride, t0, t1, cols, threadIdx.x);
            if constexpr (!kHead) {
                AG::template fetch<kWide>(stage + AX::kBytes, ga, p.a_stride, t0, t1, cols, threadIdx.x);
                if constexpr (kHasB) AG::template fetch<kWide>(stage + AX::kBytes + AG::kBytes, gb, p.b_stride, t0, t1, cols, threadIdx.x);
            }
        }
        cp_async_commit();
    };
    // gates per head: a thread's own, one stage ahead in registers
    G ha[kHead ? S : 1], hb[kHead ? S : 1];
    auto fetch_gates = [&](int q) {
        if constexpr (kHead) {
            if (q >= steps) return;
            const int64_t t = stage_start(q) + run * S;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                if (t + k >= end) continue;
                ha[k] = ga[(t + k) * p.a_stride];
                if constexpr (kHasB) hb[k] = gb[(t + k) * p.b_stride];
            }
        }
    };
    int64_t lo = 0;
    auto bounds = [&](int q) {
        if (q >= steps) return;
        const int64_t t0 = stage_start(q), t1 = min(t0 + kTokens, end);
        if (q == 0 || q == stages) lo = from == 0 ? 0 : first_entry(p, static_cast<int64_t>(p.N) + 1, t0, lane);
        const bool write = q >= steps - stages;
        lo = stage_bounds<kTokens>(p, lo, t0, t1, t1 == p.T, lane, sm.bounds[q & 1], [&](int64_t i) {
            // an empty sequence's final state is its initial one
            if (!write || !p.output_state || p.output_state == p.initial_state) return;
            const int64_t row = state_row(p, i);
            if (row < 0 || lane * 4 >= cols) return;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (p.initial_state) state_load<true>(p.initial_state, row * p.state_stride + c0, p.state_dt, lane, cols, v);
            state_store<true>(p.output_state, row * p.state_stride + c0, p.state_dt, lane, cols, v);
        });
    };

    if (warp < kColWarps) {
        for (int q = 0; q < kDepth - 1; ++q) fetch(q);
        fetch_gates(0);
    } else {
        bounds(0);
        if (blk == 0) check_bounds(p, part, sp.nt, lane);
    }
    if (threadIdx.x == 0) sm.kept_at = -1;
    float carry = 0.f, through = 1.f;  // of channel `lane`: the state (in steps that learn, from zero), the gates' product
    bool reset = false;                // whether a sequence has started
    X* y = static_cast<X*>(p.y) + c0 + l * 4;
    for (int q = 0; q < steps; ++q) {
        cp_async_wait<kDepth - 2>();
        __syncthreads();
        const StageBounds<kTokens>& bd = sm.bounds[q & 1];
        const bool learn = twice && q < stages;
        const int64_t t0 = stage_start(q), t = t0 + run * S;
        const int n = static_cast<int>(min(static_cast<int64_t>(S), max(static_cast<int64_t>(0), end - t)));
        const bool plain = (bd.plain >> (warp % kColWarps)) & 1;
        Quad a[S], u[S], A = all4(1.f), B = all4(0.f), exA, exB;
        uint32_t starts = 0;
        bool before = false;  // whether a sequence starts in the warp's runs before this one
        if (warp == kColWarps) {
            bounds(q + 1);
        } else {
            fetch(q + kDepth - 1);
            const uint8_t* stage = ring + q % kDepth * Shape::kStageBytes;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                u[k] = widen(AX::get(stage, run, k, l));
                if constexpr (kHead) {
                    a[k] = all4(to_f32(ha[k]));
                    if constexpr (kHasB) u[k] = mul(u[k], all4(to_f32(hb[k])));
                } else {
                    a[k] = widen(AG::get(stage + AX::kBytes, run, k, l));
                    if constexpr (kHasB) u[k] = mul(u[k], widen(AG::get(stage + AX::kBytes + AG::kBytes, run, k, l)));
                }
            }
            fetch_gates(q + 1);
            if (plain) {
                A = a[0];
                B = u[0];
#pragma unroll
                for (int k = 1; k < S; ++k) {
                    A = mul(A, a[k]);
                    B = fma(a[k], B, u[k]);
                }
            } else {
                starts = run_bits<S>(bd.starts, run);
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    if (k >= n) {
                        a[k] = all4(1.f);
                        u[k] = all4(0.f);
                    }
                    if ((starts >> k) & 1) {
                        if (p.initial_state && on) {
                            const int64_t row = state_row(p, bd.start_seq[run * S + k]);
                            // With states in place, a later segment may have written the row of a sequence that starts
                            // here by the time of the second pass: the last one to start, if any.  Its state is kept.
                            float4 h0 = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (twice && !learn && t + k == sm.kept_at)
                                h0 = *reinterpret_cast<const float4*>(&sm.kept[l * 4]);
                            else if (row >= 0)
                                h0 = state_quad_load(p.initial_state, row * p.state_stride + c0 + l * 4, p.state_dt);
                            if (learn && is_last_bit<kTokens>(bd.starts, run * S + k)) {
                                *reinterpret_cast<float4*>(&sm.kept[l * 4]) = h0;
                                sm.kept_at = t + k;
                            }
                            if (row >= 0) u[k] = fma(a[k], quad(h0), u[k]);
                        }
                        B = u[k];
                    } else {
                        A = mul(A, a[k]);
                        B = fma(a[k], B, u[k]);
                    }
                }
            }
            // over the warp's runs
            const uint32_t rs = (bd.warps >> warp) & 1 ? runs_with<S>(bd.starts, warp) : 0;
#pragma unroll
            for (int o = 1; o < kRuns; o <<= 1) {
                const bool mine = (rs >> max(0, sub - o + 1)) & ((1u << o) - 1u);
                const Quad oa = shift_up(A, o * kLanesRow), ob = shift_up(B, o * kLanesRow);
                if (sub >= o) {
                    B = pick(mine, B, fma(A, ob, B));
                    A = mul(A, oa);
                }
            }
            exA = shift_up(A, kLanesRow);
            exB = shift_up(B, kLanesRow);
            if (sub == 0) {
                exA = all4(1.f);
                exB = all4(0.f);
            }
            before = (rs & ((1u << sub) - 1u)) != 0;
            if (sub == kRuns - 1) {
                float4* o = reinterpret_cast<float4*>(&sm.pairs[warp][l * 4]);
                o[0] = make_float4(A.lo.x, B.lo.x, A.lo.y, B.lo.y);
                o[1] = make_float4(A.hi.x, B.hi.x, A.hi.y, B.hi.y);
            }
        }
        __syncthreads();
        float enter = carry;
        if (warp < kColWarps) {
#pragma unroll
            for (int w = 0; w < kColWarps; ++w) {
                const float2 ab = sm.pairs[w][lane];
                if (w == warp) enter = carry;
                carry = (bd.warps >> w) & 1 ? ab.y : fmaf(ab.x, carry, ab.y);
                if (learn) through *= ab.x;
            }
            reset |= bd.warps != 0;
        }
        if (learn) {
            if (q < stages - 1) continue;
            if (warp == 0) {  // hand the pair on, get the state that enters
                const int c = c0 + lane;
                uint32_t* flags = sp.flags + static_cast<int64_t>(blk) * sp.nt;
                const bool lastpart = part == sp.nt - 1;
                if (!lastpart) {
                    if (lane < cols) {
                        if (reset)
                            sp.known[part * p.C + c] = carry;
                        else
                            sp.pairs[part * p.C + c] = make_float2(through, carry);
                    }
                    publish(flags + part, reset ? kKnown : kPair, lane);
                }
                const float h = look_back(p, sp, flags, part, lane < cols ? c : p.C, lane, [](int64_t k) { return k; });
                if (!lastpart && !reset) {
                    if (lane < cols) sp.known[part * p.C + c] = fmaf(through, h, carry);
                    publish(flags + part, kKnown, lane);
                }
                sm.enter[lane] = h;
            }
            __syncthreads();
            carry = sm.enter[lane];
            continue;
        }
        if (warp < kColWarps) {
            const Quad e = {{__shfl_sync(0xffffffffu, enter, l * 4), __shfl_sync(0xffffffffu, enter, l * 4 + 1)},
                            {__shfl_sync(0xffffffffu, enter, l * 4 + 2), __shfl_sync(0xffffffffu, enter, l * 4 + 3)}};
            Quad h = pick(before, exB, fma(exA, e, exB));
            if (!on) continue;
            X* out = y + t * p.y_stride;
            if (plain) {
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    h = fma(a[k], h, u[k]);
                    store_stream(reinterpret_cast<Pack<X>*>(out), narrow(h, X{}));
                    out += p.y_stride;
                }
                if (p.tile_states && (t + S) % kTile == 0)
                    *reinterpret_cast<float4*>(p.tile_states + t / kTile * p.C + c0 + l * 4) = flat(h);
            } else {
                const uint32_t ends = run_bits<S>(bd.ends, run);
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    if (k >= n) break;
                    h = pick((starts >> k) & 1, u[k], fma(a[k], h, u[k]));
                    store_stream(reinterpret_cast<Pack<X>*>(out), narrow(h, X{}));
                    out += p.y_stride;
                    if (((ends >> k) & 1) && p.output_state) {
                        const int64_t row = state_row(p, bd.end_seq[run * S + k]);
                        if (row >= 0) state_quad_store(p.output_state, row * p.state_stride + c0 + l * 4, p.state_dt, flat(h));
                    }
                    if (p.tile_states && ((t + k) % kTile == kTile - 1 || t + k == p.T - 1))
                        *reinterpret_cast<float4*>(p.tile_states + (t + k) / kTile * p.C + c0 + l * 4) = flat(h);
                }
            }
        }
    }
    if (part == 0 && sp.nt > 1 && warp == 0) {  // the first segment's end state
        if (lane < cols) sp.known[c0 + lane] = carry;
        publish(sp.flags + static_cast<int64_t>(blk) * sp.nt, kKnown, lane);
    }
}

template <class X, class G, bool kWide, bool kHead, bool kHasB>
cudaError_t launch_column_forward(const LinearParams& p, const Segments& seg, cudaStream_t stream) {
    constexpr int kSmem = ForwardShape<X, G, kHead, kHasB>::kSmem;
    auto kernel = gdn_linear_column_forward_kernel<X, G, kWide, kHead, kHasB>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(seg.space.nt * seg.space.blocks), kColThreads, kSmem, stream>>>(p, seg);
    return cudaGetLastError();
}

template <class X, class G, bool kWide>
cudaError_t column_forward_typed(const LinearParams& p, const Segments& seg, cudaStream_t stream) {
    if (p.gate_div != 1)
        return p.b ? launch_column_forward<X, G, kWide, true, true>(p, seg, stream)
                   : launch_column_forward<X, G, kWide, true, false>(p, seg, stream);
    return p.b ? launch_column_forward<X, G, kWide, false, true>(p, seg, stream)
               : launch_column_forward<X, G, kWide, false, false>(p, seg, stream);
}

}  // namespace linear
}  // namespace gdn
