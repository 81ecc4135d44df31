// gdn_linear_column.cuh -- the gated linear recurrence with columns of
// channels streamed along the tokens (include/gdn_linear.h), for rows that can
// be copied 16 bytes at a time: forward, and what both directions share.
// Included by one .cu file for each type of x.
//
// What bounds it: 3 flops for 6 to 16 bytes, so HBM, if the loads never wait
// for the recurrence.  A block owns 32 (or 16) channels and walks the packed
// tokens; the state stays in it from stage to stage (of 256 tokens, or 512),
// so blocks hand nothing to one another, and the next stages are on their way
// into a ring in shared memory by tiled copies.  With 4096 channels that is 128
// blocks, and they fill HBM: 32768 tokens, bf16, gates per channel 166 us, 6.5
// TB/s, 0.95 of a measured copy; with fp32 gates 239 us, 0.99.
//
// In a stage a thread composes 8 successive tokens of 4 channels (h_out = A
// h_in + B, see gdn_linear_scan.cuh; two channels an instruction), the runs of
// a warp's lanes are composed by shuffles, the warps through shared memory;
// then every thread goes over its tokens once more from their true state.
// Its inputs stay in registers in between: one read of shared memory.  That
// is 430 to 560 instructions a warp and stage.  Where fewer bytes come with an
// element (gates per head: 108 us, 0.74) nothing is full: 52 % of the issue
// slots, no pipe above 33 %, and 24 of the 152 SMs without a block; what is left
// is the latency of a stage's steps.  Hence two groups of 8 warps that take the
// stages in turn, so that one composes while the other stores (145 us with one
// group), and handing the state on through shared memory takes one wait and 8
// fused multiply-adds.
//
// Tried and slower (32768 x 4096, bf16): inputs fetched by the threads
// themselves, 16 bytes each (197 us: the copies' instructions and L1's tags);
// runs of 16 tokens (280 us: too few stages in the ring); a stage's inputs read
// into registers a stage ahead (spills); 9 warps, one for the bounds (168
// registers a thread: spills in the backward pass, up to twice the time).
#pragma once

#include <type_traits>

#include "gdn_linear_scan.cuh"
#include "sm103_ptx.cuh"

namespace gdn {
namespace linear {

// A block's shape: W channels; NG groups of NW warps, which take the stages in turn; runs of R tokens; S: one of several time
// segments (of columns of 32 alone, a lane a channel).  In kernels of their own, since what segments need costs the others
// registers and instruction cache (64 sequences of 512 tokens x 4096: 208 us, in one kernel 235).
template <int W, int NW, int R, int NG, bool S = false>
struct Column {
    static constexpr int kWidth = W, kRun = R, kGroups = NG;
    static constexpr bool kSegments = S;
    static_assert(!S || W == 32, "a lane a channel");
    static constexpr int kLanesRow = W / 4;      // lanes that hold one token's channels
    static constexpr int kRuns = 32 / kLanesRow; // runs of tokens of a warp
    static constexpr int kWarpTokens = kRuns * kRun;
    static constexpr int kTokens = NW * kWarpTokens;
    static constexpr int kWarps = NW;
    static constexpr int kThreads = 32 * NW * NG;
    // Places for what a stage hands to the next one.  A place is written again kHands stages later; by then the group that
    // read it has gone on to another stage, all of it.
    static constexpr int kHands = NG + 2;
};

constexpr int kRingBytes = 192 * 1024;           // shared memory of the ring, at most

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
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
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
__device__ __forceinline__ Quad add(Quad a, Quad b) { return {add2(a.lo, b.lo), add2(a.hi, b.hi)}; }
__device__ __forceinline__ Quad shift_down(Quad v, int lanes) {
    return {{__shfl_down_sync(0xffffffffu, v.lo.x, lanes), __shfl_down_sync(0xffffffffu, v.lo.y, lanes)},
            {__shfl_down_sync(0xffffffffu, v.hi.x, lanes), __shfl_down_sync(0xffffffffu, v.hi.y, lanes)}};
}
__device__ __forceinline__ Quad shift_up(Quad v, int lanes) {
    return {{__shfl_up_sync(0xffffffffu, v.lo.x, lanes), __shfl_up_sync(0xffffffffu, v.lo.y, lanes)},
            {__shfl_up_sync(0xffffffffu, v.hi.x, lanes), __shfl_up_sync(0xffffffffu, v.hi.y, lanes)}};
}
// A gate: of four channels, or one that they share (gates of one head).
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ Quad mul(float a, Quad b) { return mul(all4(a), b); }
__device__ __forceinline__ Quad fma(float a, Quad b, Quad c) { return fma(all4(a), b, c); }
__device__ __forceinline__ float shift_up(float v, int lanes) { return __shfl_up_sync(0xffffffffu, v, lanes); }
__device__ __forceinline__ float shift_down(float v, int lanes) { return __shfl_down_sync(0xffffffffu, v, lanes); }
__device__ __forceinline__ void set_gate(float& g, float v) { g = v; }
__device__ __forceinline__ void set_gate(Quad& g, float v) { g = all4(v); }
__device__ __forceinline__ Quad of_channels(Quad g) { return g; }
__device__ __forceinline__ Quad of_channels(float g) { return all4(g); }

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

// A tiled 2-D copy of a box (channels c, tokens t) to shared memory; completes on `bar` as transaction bytes.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c, int32_t t) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                     smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c), "r"(t)
                 : "memory");
}

// A stage of one array in shared memory: rows of W channels.
template <class T, class Col>
struct StageArray {
    static constexpr int W = Col::kWidth, kTokens = Col::kTokens, kRun = Col::kRun;
    static constexpr int kRow = W * static_cast<int>(sizeof(T));
    static constexpr int kBytes = kTokens * kRow;
    static constexpr int kBox = kTokens < 256 ? kTokens : 256;  // tokens of a box

    static __device__ __forceinline__ void fetch(uint8_t* stage, const CUtensorMap* map, uint64_t* bar, int c0, int64_t t0) {
#pragma unroll
        for (int i = 0; i < kTokens / kBox; ++i)
            tma_load_2d(stage + i * kBox * kRow, map, bar, c0, static_cast<int32_t>(t0) + i * kBox);
    }
    static __device__ __forceinline__ Pack<T> get(const uint8_t* stage, int run, int k, int l) {
        return *reinterpret_cast<const Pack<T>*>(stage + (run * kRun + k) * kRow + l * 4 * static_cast<int>(sizeof(T)));
    }
    // What a thread reads of a stage becomes NaN: its copies have not come.
    static __device__ __forceinline__ void spoil(uint8_t* stage, int run, int l) {
        Pack<T> nan;
        memset(&nan, 0xff, sizeof(nan));
#pragma unroll 1
        for (int k = 0; k < kRun; ++k)
            *reinterpret_cast<Pack<T>*>(stage + (run * kRun + k) * kRow + l * 4 * static_cast<int>(sizeof(T))) = nan;
    }
};

// A stage of gates per head: the 16 bytes of each token's gates that hold the block's head.
template <class T, class Col>
struct StageGates {
    static constexpr int kTokens = Col::kTokens;
    static constexpr int kHeads = 16 / static_cast<int>(sizeof(T));
    static constexpr int kBytes = kTokens * 16;
    static constexpr int kBox = kTokens < 256 ? kTokens : 256;

    static __device__ __forceinline__ void fetch(uint8_t* stage, const CUtensorMap* map, uint64_t* bar, int head, int64_t t0) {
#pragma unroll
        for (int i = 0; i < kTokens / kBox; ++i)
            tma_load_2d(stage + i * kBox * 16, map, bar, head / kHeads * kHeads, static_cast<int32_t>(t0) + i * kBox);
    }
    static __device__ __forceinline__ float get(const uint8_t* stage, int token, int head) {
        return to_f32(reinterpret_cast<const T*>(stage)[token * kHeads + head % kHeads]);
    }
};

// The bounds of a stage's tokens.
template <int kTokens>
struct StageBounds {
    uint32_t starts[kTokens / 32], ends[kTokens / 32];
    uint32_t warps_start, warps_end;  // which warps' tokens hold a start, an end
    uint32_t plain;                   // which warps' tokens are all there, with neither
    int32_t start_seq[kTokens], end_seq[kTokens];
};

// An entry of cu_seqlens, c at place i, with its neighbours: marks the token of [t0, t1) that starts a sequence with it,
// and the one that ends the sequence before.  mark(start, sequence) is called for each.  Returns whether an empty sequence
// lies at c.  Entries are taken as they are: a malformed cu_seqlens gives wrong bounds, none outside.
template <int kTokens, class Mark>
__device__ __forceinline__ bool mark_entry(const LinearParams& p, int64_t i, int64_t c, int64_t prev, int64_t next, int64_t t0, int64_t t1,
                                           bool last, StageBounds<kTokens>& b, Mark mark) {
    if (i < 0 || i > p.N || c < t0 || c > t1) return false;
    if (i < p.N && c < t1 && next > c) {
        b.start_seq[c - t0] = static_cast<int32_t>(i);
        atomicOr(&b.starts[(c - t0) / 32], 1u << ((c - t0) % 32));
        mark(true, i);
    }
    if (i > 0 && c > t0 && prev < c) {
        b.end_seq[c - 1 - t0] = static_cast<int32_t>(i - 1);
        atomicOr(&b.ends[(c - 1 - t0) / 32], 1u << ((c - 1 - t0) % 32));
        mark(false, i - 1);
    }
    return i < p.N && next == c && (c < t1 || (last && c == t1));
}

template <int kTokens>
__device__ __forceinline__ void clear_bounds(StageBounds<kTokens>& b, int lane) {
    if (lane < kTokens / 32) b.starts[lane] = b.ends[lane] = 0;
    __syncwarp();
}

// Which warps' tokens hold what was marked.
template <int kTokens, int kWarpTokens>
__device__ __forceinline__ void sum_up_bounds(int64_t t0, int64_t t1, int lane, StageBounds<kTokens>& b) {
    __syncwarp();
    uint32_t s = 0, e = 0;
    constexpr int kWords = kTokens / kWarpTokens;
    if (lane < kWords) {
        static_assert(kWarpTokens == 16 || kWarpTokens == 32 || kWarpTokens == 64, "half a word of bounds a warp, one or two");
        if constexpr (kWarpTokens == 64) {
            s = b.starts[2 * lane] | b.starts[2 * lane + 1];
            e = b.ends[2 * lane] | b.ends[2 * lane + 1];
        } else {
            constexpr uint32_t kMask = kWarpTokens == 32 ? 0xffffffffu : 0xffffu;
            s = (b.starts[lane * kWarpTokens / 32] >> (lane * kWarpTokens % 32)) & kMask;
            e = (b.ends[lane * kWarpTokens / 32] >> (lane * kWarpTokens % 32)) & kMask;
        }
    }
    const uint32_t ws = __ballot_sync(0xffffffffu, s != 0), we = __ballot_sync(0xffffffffu, e != 0);
    const uint32_t plain = __ballot_sync(0xffffffffu, lane < kWords && (s | e) == 0 && t0 + (lane + 1) * kWarpTokens <= t1);
    if (lane == 0) {
        b.warps_start = ws;
        b.warps_end = we;
        b.plain = plain;
    }
}

// Fills the bounds of tokens [t0, t1) (one warp) from memory; no entry of cu_seqlens before `lo` is at or past t0.
// empty(i) is called by the whole warp for every empty sequence.
template <int kTokens, int kWarpTokens, class Empty>
__device__ __forceinline__ void fill_bounds(const LinearParams& p, int64_t lo, int64_t t0, int64_t t1, bool last, int lane,
                                         StageBounds<kTokens>& b, Empty empty) {
    clear_bounds<kTokens>(b, lane);
    for (;; lo += 32) {
        const int64_t i = lo + lane;
        const int64_t c = i <= p.N ? cu_at(p, i) : t1 + 1;
        const int64_t next = i < p.N ? cu_at(p, i + 1) : c, prev = i > 0 && i <= p.N ? cu_at(p, i - 1) : c;
        const bool gap = mark_entry<kTokens>(p, i, c, prev, next, t0, t1, last, b, [](bool, int64_t) {});
        for (uint32_t m = __ballot_sync(0xffffffffu, gap); m; m &= m - 1) empty(lo + __ffs(m) - 1);
        if (__any_sync(0xffffffffu, c > t1)) break;
    }
    sum_up_bounds<kTokens, kWarpTokens>(t0, t1, lane, b);
}

// 32 entries of cu_seqlens in a warp's registers, a lane's at place `first` + lane (step = 1) or `first` - lane (step = -1).
// Loaded a stage before they are looked at, so that a stage with bounds does not wait for memory.
struct Window {
    int64_t first, c;
    __device__ __forceinline__ void load(const LinearParams& p, int64_t at, int step, int lane) {
        first = at;
        const int64_t i = at + step * lane;
        c = i < 0 ? -1 : i <= p.N ? cu_at(p, i) : INT64_MAX;
    }
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int kTokens>
__device__ __forceinline__ void no_bounds(StageBounds<kTokens>& b, int lane) {
    if (lane == 0) {
        b.warps_start = b.warps_end = 0;
        b.plain = 0xffffffffu;
    }
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

// A run's bounds, a bit a token.
template <int kRun>
__device__ __forceinline__ uint32_t run_bits(const uint32_t* words, int run) {
    return (words[run * kRun / 32] >> (run * kRun % 32)) & ((1u << kRun) - 1u);
}

// Which of a warp's runs hold a bound, a bit a run.
template <int kRun, int kRuns>
__device__ __forceinline__ uint32_t runs_with(const uint32_t* words, int warp) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) r |= (run_bits<kRun>(words, warp * kRuns + i) ? 1u : 0u) << i;
    return r;
}

// Which tokens of any of a warp's runs hold a bound: what a warp tests before it looks at its own run's.
template <int kRun, int kRuns>
__device__ __forceinline__ uint32_t any_run_bits(const uint32_t* words, int warp) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) r |= run_bits<kRun>(words, warp * kRuns + i);
    return r;
}

// Whether no bit is set after bit `at`.
template <int kTokens>
__device__ __forceinline__ bool is_last_bit(const uint32_t* words, int at) {
    uint32_t after = at % 32 == 31 ? 0u : words[at / 32] >> (at % 32 + 1);
    for (int w = at / 32 + 1; w < kTokens / 32; ++w) after |= words[w];
    return after == 0;
}

// Time segments of a column, where there are too few columns for the GPU's SMs.  Segments after the first go over their
// tokens twice: once to learn what they do to a state, and, when the state that enters is known, once more (from HBM,
// mostly: 368 MB read for 201 MB of inputs of 32768 x 1024, bf16).
struct Segments {
    ScanSpace space;               // nt = segments; flags [blocks][nt]
    int32_t first, stages;         // stages of the first segment, and of the others
};

// At the end of a block that gave up a wait: what copies are under way get time to land, before the block's shared memory goes
// (one thread).  A place's phase that is under way is of one parity, and of the other the wait is over at once.
template <int kDepth>
__device__ __forceinline__ void drain(uint64_t (&full)[kDepth], long long cycles) {
    for (int i = 0; i < kDepth; ++i)
        for (uint32_t parity = 0; parity < 2; ++parity) mbar_wait(&full[i], parity, cycles / 8);
}

// Maps of the inputs for tiled copies (not of gates of any heads).
struct ColumnMaps {
    CUtensorMap x, a, b, dy;
};

constexpr int kForwardWarps = 8, kForwardGroups = 2;

// How gates are found: per channel; of one head for the block's channels (the head's channels are a multiple of them, and
// rows of gates can be copied); or of any heads (4 channels of a lane share one), by plain loads.
enum Gates { kPerChannel, kOneHead, kAnyHead };

template <class X, class G, int kGates, bool kHasB, class Col>
struct ForwardShape {
    static constexpr int W = Col::kWidth, kTokens = Col::kTokens;
    using AX = StageArray<X, Col>;
    using AG = std::conditional_t<kGates == kOneHead, StageGates<G, Col>, StageArray<G, Col>>;
    static constexpr int kStageBytes = AX::kBytes + (kGates == kAnyHead ? 0 : kHasB ? 2 : 1) * AG::kBytes;
    static constexpr int kDepth = kRingBytes / kStageBytes < 4 ? kRingBytes / kStageBytes : 4;
    struct Group {
        StageBounds<kTokens> bounds[3];
        alignas(16) float2 pairs[2][Col::kWarps][W];
        alignas(16) float kept[W];  // initial state of the last sequence that starts in the segment's stages of this group
        int64_t kept_at;            // its first token
    };
    struct Tables {
        Group groups[Col::kGroups];
        float hand[Col::kHands][W];   // the state that enters a stage
        int32_t hand_reset[Col::kHands];
        Product product[Col::kSegments ? Col::kGroups * Col::kWarps : 1][W];  // of the gates of a warp's steps that learn
        uint64_t full[kDepth];        // a stage's inputs have come
        uint64_t handed[Col::kHands];
        uint32_t ticket;
    };
    static constexpr int kSmem = kDepth * kStageBytes + static_cast<int>(sizeof(Tables));
    static_assert(kStageBytes % 128 == 0 && alignof(Tables) == 16, "boxes and tables lie aligned");
    static_assert(kDepth >= 2, "the next stage comes while one is worked on");
};

template <class X, class G, int kGates, bool kHasB, class Col>
__global__ void __launch_bounds__(Col::kThreads, 1)
    gdn_linear_column_forward_kernel(const LinearParams p, const Segments seg, const __grid_constant__ ColumnMaps maps) {
    using Shape = ForwardShape<X, G, kGates, kHasB, Col>;
    using AX = typename Shape::AX;
    using AG = typename Shape::AG;
    constexpr int W = Shape::W, kTokens = Shape::kTokens, kDepth = Shape::kDepth, kRuns = Col::kRuns, kLanesRow = Col::kLanesRow;
    constexpr int kColWarps = Col::kWarps, kWarpTokens = Col::kWarpTokens, kRun = Col::kRun, kGroups = Col::kGroups;
    constexpr int kHands = Col::kHands;
    extern __shared__ __align__(1024) uint8_t ring[];
    typename Shape::Tables& sm = *reinterpret_cast<typename Shape::Tables*>(ring + kDepth * Shape::kStageBytes);
    const int group = threadIdx.x / (32 * kColWarps), warp = threadIdx.x / 32 % kColWarps, lane = threadIdx.x % 32;
    typename Shape::Group& gr = sm.groups[group];
    const bool leader = warp == 0 && lane == 0;  // of the group
    const int sub = lane / kLanesRow, l = lane % kLanesRow, run = warp * kRuns + sub, ch = lane % W;
    const ScanSpace& sp = seg.space;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kDepth; ++i) mbar_init(&sm.full[i], 1);
        for (int i = 0; i < kHands; ++i) mbar_init(&sm.handed[i], 1);
        fence_mbar_init();
        mbar_arrive(&sm.handed[0]);  // nothing is handed to stage 0: its place's first turn is over
        for (int i = 0; i < kGroups; ++i) sm.groups[i].kept_at = -1;
        if (Col::kSegments) sm.ticket = atomicAdd(sp.ticket, 1u);
    }
    if (Col::kSegments) sm.product[threadIdx.x / 32][lane] = Product{1.f, 0};
    __syncthreads();
    const uint32_t ticket = Col::kSegments ? sm.ticket : blockIdx.x;
    const int64_t part = Col::kSegments ? ticket / sp.blocks : 0;
    const uint32_t blk = Col::kSegments ? ticket % sp.blocks : ticket;
    const int c0 = static_cast<int>(blk) * W, cols = min(W, p.C - c0);
    const int64_t from = part == 0 ? 0 : (seg.first + (part - 1) * seg.stages) * static_cast<int64_t>(kTokens);
    const int64_t end = !Col::kSegments || part == sp.nt - 1 ? p.T : (seg.first + part * seg.stages) * static_cast<int64_t>(kTokens);
    const int stages = static_cast<int>(max(static_cast<int64_t>(1), (end - from + kTokens - 1) / kTokens));
    // A later segment learns what it does to a state in steps 0 .. stages - 1.
    const bool twice = Col::kSegments && part > 0;
    const int steps = p.T == 0 ? 0 : twice ? 2 * stages : stages;
    const bool on = l * 4 < cols;

    const int head = kGates == kPerChannel ? c0 : (c0 + (kGates == kAnyHead && on ? l * 4 : 0)) / p.D;
    const G* ga = static_cast<const G*>(p.a) + head;
    const G* gb = kHasB ? static_cast<const G*>(p.b) + head : nullptr;
    auto stage_start = [&](int q) { return from + static_cast<int64_t>(q < stages ? q : q - stages) * kTokens; };
    auto fetch = [&](int q) {  // one thread
        if (q >= steps) return;
        uint8_t* stage = ring + q % kDepth * Shape::kStageBytes;
        uint64_t* bar = &sm.full[q % kDepth];
        const int64_t t0 = stage_start(q);
        mbar_arrive_expect_tx(bar, Shape::kStageBytes);
        AX::fetch(stage, &maps.x, bar, c0, t0);
        if constexpr (kGates != kAnyHead) {
            const int at = kGates == kOneHead ? head : c0;
            AG::fetch(stage + AX::kBytes, &maps.a, bar, at, t0);
            if constexpr (kHasB) AG::fetch(stage + AX::kBytes + AG::kBytes, &maps.b, bar, at, t0);
        }
    };
    // A thread's inputs of a stage: x and gates per channel of its run; of gates of one head the token that is its lane's
    // in the run; of gates of any heads its run's.
    constexpr int kHeld = kGates == kOneHead ? kRun / kLanesRow : kRun;
    Pack<X> px[kRun];
    Pack<G> pa[kGates == kPerChannel ? kRun : 1], pb[kGates == kPerChannel ? kRun : 1];
    float ha[kHeld], hb[kHeld];
    bool ok = true;  // until a wait runs out; then what this thread adds to the results is NaN
    auto wait = [&](uint64_t* bar, uint32_t parity, long long cycles) {
        if (!ok || mbar_wait(bar, parity, cycles)) return;
        ok = false;
        report(p.status, GDN_DEVICE_ERR_TIMEOUT);
    };
    auto take = [&](int q) {
        if (kGates == kAnyHead) {
            const int64_t t = stage_start(q) + run * kRun;
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                ha[k] = hb[k] = 1.f;
                if (t + k >= end) continue;
                ha[k] = to_f32(ga[(t + k) * p.a_stride]);
                if constexpr (kHasB) hb[k] = to_f32(gb[(t + k) * p.b_stride]);
            }
        }
        uint8_t* stage = ring + q % kDepth * Shape::kStageBytes;
        wait(&sm.full[q % kDepth], (q / kDepth) & 1, copy_wait(sp.wait_cycles));
        if (!ok) AX::spoil(stage, run, l);
        const uint8_t *sa = stage + AX::kBytes, *sb = sa + AG::kBytes;
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            px[k] = AX::get(stage, run, k, l);
            if constexpr (kGates == kPerChannel) {
                pa[k] = AG::get(sa, run, k, l);
                if constexpr (kHasB) pb[k] = AG::get(sb, run, k, l);
            }
        }
        if constexpr (kGates == kOneHead) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int tok = run * kRun + i * kLanesRow + l;
                ha[i] = AG::get(sa, tok, head);
                if constexpr (kHasB) hb[i] = AG::get(sb, tok, head);
            }
        }
    };
    Window win{0, 0};  // from the last entry before the tokens to come on
    auto bounds = [&](int q) {
        if (q >= max(steps, 1)) return;  // without tokens, the empty sequences
        const int64_t t0 = stage_start(q), t1 = min(t0 + kTokens, end);
        if (q < kGroups || (q >= stages && q < stages + kGroups))
            win.load(p, first_entry(p, static_cast<int64_t>(p.N) + 1, t0, lane) - 1, 1, lane);
        StageBounds<kTokens>& b = gr.bounds[q / kGroups % 3];
        if (t1 == t0 + kTokens && !__any_sync(0xffffffffu, win.c >= t0 && win.c <= t1) && __any_sync(0xffffffffu, win.c > t1)) {
            no_bounds(b, lane);  // most stages
            return;
        }
        const bool write = q >= steps - stages, last = t1 == p.T;
        auto empty = [&](int64_t i) {  // an empty sequence's final state is its initial one
            if (!write) return;
            const int64_t row = state_row(p, i);  // looked at, and reported, whether or not there is anything to copy
            if (row < 0 || !p.output_state || p.output_state == p.initial_state || lane * 4 >= cols) return;
            const int64_t off = row * p.state_stride + c0 + lane * 4;
            state_quad_store(p.output_state, off, p.state_dt,
                             p.initial_state ? state_quad_load(p.initial_state, off, p.state_dt) : make_float4(0.f, 0.f, 0.f, 0.f));
        };
        if (__shfl_sync(0xffffffffu, win.c, 31) > t1) {  // the window holds all of the stage's entries
            clear_bounds<kTokens>(b, lane);
            const int64_t next = __shfl_down_sync(0xffffffffu, win.c, 1), prev = __shfl_up_sync(0xffffffffu, win.c, 1);
            const bool gap = lane > 0 && mark_entry<kTokens>(p, win.first + lane, win.c, prev, next, t0, t1, last, b, [&](bool start, int64_t i) {
                if (start && p.initial_state && !p.state_indices)
                    prefetch_l2(static_cast<const uint8_t*>(p.initial_state) + (i * p.state_stride + c0) * dtype_bytes(p.state_dt));
            });
            for (uint32_t m = __ballot_sync(0xffffffffu, gap); m; m &= m - 1) empty(win.first + __ffs(m) - 1);
            sum_up_bounds<kTokens, kWarpTokens>(t0, t1, lane, b);
            win.load(p, win.first + __popc(__ballot_sync(0xffffffffu, win.c < t1)) - 1, 1, lane);
        } else {
            const int64_t lo = first_entry(p, static_cast<int64_t>(p.N) + 1, t0, lane);
            fill_bounds<kTokens, kWarpTokens>(p, lo, t0, t1, last, lane, b, empty);
            win.load(p, first_entry(p, static_cast<int64_t>(p.N) + 1, t1, lane) - 1, 1, lane);
        }
    };

    if (threadIdx.x == 0)
        for (int q = 0; q < kDepth; ++q) fetch(q);
    if (warp == kColWarps - 1) bounds(group);
    if (group == 0 && warp == 0 && blk == 0) check_bounds(p, part, sp.nt, lane);
    __syncthreads();
    X* y = static_cast<X*>(p.y) + c0 + l * 4;
    auto wait_hand = [&](int q) { wait(&sm.handed[q % kHands], (q / kHands) & 1, hand_wait(sp.wait_cycles)); };
    for (int q = group; q < steps; q += kGroups) {
        const StageBounds<kTokens>& bd = gr.bounds[q / kGroups % 3];
        const bool learn = twice && q < stages;
        const int64_t t = stage_start(q) + run * kRun;
        if (twice && q >= stages && q < stages + kGroups) wait_hand(q);  // all that learns has been done: states are kept
        using Gate = std::conditional_t<kGates == kPerChannel, Quad, float>;
        Gate a[kRun], A, exA;
        Quad u[kRun], B, exB;
        uint32_t starts = 0, ends = 0;
        int n = kRun;
        bool plain = true, before = false;  // before: whether a sequence starts in the warp's runs before this one
        if (warp == kColWarps - 1) bounds(q + kGroups);
        plain = (bd.plain >> warp) & 1;
        take(q);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            u[k] = widen(px[k]);
            if constexpr (kGates == kOneHead) {
                const int from_lane = sub * kLanesRow + k % kLanesRow;
                a[k] = __shfl_sync(0xffffffffu, ha[k / kLanesRow], from_lane);
                if constexpr (kHasB) u[k] = mul(__shfl_sync(0xffffffffu, hb[k / kLanesRow], from_lane), u[k]);
            } else if constexpr (kGates == kAnyHead) {
                a[k] = ha[k];
                if constexpr (kHasB) u[k] = mul(hb[k], u[k]);
            } else {
                a[k] = widen(pa[k]);
                if constexpr (kHasB) u[k] = mul(u[k], widen(pb[k]));
            }
        }
        set_gate(A, 1.f);
        B = all4(0.f);
        uint32_t any = 0;
        if (!plain) {
            n = static_cast<int>(min(static_cast<int64_t>(kRun), max(static_cast<int64_t>(0), end - t)));
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                if (k < n) continue;
                set_gate(a[k], 1.f);
                u[k] = all4(0.f);
            }
            starts = run_bits<kRun>(bd.starts, run);
            ends = run_bits<kRun>(bd.ends, run);
            any = any_run_bits<kRun, kRuns>(bd.starts, warp);
        }
        // `whole`: all of the warp's tokens are there, with neither a start nor an end: code without a branch.
        auto compose = [&](auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                if (!kWhole && ((any >> k) & 1) && ((starts >> k) & 1)) {
                    if (p.initial_state && on) {
                        const int64_t row = state_row(p, bd.start_seq[run * kRun + k]);
                        // With states in place, a later segment may have written the row of a sequence that starts
                        // here by the time of the second pass: the last one to start, if any.  Its state is kept.
                        float4 h0 = make_float4(0.f, 0.f, 0.f, 0.f);
                        bool kept = false;
                        if (twice && !learn)
                            for (int i = 0; i < kGroups; ++i)
                                if (t + k == sm.groups[i].kept_at) {
                                    h0 = *reinterpret_cast<const float4*>(&sm.groups[i].kept[l * 4]);
                                    kept = true;
                                }
                        if (!kept && row >= 0)
                            h0 = state_quad_load(p.initial_state, row * p.state_stride + c0 + l * 4, p.state_dt);
                        if (learn && is_last_bit<kTokens>(bd.starts, run * kRun + k)) {
                            *reinterpret_cast<float4*>(&gr.kept[l * 4]) = h0;
                            gr.kept_at = t + k;
                        }
                        if (row >= 0) u[k] = fma(a[k], quad(h0), u[k]);
                    }
                    B = all4(0.f);
                }
                A = mul(A, a[k]);
                B = fma(a[k], B, u[k]);
            }
        };
        if (plain)
            compose(std::true_type{});
        else
            compose(std::false_type{});
        // over the warp's runs
        const uint32_t rs = (bd.warps_start >> warp) & 1 ? runs_with<kRun, kRuns>(bd.starts, warp) : 0;
#pragma unroll
        for (int o = 1; o < kRuns; o <<= 1) {
            const bool mine = (rs >> max(0, sub - o + 1)) & ((1u << o) - 1u);
            const Gate oa = shift_up(A, o * kLanesRow);
            const Quad ob = shift_up(B, o * kLanesRow);
            if (sub >= o) {
                B = pick(mine, B, fma(A, ob, B));
                A = mul(A, oa);
            }
        }
        exA = shift_up(A, kLanesRow);
        exB = shift_up(B, kLanesRow);
        if (sub == 0) {
            set_gate(exA, 1.f);
            exB = all4(0.f);
        }
        before = (rs & ((1u << sub) - 1u)) != 0;
        if (sub == kRuns - 1) {
            float4* o = reinterpret_cast<float4*>(&gr.pairs[q / kGroups & 1][warp][l * 4]);
            const Quad g = of_channels(A);
            o[0] = make_float4(g.lo.x, B.lo.x, g.lo.y, B.lo.y);
            o[1] = make_float4(g.hi.x, B.hi.x, g.hi.y, B.hi.y);
        }
        if (learn) {
            __syncwarp();
            Product& mine = sm.product[threadIdx.x / 32][lane];
            mine = times(mine, gr.pairs[q / kGroups & 1][warp][lane].x);
        }
        // The group's one barrier of a step.  Past it: every warp's pair is there and every thread has its inputs of this
        // stage, so its place in the ring is free; the bounds of the group's next stage are known.
        named_bar_sync(1 + group, 32 * kColWarps);
        if (leader && ok) fetch(q + kDepth);
        float2 ab[kColWarps];
#pragma unroll
        for (int w = 0; w < kColWarps; ++w) ab[w] = gr.pairs[q / kGroups & 1][w][ch];
        const uint32_t resets = bd.warps_start;
        // What the stage before hands on: the state (in steps that learn, from zero).
        float carry = 0.f;
        if (q > 0) {
            wait_hand(q);
            carry = ok ? sm.hand[q % kHands][ch] : nanf("");
        }
        float enter = carry;
#pragma unroll
        for (int w = 0; w < kColWarps; ++w) {
            if (w == warp) enter = carry;
            carry = fmaf(ab[w].x, carry, ab[w].y);
            if (resets != 0 && ((resets >> w) & 1)) carry = ab[w].y;
        }
        if (warp == 0) {
            const bool reset = resets != 0 || (learn && q > 0 && sm.hand_reset[q % kHands] != 0);
            const int c = c0 + lane;
            uint32_t* flags = sp.flags + static_cast<int64_t>(blk) * sp.nt;
            if (learn && q == stages - 1) {  // the segment's pair goes on, the state that enters it comes
                const bool lastpart = part == sp.nt - 1;
                Product whole{1.f, 0};
                for (int i = 0; i < kGroups * kColWarps; ++i) whole = times(whole, sm.product[i][lane]);
                whole = folded(whole);
                if (!lastpart) {
                    if (lane < cols) {
                        if (reset) {
                            sp.known[part * p.C + c] = carry;
                        } else {
                            sp.pairs[part * p.C + c] = make_float2(whole.m, carry);
                            sp.exponents[part * p.C + c] = whole.e;
                        }
                    }
                    const bool scaled = __any_sync(0xffffffffu, whole.e != 0);
                    publish(flags + part, reset ? kKnown : scaled ? kScaledPair : kPair, lane);
                }
                const float h = look_back<true>(p, sp, flags, part, lane < cols ? c : p.C, lane, [](int64_t k) { return k; });
                if (!lastpart && !reset) {
                    if (lane < cols) sp.known[part * p.C + c] = pass_on(whole, h, carry);
                    publish(flags + part, kKnown, lane);
                }
                carry = h;
            } else if (Col::kSegments && part == 0 && q == steps - 1) {  // the first segment's end state
                if (lane < cols) sp.known[c] = carry;
                publish(flags, kKnown, lane);
            }
            if (lane < W) sm.hand[(q + 1) % kHands][lane] = carry;
            if (lane == 0) sm.hand_reset[(q + 1) % kHands] = reset;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.handed[(q + 1) % kHands]);
        }
        if (learn) continue;
        const Quad e = {{__shfl_sync(0xffffffffu, enter, l * 4), __shfl_sync(0xffffffffu, enter, l * 4 + 1)},
                        {__shfl_sync(0xffffffffu, enter, l * 4 + 2), __shfl_sync(0xffffffffu, enter, l * 4 + 3)}};
        Quad h = pick(before, exB, fma(exA, e, exB));
        if (!on) continue;
        X* out = y + t * p.y_stride;
        auto tokens = [&](auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                if (!kWhole && ((starts >> k) & 1)) h = all4(0.f);
                h = fma(a[k], h, u[k]);
                if (kWhole || k < n) store_stream(reinterpret_cast<Pack<X>*>(out), narrow(h, X{}));
                out += p.y_stride;
                if (!kWhole && ((ends >> k) & 1)) {
                    if (p.output_state) {
                        const int64_t row = state_row(p, bd.end_seq[run * kRun + k]);
                        if (row >= 0) state_quad_store(p.output_state, row * p.state_stride + c0 + l * 4, p.state_dt, flat(h));
                    }
                    if (p.tile_states && t + k == p.T - 1)
                        *reinterpret_cast<float4*>(p.tile_states + (t + k) / kTile * p.C + c0 + l * 4) = flat(h);
                }
            }
        };
        if (plain)
            tokens(std::true_type{});
        else
            tokens(std::false_type{});
        if (p.tile_states && (t + kRun) % kTile == 0 && n == kRun)
            *reinterpret_cast<float4*>(p.tile_states + t / kTile * p.C + c0 + l * 4) = flat(h);
    }
    if (leader && !ok) drain(sm.full, sp.wait_cycles);
}

template <class X, class G, int kGates, bool kHasB, class Col>
cudaError_t launch_column_forward(const LinearParams& p, const Segments& seg, cudaStream_t stream) {
    using Shape = ForwardShape<X, G, kGates, kHasB, Col>;
    ColumnMaps maps{};
    bool ok = p.T == 0 || encode_rows(&maps.x, p.x, p.x_dt, p.x_stride, p.C, p.T, Shape::W, Shape::AX::kBox);
    if (kGates != kAnyHead && p.T > 0) {
        const int64_t row = kGates == kOneHead ? p.H : p.C;
        const int width = kGates == kOneHead ? 16 / static_cast<int>(sizeof(G)) : Shape::W;
        ok = ok && encode_rows(&maps.a, p.a, p.gate_dt, p.a_stride, row, p.T, width, Shape::AG::kBox);
        if (kHasB) ok = ok && encode_rows(&maps.b, p.b, p.gate_dt, p.b_stride, row, p.T, width, Shape::AG::kBox);
    }
    if (!ok) return cudaErrorInvalidValue;
    auto kernel = gdn_linear_column_forward_kernel<X, G, kGates, kHasB, Col>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(seg.space.nt * seg.space.blocks), Col::kThreads, Shape::kSmem, stream>>>(p, seg, maps);
    return cudaGetLastError();
}

template <class X, class G, int kGates>
cudaError_t column_forward_gates(const LinearParams& p, const Segments& seg, int width, cudaStream_t stream) {
    constexpr int kWarps = kForwardWarps, kGroups = kForwardGroups;
    if (seg.space.nt > 1)
        return p.b ? launch_column_forward<X, G, kGates, true, Column<32, kWarps, 8, kGroups, true>>(p, seg, stream)
                   : launch_column_forward<X, G, kGates, false, Column<32, kWarps, 8, kGroups, true>>(p, seg, stream);
    if (width == 32)
        return p.b ? launch_column_forward<X, G, kGates, true, Column<32, kWarps, 8, kGroups>>(p, seg, stream)
                   : launch_column_forward<X, G, kGates, false, Column<32, kWarps, 8, kGroups>>(p, seg, stream);
    return p.b ? launch_column_forward<X, G, kGates, true, Column<16, kWarps, 8, kGroups>>(p, seg, stream)
               : launch_column_forward<X, G, kGates, false, Column<16, kWarps, 8, kGroups>>(p, seg, stream);
}

// Whether a block of `width` channels has one head, and its gates can be copied.
inline bool one_head(const LinearParams& p, int width) {
    const auto rows = [&](const void* g, int64_t stride) {
        return reinterpret_cast<uintptr_t>(g) % 16 == 0 && stride * dtype_bytes(p.gate_dt) % 16 == 0;
    };
    return p.D % width == 0 && rows(p.a, p.a_stride) && rows(p.b, p.b_stride);
}

template <class X, class G>
cudaError_t column_forward_typed(const LinearParams& p, const Segments& seg, int width, cudaStream_t stream) {
    if (p.gate_div == 1) return column_forward_gates<X, G, kPerChannel>(p, seg, width, stream);
    if (one_head(p, width)) return column_forward_gates<X, G, kOneHead>(p, seg, width, stream);
    return column_forward_gates<X, G, kAnyHead>(p, seg, width, stream);
}

}  // namespace linear
}  // namespace gdn
