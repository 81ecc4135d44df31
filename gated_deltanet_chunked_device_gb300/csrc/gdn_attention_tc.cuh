// gdn_attention_tc.cuh -- attention over a paged cache on the tensor cores (bf16 and fp16).
//
// A unit's rows (token, head of the group) are the 128 rows of tcgen05 products; grouped heads and speculated tokens fill them
// where tokens alone would not.  Keys and values come by tiled copies, a box a page (or piece of one), straight from the caller's
// cache in any strides; what lies outside a page, a head or the cache reads as zeros.  Per tile of keys:
//
//     S = Q K^T               fp32 in TMEM
//     P = exp2(S - m)         a thread a row, from TMEM to registers and back as 16-bit pairs over S
//     O += P V                P from TMEM, O fp32 in TMEM
//
// m is the row's running maximum, raised (and O and the sum l scaled down) only when it has grown by more than 2^8: P stays
// below 1 (fp16: 2^15), and any m gives the same quotient.  P is rounded to 16 bits for the product, relative to itself; l sums the
// unrounded weights in fp32.
//
// Two shapes.  kStreams = 2, for many rows: two row tiles against the same keys, each with a warpgroup of its own for the
// exponentials, so that the tensor cores work on one while the other's are computed.  kStreams = 1, for few rows, or heads of
// 256: one row tile, the scores of the next keys ahead of the exponentials of the present ones; what counts there is the stream of
// keys and values, 160 KB of which are on their way at any time.
//
// Bounds and figures (GB300).  Many rows: the chain scores - exponentials - weights - products of two streams; the tensor pipe works
// 59 % of the time (2048 tokens over 30720, 32 heads on 16 of 128, fp16: 0.9 ms, 1.17 PFLOP/s; 8 prompts of 33720 tokens, 32 heads on
// 8, bf16: 1.42 ms, 1.18 PFLOP/s).  Single tokens over long contexts: HBM (512 sequences of up to 8192, bf16: 331 us, 0.97 of a
// measured copy).  Four tokens under a window of 1024, heads of 64, pages of 16: a tile's steps and a copy a page of 2 KB (72 us, floor
// 20; four warps that share a tile's keys brought 80 to 67, a division that suits short sequences cost 4, looking through the values of
// cut tiles 2).  Heads of 256 with many rows: the chain of a single row tile (tensor pipe 35 %).
//
// Where tiled copies cannot fetch the rows (pages of sizes that are no multiple of 8, heads of 100 channels) warps 0 and 3 copy them
// piece by piece into the same layout; that bounds the kernel then (a chunk of 4096 tokens over as many, 16 heads on 2: 197 us with
// tiled copies, 850 in pieces of 16 bytes).
//
// Warps: 0 finds the work and copies, 1 (and 2) issue the products, 2 owns TMEM, 3 helps with plain copies, 4.. exponentials and results.
#pragma once

#include <type_traits>

#include "gdn_attention.cuh"
#include "sm103_ptx.cuh"

namespace gdn {
namespace attn_tc {

constexpr int kRowTile = 128;
constexpr float kGrowth = 8.f;      // log2 of how far a row's maximum may fall behind
// log2 of a row's largest weight as P holds it, when its maximum has just been taken.  fp16: weights are lifted out of its subnormals, and
// stay below 2^15.  bf16 has the range of fp32: weights stay below 1, so that sums of them times large values overflow no sooner than
// a softmax's does.
template <class E>
constexpr float weight_offset() { return std::is_same<E, __half>::value ? 7.f : -kGrowth; }
constexpr int kParts = 4;           // parts handed from the producer to the others ahead

template <int kDim, int kStreams>
struct Shape {
    static_assert(kDim == 64 || kDim == 128 || (kDim == 256 && kStreams == 1), "TMEM holds no more");
    static constexpr int kKeys = 128;                                // keys a tile
    static constexpr int kHalves = kDim == 256 ? 2 : 1;              // stages a tile of keys or values takes: 128 channels each at most
    static constexpr int kChunks = kDim / 64 / kHalves;              // swizzled columns of 64 channels in a stage
    static constexpr int kQBytes = kHalves * kChunks * kRowTile * 128;
    static constexpr int kKvBytes = kChunks * kKeys * 128;
    static constexpr int kQSlots = kStreams == 1 && kDim < 256 ? 2 : 1;  // units whose Q is there
    static constexpr int kQTiles = kQSlots * kStreams;
    static constexpr int kStages = (224 * 1024 - kQTiles * kQBytes) / kKvBytes;
    static constexpr int kTileBytes = kQTiles * kQBytes + kStages * kKvBytes;
    static constexpr int kThreads = 128 + 128 * kStreams;
    static constexpr uint32_t kTmemO = 256;                          // S slots at columns 0 and 128
};

// What the launch adds to AttnParams.
struct TcParams {
    AttnParams a;
    int32_t row_tokens;            // tokens a row tile
    int32_t box_keys;              // keys a box: what pages and tiles have in common
    int32_t boxes;                 // of a tile, along the keys
    int32_t k_steps;               // steps of 16 channels a stage
    uint32_t idesc_qk, idesc_pv;
    float scale_log2;              // positive: a negative scale negates Q in the product
    int32_t out_vec;               // results can be written 16 bytes at a time
    int32_t quarters;              // units of at most 32 rows: each warp of exponentials has a quarter of the keys
    int32_t plain;                 // bytes of a plain copy (16, 8 or 4) where tiled copies cannot fetch the rows; 0: tiled copies
    long long wait_cycles;         // limit of a wait
};

template <class S>
struct Misc {
    uint64_t kv_full[S::kStages], kv_empty[S::kStages], q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], pv_done[2];
    uint64_t part_full[kParts], part_empty[kParts], both, mix, turn[2], drain[2];
    uint4 stage_keys[S::kStages], slot_keys[2];  // keys that have a page (or lie behind the sequence), a bit each
    uint32_t slot_missing[2];      // whether some of a slot's keys have none
    int2 rows[2][2][64];           // plain copies: page and place of a warp's half of the keys of two tiles
    uint32_t tmem;
    int32_t abort;
    AttnPart parts[kParts];
    AttnScan<S::kThreads> scan;
    // Tiles [x, y) of a stream's part that had values set apart, for every second part: in the place of the scan's sums, which have done
    // their work when the walk starts.
    __device__ __forceinline__ int2& unfinite(int stream, uint32_t part) { return reinterpret_cast<int2*>(scan.sums)[2 * stream + (part & 1)]; }
};

template <class S>
constexpr size_t smem_bytes() { return S::kTileBytes + sizeof(Misc<S>); }

constexpr long long kWaitCycles = 2000000000LL;  // about a second

// Waits up to a limit; the first wait that runs out makes all others give up.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, int32_t* abort, int32_t* status, long long limit) {
    const long long t0 = clock64();
    while (!mbar_try_wait_sleep(bar, parity, 1000)) {
        if (*static_cast<volatile int32_t*>(abort)) return false;
        if (clock64() - t0 > limit) {
            *static_cast<volatile int32_t*>(abort) = 1;
            kv_report(status, GDN_DEVICE_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The lowest n bits, n of any size and sign.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// A bit a key from a bit a box of `keys` keys.
__device__ __forceinline__ uint4 spread_boxes(uint32_t mask, int boxes, int keys) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0;
        for (int b = 0; b < boxes; ++b)
            if (mask >> b & 1) w[i] |= low_bits((b + 1) * keys - 32 * i) & ~low_bits(b * keys - 32 * i);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// By a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int32_t* abort, int32_t* status, long long limit) {
    return __all_sync(~0u, mbar_try_wait(bar, parity) || wait_long(bar, parity, abort, status, limit));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t both(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma_both(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_both(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <class E>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (sizeof(E) == 2 && std::is_same<E, __half>::value)
        return pack_f16x2(lo, hi);
    else
        return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ float wide16(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float wide16(__half x) { return __half2float(x); }
template <class E>
__device__ __forceinline__ E narrow16(float x) {
    if constexpr (std::is_same<E, __half>::value)
        return __float2half_rn(x);
    else
        return __float2bfloat16_rn(x);
}

// Tiles of row tile s of a part that some of its rows see (what lies behind, only later rows see).
__device__ __forceinline__ int32_t stream_end(const TcParams& p, const AttnPart& a, int s, int32_t keys_a_tile) {
    const int32_t t1 = min(a.tokens, (s + 1) * p.row_tokens);
    if (s * p.row_tokens >= a.tokens) return a.tile0;
    if (!p.a.causal) return a.tile1;
    const int64_t hi = min(max(static_cast<int64_t>(a.pos0) + t1, int64_t{0}), static_cast<int64_t>(a.keys));
    return max(a.tile0, static_cast<int32_t>(min(static_cast<int64_t>(a.tile1), (hi + keys_a_tile - 1) / keys_a_tile)));
}

// The lane `with` away gets one's second value for its own first: lanes whose bit is set keep their second.
__device__ __forceinline__ void swap_quads(uint4& a, uint4& b, int bit, int with) {
    const uint4 give = bit ? a : b;
    const uint4 got = make_uint4(__shfl_xor_sync(~0u, give.x, with), __shfl_xor_sync(~0u, give.y, with), __shfl_xor_sync(~0u, give.z, with),
                                 __shfl_xor_sync(~0u, give.w, with));
    if (bit)
        a = got;
    else
        b = got;
}

// Where a row's result goes.
template <class E>
struct RowOut {
    E* o;                          // whole units
    float* lse;
    float* part;                   // parts
    float2* ml;
};

template <class E>
__device__ __forceinline__ RowOut<E> row_out(const AttnParams& p, const AttnPart& a, int32_t block, int t, int g) {
    RowOut<E> r{};
    const int D = p.c.head_dim;
    if (a.tile0 == a.first && a.tile1 == a.last) {
        r.o = static_cast<E*>(p.o) + (a.row0 + t) * p.o_stride + static_cast<int64_t>(a.head0 + g) * D;
        if (p.lse) r.lse = p.lse + (a.row0 + t) * p.heads + a.head0 + g;
    } else {
        const int64_t at = static_cast<int64_t>(attn_slot(a, block)) * (p.unit_tokens * p.group) + t * a.heads + g;
        r.part = p.part_o + at * D;
        r.ml = p.part_ml + at;
    }
    return r;
}

// Values that are not finite, two at a time (16 bits each): marked by their sign bits; and left out.
template <class E>
__device__ __forceinline__ uint32_t unfinite_signs(uint32_t x) {
    if constexpr (std::is_same<E, __half>::value) return ((x & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
    return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
template <class E>
__device__ __forceinline__ uint32_t finite_only(uint32_t x) {
    return x & ~((unfinite_signs<E>(x) >> 15) * 0xffffu);
}
// x * 0 + sum: NaN from the first x on that is not finite.
template <class E>
__device__ __forceinline__ uint32_t taint(uint32_t x, uint32_t sum) {
    uint32_t r;
    if constexpr (std::is_same<E, __half>::value)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
    return r;
}

// Keys [every0, every1): those of the sequence that all rows of a part see (every1 may be the smaller one).
__device__ __forceinline__ void keys_of_all(const AttnParams& p, const AttnPart& a, int32_t& every0, int32_t& every1) {
    const int64_t pos = a.pos0;
    every0 = p.window ? static_cast<int32_t>(max(pos + a.tokens - p.window, int64_t{0})) : 0;
    every1 = p.causal ? static_cast<int32_t>(min(max(pos + 1, int64_t{0}), static_cast<int64_t>(a.keys))) : a.keys;
}
// Whether all rows see what the sequence has of keys [key, key + n).
__device__ __forceinline__ bool seen_by_all(const AttnPart& a, int64_t key, int n, int32_t every0, int32_t every1) {
    return key >= a.keys || (key >= every0 && (every1 == a.keys || key + n <= every1));
}
// How many of the tile's 128 keys the sequence has.
__device__ __forceinline__ int held_of(const AttnPart& a, int32_t tile) {
    return static_cast<int>(min(a.keys - static_cast<int64_t>(tile) * 128, int64_t{128}));
}
// The tile's blocks of 32 keys that some row does not see whole, a bit each.
__device__ __forceinline__ uint32_t cut_blocks(const AttnPart& a, int32_t tile, int32_t every0, int32_t every1) {
    uint32_t cut = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (!seen_by_all(a, static_cast<int64_t>(tile) * 128 + 32 * b, 32, every0, every1)) cut |= 1u << b;
    return cut;
}

// What rows get of the values that are not finite among those that they see, from the cache itself: by a warp, its lanes' rows (row:
// there is one, with keys) against `tiles`.  It is added to a row's result, in blocks of keys that some row does not see whole (in
// others the products have taken it), or takes its place (kInstead: the rows of lanes 0, 4, 8 ..).  A seen value counts however small
// its weight is.  A lane has two neighbouring channels of each 64; of 32 keys it notes, a bit a key, where they are infinite of either
// sign (NaN: both), which answers for all rows: a block takes some thousand cycles whatever it holds.
template <class E, bool kInstead>
__device__ __forceinline__ void add_unfinite(const AttnParams& p, const AttnPart& a, bool row, int t, int g, int32_t lo, int32_t hi, int2 tiles,
                                             int32_t block, int lane) {
    constexpr uint32_t kMantissa = std::is_same<E, __half>::value ? 0x03ffu : 0x007fu;
    const int D = p.c.head_dim;
    uint64_t placed = 0;           // kInstead: channels whose results have been replaced, 8 bits a row
    uint32_t all_pos[4]{}, all_neg[4]{};  // kInstead: channels that keys of all rows make infinite, by the signs of a lane's pairs
    // Row r (a lane's) gets infinities in the channels that the bits name.
    auto give = [&](int r, uint32_t up, uint32_t down) {
        if (!__any_sync(~0u, (up | down) != 0)) return;
        const RowOut<E> out = row_out<E>(p, a, block, __shfl_sync(~0u, t, r), __shfl_sync(~0u, g, r));
        bool over = true;          // all of the row is NaN, and nothing changes that
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int d = 2 * lane + 64 * (c / 2) + c % 2;
            if (d >= D) break;
            const bool plus = up >> c & 1, minus = down >> c & 1;
            const uint64_t bit = 1ull << (2 * (r & 28) + c);
            float now = out.o ? wide16(out.o[d]) : out.part[d];
            if (plus || minus) {
                const float x = plus && minus ? __int_as_float(0x7fffffff) : plus ? INFINITY : -INFINITY;
                now = kInstead && !(placed & bit) ? x : now + x;
                placed |= bit;
                if (out.o)
                    out.o[d] = narrow16<E>(now);
                else
                    out.part[d] = now;
            }
            over &= now != now && (!kInstead || (placed & bit));
        }
        if (__all_sync(~0u, over) && lane == r) row = false;
    };
    if (!__any_sync(~0u, row)) return;
    int32_t every0, every1;
    keys_of_all(p, a, every0, every1);
    __syncwarp();  // the rows' other results are there for all lanes
    for (int64_t key0 = static_cast<int64_t>(tiles.x) * 128; key0 < static_cast<int64_t>(tiles.y) * 128; key0 += 32) {
        const bool whole = seen_by_all(a, key0, 32, every0, every1);
        if (!kInstead && whole) continue;
        const int64_t key = key0 + lane;
        const int first = static_cast<int>(min(max(lo - key0, int64_t{0}), int64_t{32})), end = static_cast<int>(min(max(hi - key0, int64_t{0}), int64_t{32}));
        const uint32_t seen = row ? low_bits(end) & ~low_bits(first) : 0u, some = __reduce_or_sync(~0u, seen);
        int64_t at = -1;  // where the key's values are
        if (some >> lane & 1 && key < a.keys) {
            const int32_t i = static_cast<int32_t>(key) / p.b.page_tokens, slot = static_cast<int32_t>(key) - i * p.b.page_tokens;
            const int32_t page = p.b.table[static_cast<int64_t>(a.table_row) * p.b.max_pages + i];
            if (page >= 0 && page < p.b.n_pages) at = page * p.c.v_page_stride + slot * p.c.v_token_stride + a.kv_head * p.c.v_head_stride;
        }
        // Of keys i0 .., the pair of channels from d on; rows are multiples of 4 bytes here.  All loads go out at once: what is not there
        // reads the cache's first pair, and is dropped.
        const uint32_t there = __ballot_sync(~0u, at >= 0);
        at = max(at, int64_t{0});
        auto load = [&](auto& x, int i0, int d) {
            constexpr int kLoads = static_cast<int>(sizeof(x) / 4);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                x[i] = *reinterpret_cast<const volatile uint32_t*>(static_cast<const E*>(p.c.v) + __shfl_sync(~0u, at, i0 + i) + (d < D ? d : 0));
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (d >= D || !(there >> (i0 + i) & 1)) x[i] = 0;
        };
        if (kInstead && whole) {
            bool nan = true;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (64 * c >= D) break;
#pragma unroll 1
                for (int i0 = 0; i0 < 32; i0 += 16) {
                    uint32_t x[16];
                    load(x, i0, 2 * lane + 64 * c);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t bad = unfinite_signs<E>(x[i]), is_nan = (x[i] & (kMantissa | kMantissa << 16)) + 0x7fff7fffu;
                        all_pos[c] |= bad & (~x[i] | is_nan);
                        all_neg[c] |= bad & (x[i] | is_nan);
                    }
                }
                if (2 * lane + 64 * c < D) nan &= (all_pos[c] & all_neg[c]) == 0x80008000u;
            }
            if (__all_sync(~0u, nan)) break;
            continue;
        }
        uint32_t pos[8]{}, neg[8]{};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (64 * c >= D) break;
#pragma unroll 1
            for (int i0 = 0; i0 < 32; i0 += 8) {
                if (!(some >> i0 & 0xffu)) continue;
                uint32_t x[8];
                load(x, i0, 2 * lane + 64 * c);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t bad = unfinite_signs<E>(x[i]);
                    if (!bad) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t v = x[i] >> (16 * h) & 0xffffu, bit = bad >> (15 + 16 * h) & 1u;
                        const bool nan = v & kMantissa;
                        if (nan || !(v & 0x8000u)) pos[2 * c + h] |= bit << (i0 + i);
                        if (nan || (v & 0x8000u)) neg[2 * c + h] |= bit << (i0 + i);
                    }
                }
            }
        }
        for (unsigned rows = __ballot_sync(~0u, seen != 0); rows; rows &= rows - 1) {
            const int r = __ffs(rows) - 1;
            const uint32_t keys = __shfl_sync(~0u, seen, r);
            uint32_t up = 0, down = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (pos[c] & keys) up |= 1u << c;
                if (neg[c] & keys) down |= 1u << c;
            }
            give(r, up, down);
        }
        if (!__any_sync(~0u, row)) return;
    }
    if (kInstead) {
        uint32_t up = 0, down = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            up |= (all_pos[c / 2] >> (15 + 16 * (c % 2)) & 1u) << c;
            down |= (all_neg[c / 2] >> (15 + 16 * (c % 2)) & 1u) << c;
        }
        for (unsigned rows = __ballot_sync(~0u, row); rows; rows &= rows - 1) give(__ffs(rows) - 1, up, down);
    }
}

// Notes a unit that later blocks go on with, so that the join comes to its rows.
__device__ __forceinline__ void note_cut(const AttnParams& p, const AttnPart& a, int32_t block, const AttnWalk& walk) {
    if (a.tile0 == a.first && a.tile1 < a.last) attn_note_join(p, a, block, walk.at.share);
}

// A row's result without keys (zero), or after a wait that ran out (NaN).
template <class E>
__device__ __forceinline__ void fill_row(const AttnParams& p, const AttnPart& a, int t, int g, float value, int32_t block) {
    const RowOut<E> out = row_out<E>(p, a, block, t, g);
    for (int d = 0; d < p.c.head_dim; ++d) {
        if (out.o)
            out.o[d] = narrow16<E>(value);
        else
            out.part[d] = value;
    }
    if (out.lse) *out.lse = value == 0.f ? -INFINITY : value;
    if (out.ml) *out.ml = make_float2(value == 0.f ? -INFINITY : 0.f, value);
}

// A row of products issued from a converged warp, one lane chosen once: kSteps steps of 16 channels of row tiles and keys (chunks of 64
// channels, 16 KB each), and four steps of 16 keys of weights and values.  (Issued one by one, each with an election of its own
// and its descriptors made in between, they cost the issuing warp more time than the tensor cores.)
template <int kSteps>
__device__ __forceinline__ void issue_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc, uint32_t add) {
    if constexpr (kSteps == 8)
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.eq.b32 t, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 1024;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 1026;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 1028;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 1030;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "}"
            ::"r"(d), "l"(q), "l"(k), "r"(idesc), "r"(add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.eq.b32 t, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "}"
            ::"r"(d), "l"(q), "l"(k), "r"(idesc), "r"(add)
            : "memory");
}
__device__ __forceinline__ void issue_values(uint32_t d, uint32_t w, uint64_t v, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "}"
        ::"r"(d), "r"(w), "l"(v), "r"(idesc), "r"(add)
        : "memory");
}

// ------------------------------------------------------------------------------------------------ warp 0: work and copies
template <class S, int kStreams>
__device__ void produce(const TcParams& p, const CUtensorMap* map_q, const CUtensorMap* map_k, const CUtensorMap* map_v, Misc<S>& sh,
                        uint8_t* q_s, uint8_t* kv_s, int lane) {
    const AttnParams& ap = p.a;
    const int32_t pt = ap.b.page_tokens;
    int32_t* status = ap.b.device_status;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, &sh.abort, status, p.wait_cycles); };
    AttnWalk walk;
    walk.begin(sh.scan.start);
    AttnPart a{};
    uint32_t n = 0, qn = 0, err = 0;
    bool ok = true;

    // Lane i: the page of box i of the `span` tiles from `tile` on, and the box's first token in it; loaded well before it is used.
    const int span = 32 / p.boxes;
    struct Boxes {
        int32_t page, token;
        bool inside;               // before the sequence's end
    };
    auto look_up = [&](int32_t tile) {
        Boxes x{0, 0, false};
        const int64_t key = static_cast<int64_t>(tile) * S::kKeys + lane * p.box_keys;
        if (key < a.keys && tile + lane / p.boxes < a.tile1) {
            const int32_t i = static_cast<int32_t>(key) / pt;
            x.inside = true;
            x.token = static_cast<int32_t>(key) - i * pt;
            x.page = ap.b.table[static_cast<int64_t>(a.table_row) * ap.b.max_pages + i];
        }
        return x;
    };
    // What is behind the sequence or has no page is fetched from behind the cache's end, which reads as zeros.
    auto settle = [&](Boxes& x) {
        const bool bad = x.inside && (x.page < 0 || x.page >= ap.b.n_pages);
        if (!x.inside || bad) x.page = ap.b.n_pages;
        if (bad) err |= GDN_PAGES_ERR_PAGE;
        return ~__ballot_sync(~0u, bad);  // boxes that have a page, or need none
    };
    // Tile i of the span.
    auto load_half = [&](const CUtensorMap* map, const Boxes& x, uint32_t mask, int i, int half) {
        const uint32_t st = n % S::kStages, use = n / S::kStages;
        if (use > 0 && !wait(sh.kv_empty + st, (use - 1) & 1)) return false;
        if (elect_one()) {
            sh.stage_keys[st] = mask == ~0u ? make_uint4(~0u, ~0u, ~0u, ~0u) : spread_boxes(mask >> (i * p.boxes), p.boxes, p.box_keys);
            mbar_arrive_expect_tx(sh.kv_full + st, S::kKvBytes);
        }
        __syncwarp();
        const int b = lane / S::kChunks, c = lane % S::kChunks;  // at most 16 boxes of 2 chunks
        const int32_t page = __shfl_sync(~0u, x.page, (i * p.boxes + b) & 31), token = __shfl_sync(~0u, x.token, (i * p.boxes + b) & 31);
        if (b < p.boxes)
            tma_load_4d(kv_s + st * S::kKvBytes + c * (S::kKeys * 128) + b * p.box_keys * 128, map, sh.kv_full + st,
                        (half * S::kChunks + c) * 64, token, a.kv_head, page);
        __syncwarp();
        ++n;
        return true;
    };
    auto load = [&](const CUtensorMap* map, const Boxes& x, uint32_t mask, int i) {
        for (int half = 0; half < S::kHalves; ++half)
            if (!load_half(map, x, mask, i, half)) return false;
        return true;
    };

    for (uint32_t k = 0; ok; ++k) {
        const bool more = walk.next(ap, a);
        if (!more) a.tokens = 0;
        if (k >= kParts && !wait(sh.part_empty + k % kParts, (k / kParts - 1) & 1)) break;
        if (elect_one()) {
            sh.parts[k % kParts] = a;
            mbar_arrive(sh.part_full + k % kParts);
        }
        __syncwarp();
        if (!more) break;
        if (lane == 0) note_cut(ap, a, blockIdx.x, walk);
        if (a.first == a.last) continue;
        const uint32_t slot = qn % S::kQSlots, use = qn / S::kQSlots;
        if (use > 0 && !wait(sh.q_empty + slot, (use - 1) & 1)) break;
        const int active = a.tokens > p.row_tokens ? kStreams : 1;
        if (elect_one()) {
            constexpr int kAll = S::kHalves * S::kChunks;
            const int times = p.quarters ? 4 : active;  // the same rows in every quarter, or a stream's own
            mbar_arrive_expect_tx(sh.q_full + slot, times * kAll * ap.group * p.row_tokens * 128);
            for (int s = 0; s < times; ++s)
#pragma unroll
                for (int c = 0; c < kAll; ++c)
                    tma_load_3d(q_s + slot * S::kQBytes + s * (p.quarters ? 32 * 128 : S::kQBytes) + c * (kRowTile * 128), map_q,
                                sh.q_full + slot, c * 64, a.head0, static_cast<int32_t>(a.row0 + (p.quarters ? 0 : s * p.row_tokens)));
        }
        __syncwarp();
        ++qn;
        // Two spans of pages: the one that keys are fetched from (kStreams == 1: a tile ahead of the values), and the next one.
        Boxes ahead = look_up(a.tile0), keys = ahead, vals = ahead;
        uint32_t key_mask = 0, val_mask = 0;
        auto load_keys = [&](int32_t j) {
            const int i = j % span;
            if (i == 0) {
                keys = ahead;
                ahead = look_up(a.tile0 + j + span);
                key_mask = settle(keys);
            }
            return load(map_k, keys, key_mask, i);
        };
        const int32_t tiles = a.tile1 - a.tile0;
        if (kStreams == 1) ok = load_keys(0);
        for (int32_t j = 0; ok && j < tiles; ++j) {
            if (kStreams == 2) ok = load_keys(j);
            if (j % span == 0) {  // the values' pages are those of the keys, before these go on
                vals = keys;
                val_mask = key_mask;
            }
            if (kStreams == 1 && j + 1 < tiles) ok = load_keys(j + 1);
            ok = ok && load(map_v, vals, val_mask, j % span);
        }
    }
    kv_report(status, err);
    // No copy may be under way when the block ends: another warp's wait may run out after this one has gone through.
    const long long t0 = clock64();
    auto settled = [&](uint64_t* bar, uint32_t parity) {
        while (!mbar_try_wait(bar, parity) && clock64() - t0 < kWaitCycles / 4) {
        }
    };
    for (uint32_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i) settled(sh.kv_full + i % S::kStages, i / S::kStages & 1);
    for (uint32_t i = qn > S::kQSlots ? qn - S::kQSlots : 0; i < qn; ++i) settled(sh.q_full + i % S::kQSlots, i / S::kQSlots & 1);
}

// ------------------------------------------------------------------------------------------------ warps 0 and 3: plain copies
// `bytes` (16, 8 or 4) from global to shared memory, asynchronously, or zeros.
__device__ __forceinline__ void copy_piece(int bytes, uint8_t* dst, const void* src, bool there) {
    if (bytes == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 8 : 0) : "memory");
    else if (bytes == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// What produce does, without tiled copies: warp `id` (0 or 1) brings its half of the rows, 64 threads arrive at a stage.  Copies of
// kAhead stages are under way at a time; a thread waits for its own, makes them visible to the tensor cores and arrives.
template <class E, class S, int kStreams>
__device__ void produce_plain(const TcParams& p, Misc<S>& sh, uint8_t* q_s, uint8_t* kv_s, int id, int lane) {
    constexpr int kAhead = 2;
    const int bytes = p.plain, elems = bytes / 2;
    const AttnParams& ap = p.a;
    const int D = ap.c.head_dim;
    int32_t* status = ap.b.device_status;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, &sh.abort, status, p.wait_cycles); };
    AttnWalk walk;
    walk.begin(sh.scan.start);
    AttnPart a{};
    uint32_t n = 0, told = 0, qn = 0, err = 0;  // stages begun and handed over; units
    bool ok = true;

    auto tell = [&](uint32_t upto) {  // all but the last stages' copies are there
        for (; told < upto; ++told) mbar_arrive(sh.kv_full + told % S::kStages);
    };
    auto flush = [&]() {
        cp_async_wait<0>();
        fence_proxy_async_smem();
        tell(n);
    };
    // Page and place of this warp's keys of a tile; the bits of those that have one or need none.
    auto look_up = [&](int32_t tile, uint32_t (&bits)[2]) {
        __syncwarp();  // the places it overwrites have been read
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t key = static_cast<int64_t>(tile) * S::kKeys + 64 * id + 32 * h + lane;
            int2 at = make_int2(-1, 0);
            bool bad = false;
            if (key < a.keys) {
                const int32_t i = static_cast<int32_t>(key) / ap.b.page_tokens;
                at = make_int2(ap.b.table[static_cast<int64_t>(a.table_row) * ap.b.max_pages + i], static_cast<int32_t>(key) - i * ap.b.page_tokens);
                bad = at.x < 0 || at.x >= ap.b.n_pages;
                if (bad) at.x = -1;
            }
            if (bad) err |= GDN_PAGES_ERR_PAGE;
            sh.rows[id][tile & 1][32 * h + lane] = at;
            bits[h] = ~__ballot_sync(~0u, bad);
        }
        __syncwarp();
    };
    auto load = [&](bool values, int32_t tile, const uint32_t (&bits)[2]) {
        const E* base = static_cast<const E*>(values ? ap.c.v : ap.c.k) + a.kv_head * (values ? ap.c.v_head_stride : ap.c.k_head_stride);
        const int64_t page = values ? ap.c.v_page_stride : ap.c.k_page_stride, token = values ? ap.c.v_token_stride : ap.c.k_token_stride;
        for (int half = 0; half < S::kHalves; ++half) {
            const uint32_t st = n % S::kStages, use = n / S::kStages;
            if (use > 0 && !wait(sh.kv_empty + st, (use - 1) & 1)) return false;
            if (lane == 0) {
                uint32_t* w = reinterpret_cast<uint32_t*>(sh.stage_keys + st) + 2 * id;
                w[0] = bits[0];
                w[1] = bits[1];
            }
            const int pieces = (min(D - half * 128, 128) + elems - 1) / elems;
            for (int r = lane / 8; r < 64; r += 4) {  // eight lanes a row
                const int2 at = sh.rows[id][tile & 1][r];
                const E* src = base + max(at.x, 0) * page + at.y * token + half * 128;
                const int row = 64 * id + r;
                for (int i = lane % 8; i < pieces; i += 8) {
                    const int x = i * bytes % 128, c = i * bytes / 128;
                    copy_piece(bytes, kv_s + st * S::kKvBytes + c * (S::kKeys * 128) + sw128_offset(row, x / 16) + x % 16, src + i * elems, at.x >= 0);
                }
            }
            cp_async_commit();
            ++n;
            cp_async_wait<kAhead>();
            fence_proxy_async_smem();
            if (n > kAhead) tell(n - kAhead);
        }
        return true;
    };

    for (uint32_t k = 0; ok; ++k) {
        const bool more = walk.next(ap, a);
        if (!more) a.tokens = 0;
        if (id == 0) {
            if (k >= kParts && !wait(sh.part_empty + k % kParts, (k / kParts - 1) & 1)) break;
            if (lane == 0) {
                sh.parts[k % kParts] = a;
                mbar_arrive(sh.part_full + k % kParts);
                if (more) note_cut(ap, a, blockIdx.x, walk);
            }
            __syncwarp();
        }
        if (!more) break;
        if (a.first == a.last) continue;
        const uint32_t slot = qn % S::kQSlots, use = qn / S::kQSlots;
        if (use > 0 && !wait(sh.q_empty + slot, (use - 1) & 1)) break;
        const int active = a.tokens > p.row_tokens ? kStreams : 1, pieces = D / elems, padded = S::kHalves * p.k_steps * 16 / elems;
        for (int s = 0; s < active; ++s) {
            for (int r = id * 4 + lane / 8; r < p.row_tokens * ap.group; r += 8) {
                const int t = r / ap.group, g = r - t * ap.group, token = s * p.row_tokens + t;
                const bool there = token < a.tokens && g < a.heads;
                const E* src = static_cast<const E*>(ap.q) + (a.row0 + (there ? token : 0)) * ap.q_stride + static_cast<int64_t>(a.head0 + (there ? g : 0)) * D;
                for (int i = lane % 8; i < padded; i += 8) {  // zeros behind the head's end: joined quarters leave anything there
                    const int x = i * bytes % 128, c = i * bytes / 128;
                    const bool in = there && i < pieces;
                    uint8_t* to = q_s + (slot + s) * S::kQBytes + c * (kRowTile * 128) + sw128_offset(r, x / 16) + x % 16;
                    for (int w = 0; w < (p.quarters ? 4 : 1); ++w) copy_piece(bytes, to + w * (32 * 128), in ? src + i * elems : src, in);
                }
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(sh.q_full + slot);
        ++qn;
        uint32_t now[2], then[2] = {~0u, ~0u};
        look_up(a.tile0, now);
        if (kStreams == 1) ok = load(false, a.tile0, now);
        for (int32_t tile = a.tile0; ok && tile < a.tile1; ++tile) {
            const bool next = tile + 1 < a.tile1;
            if (kStreams == 2) ok = load(false, tile, now);
            if (next) look_up(tile + 1, then);
            if (kStreams == 1 && next) ok = load(false, tile + 1, then);
            ok = ok && load(true, tile, now);
            now[0] = then[0];
            now[1] = then[1];
        }
        flush();  // before any wait for this part's end: it ends with these stages
    }
    flush();  // after a wait that ran out: no copy may be under way when the block ends
    kv_report(status, err);
}

// A weight of zero makes nothing of a value only if that is finite.  So the products must not see what the page of a sequence's last
// tile holds behind the sequence (rows from `held` on: anything), nor, in blocks of 32 keys of which some row does not see all,
// values that are not finite: these become zero in shared memory, and reach the rows that see them by add_unfinite.  By a whole warp,
// eight lanes a row of a chunk, four rows at a time.  It runs once or twice a unit, between code that fills the instruction cache: short
// loops, with four loads at a time (8 prompts, heads of 256: 1581 us; unrolled over 32 rows 1611, with a test before each load 1886).
template <class S>
__device__ __forceinline__ uint4* stage_rows(uint8_t* stage, int chunk, int row, int lane) {
    return reinterpret_cast<uint4*>(stage + chunk * (S::kKeys * 128) + row * 128 + lane * 16);
}
// Clears the rows behind the end; returns whether the blocks hold values that are not finite.
template <class E, class S>
__device__ __forceinline__ bool settle_values(uint8_t* stage, int held, uint32_t blocks, int lane) {
    uint32_t sum[4]{};
#pragma unroll 1
    for (int c = 0; c < S::kChunks; ++c) {
        if (held < S::kKeys) {
            uint4 *at = stage_rows<S>(stage, c, held & ~3, lane), *end = stage_rows<S>(stage, c, S::kKeys, 0);
            if (lane / 8 >= (held & 3)) *at = make_uint4(0, 0, 0, 0);
#pragma unroll 1
            for (at += 32; at < end; at += 32) *at = make_uint4(0, 0, 0, 0);
        }
#pragma unroll 1
        for (int i0 = blocks ? 0 : S::kKeys; i0 < S::kKeys; i0 += 16) {
            if (!(blocks >> (i0 / 32) & 1)) continue;
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *stage_rows<S>(stage, c, i0 + 4 * i, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum[0] = taint<E>(x[i].x, sum[0]), sum[1] = taint<E>(x[i].y, sum[1]), sum[2] = taint<E>(x[i].z, sum[2]), sum[3] = taint<E>(x[i].w, sum[3]);
        }
    }
    return __any_sync(~0u, (unfinite_signs<E>(sum[0]) | unfinite_signs<E>(sum[1]) | unfinite_signs<E>(sum[2]) | unfinite_signs<E>(sum[3])) != 0);
}
// Makes them zero, in every `of`-th group of four rows.
template <class E, class S>
__device__ __forceinline__ void set_apart(uint8_t* stage, int first, int of, uint32_t blocks, int lane) {
#pragma unroll 1
    for (int c = 0; c < S::kChunks; ++c)
#pragma unroll 1
        for (int i = 4 * first; i < S::kKeys; i += 4 * of) {
            if (!(blocks >> (i / 32) & 1)) continue;
            uint4* at = stage_rows<S>(stage, c, i, lane);
            const uint4 x = *at;
            *at = make_uint4(finite_only<E>(x.x), finite_only<E>(x.y), finite_only<E>(x.z), finite_only<E>(x.w));
        }
}

// ------------------------------------------------------------------------------------------------ warps 1 and 2: products
// A warp a stream.  All of it goes through this converged, so that addresses and descriptors stay in uniform registers; one lane issues.
// What a warp issues completes in order, so that a product may overwrite the S whose P an earlier one reads.  (One warp for both
// streams was what bound the kernel: waits, barriers and bookkeeping between two rows of products cost it more than the products.)
template <class E, class S, int kStreams>
__device__ void multiply(const TcParams& p, Misc<S>& sh, uint8_t* q_s, uint8_t* kv_s, uint32_t tmem, int stream, int lane) {
    int32_t* status = p.a.b.device_status;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, &sh.abort, status, p.wait_cycles); };
    const uint64_t dq0 = desc_kmajor_sw128(smem_u32(q_s) + stream * S::kQBytes), dk0 = desc_kmajor_sw128(smem_u32(kv_s));
    const uint64_t dv0 = desc_mnmajor_sw128(smem_u32(kv_s), S::kKeys * 128);
    const bool full = p.k_steps == S::kChunks * 4;
    const uint32_t o_at = tmem + S::kTmemO + stream * 128;
    uint32_t st = 0, ph = 0, qn = 0, g = 0, seen = 0, turns = 0;  // stage and its phase; units; tiles
    uint32_t met = 0;  // meetings of the two warps

    auto arrived = [&]() { return wait(sh.kv_full + st, ph); };
    auto arrived_next = [&]() { return st + 1 == S::kStages ? wait(sh.kv_full, ph ^ 1) : wait(sh.kv_full + st + 1, ph); };
    // The two warps take turns, so that the tensor cores finish one stream's products while the other's exponentials are computed;
    // first come, first served, they end up in step, with both waiting for either.
    auto turn = [&]() {
        const bool mine = stream == 0 && turns == 0;
        const uint32_t phase = turns++ - (stream == 0 ? 1 : 0);
        return mine || wait(sh.turn + stream, phase & 1);
    };
    auto pass = [&]() {
        if (lane == 0) mbar_arrive(sh.turn + 1 - stream);
        __syncwarp();
    };
    auto advance = [&]() {
        if (++st == S::kStages) {
            st = 0;
            ph ^= 1;
        }
    };
    // S in slot `slot` (+)= row tile q times the keys of the present stage; with the last half the slot's mask goes along.
    auto scores = [&](int slot, uint32_t q, int half) {
        const uint4 keys = sh.stage_keys[st];
        const uint64_t dq = dq0 + (q * S::kQBytes + half * (S::kChunks * kRowTile * 128)) / 16, dk = dk0 + st * (S::kKvBytes / 16);
        if (full)
            issue_scores<S::kChunks * 4>(tmem + slot * 128, dq, dk, p.idesc_qk, half > 0);
        else
            for (int i = 0; i < p.k_steps; ++i)
                mma_ss_elect(tmem + slot * 128, dq + (i / 4) * 1024 + (i % 4) * 2, dk + (i / 4) * 1024 + (i % 4) * 2, p.idesc_qk, i > 0);
        if (half == S::kHalves - 1) {
            mma_commit_elect(sh.s_full + slot);
            if (lane == 0) {
                const uint32_t missing = ~(keys.x & keys.y & keys.z & keys.w);
                sh.slot_missing[slot] = missing;
                if (missing) sh.slot_keys[slot] = keys;
                mbar_arrive(sh.s_full + slot);
            }
            __syncwarp();
        }
        mma_commit_elect(sh.kv_empty + st);
    };
    // O (+)= P in slot `slot`, the first or the last 64 keys of it, times the values of the present stage.
    auto values = [&](int slot, int half, int keys64, bool add) {
        issue_values(o_at + half * 128, tmem + slot * 128 + keys64 * 32, dv0 + st * (S::kKvBytes / 16) + keys64 * (64 * 128 / 16), p.idesc_pv, add);
    };
    auto skip = [&]() {  // a stage that this stream has no use for
        if (lane == 0) mbar_arrive(sh.kv_empty + st);
        __syncwarp();
    };
    auto meet = [&]() {  // the two warps
        __syncwarp();
        if (kStreams == 1) return true;
        if (lane == 0) mbar_arrive(&sh.both);
        return wait(&sh.both, met++ & 1);
    };
    // The values of a stage become as a product may have them, while the tile's exponentials are under way.  Each warp looks through
    // the blocks on its own; only where they hold what has to be set apart the two meet, before one of them changes what the other
    // may still have to read.
    auto settle = [&](int held, uint32_t blocks, bool& found) {
        uint8_t* tile = kv_s + st * S::kKvBytes;
        found = settle_values<E, S>(tile, held, blocks, lane);
        if (found) {
            if (!meet()) return false;
            set_apart<E, S>(tile, stream, kStreams, blocks, lane);
        }
        fence_proxy_async_smem();
        __syncwarp();
        return !found || meet();
    };
    auto run = [&]() {
        for (uint32_t k = 0;; ++k) {
            if (!wait(sh.part_full + k % kParts, k / kParts & 1)) return;
            const AttnPart a = sh.parts[k % kParts];
            __syncwarp();
            if (lane == 0) mbar_arrive(sh.part_empty + k % kParts);
            __syncwarp();
            if (a.tokens == 0) return;
            if (a.first == a.last) continue;
            const uint32_t slot = qn % S::kQSlots;
            if (!wait(sh.q_full + slot, qn / S::kQSlots & 1)) return;
            ++qn;
            const int32_t count = a.tile1 - a.tile0;
            int32_t every0, every1;
            keys_of_all(p.a, a, every0, every1);
            // tiles that need nothing: all rows see all of their keys, and the sequence has them all
            const int32_t whole0 = static_cast<int32_t>((static_cast<int64_t>(every0) + S::kKeys - 1) / S::kKeys) - a.tile0, whole1 = every1 / S::kKeys - a.tile0;
            int2 unfinite = make_int2(0x7fffffff, 0);
            auto settle_tile = [&](int32_t j) {
                if (j >= whole0 && j < whole1) return true;
                const int32_t tile = a.tile0 + j;
                bool found = false;
                if (!settle(held_of(a, tile), cut_blocks(a, tile, every0, every1), found)) return false;
                if (found) unfinite = make_int2(min(unfinite.x, tile), tile + 1);
                return true;
            };
            // The part's last product is out (kStreams == 1: one product more): told with the tiles that had values set apart.
            auto tell_done = [&](int slot, bool last) {
                if (lane == 0) {
                    if (last) sh.unfinite(stream, qn) = unfinite;
                    mbar_arrive(sh.pv_done + slot);
                }
                __syncwarp();
                mma_commit_elect(sh.pv_done + slot);
            };
            if constexpr (kStreams == 2) {
                const int32_t end = stream_end(p, a, stream, S::kKeys) - a.tile0;
                if (!arrived() || !turn()) return;
                tc_fence_after();
                if (end > 0)
                    scores(stream, 0, 0);
                else
                    skip();
                pass();
                if (count == 1) mma_commit_elect(sh.q_empty);
                advance();
                for (int32_t j = 0; j < count; ++j) {
                    const bool next = j + 1 < count;
                    if (!arrived()) return;
                    if (!settle_tile(j)) return;
                    if (next && !arrived_next()) return;
                    if (j < end && !wait(sh.p_half + stream, seen & 1)) return;
                    if (!turn()) return;
                    if (j < end) {
                        tc_fence_after();
                        values(stream, 0, 0, j > 0);
                        if (!wait(sh.p_full + stream, seen++ & 1)) return;
                        tc_fence_after();
                        values(stream, 0, 1, true);
                        if (j + 1 == end) tell_done(stream, true);
                        mma_commit_elect(sh.kv_empty + st);
                    } else {
                        skip();
                    }
                    advance();
                    if (next) {
                        if (j + 1 < end)
                            scores(stream, 0, 0);
                        else
                            skip();
                        if (j + 2 == count) mma_commit_elect(sh.q_empty);
                        advance();
                    }
                    pass();
                }
            } else {
                auto all_scores = [&](int s_slot) {
                    for (int half = 0; half < S::kHalves; ++half) {
                        if (!arrived()) return false;
                        tc_fence_after();
                        scores(s_slot, slot, half);
                        advance();
                    }
                    return true;
                };
                if (!all_scores(g & 1)) return;
                if (count == 1 && !p.quarters) mma_commit_elect(sh.q_empty + slot);  // quarters: when their results are joined there
                for (int32_t j = 0; j < count; ++j, ++g) {
                    if (j + 1 < count && !all_scores((g + 1) & 1)) return;
                    if (j + 2 == count && !p.quarters) mma_commit_elect(sh.q_empty + slot);
                    for (int half = 0; half < S::kHalves; ++half) {
                        if (!arrived()) return;
                        if (!settle_tile(j)) return;
                        for (int h = 0; h < 2; ++h) {
                            if (half == 0 && !wait((h ? sh.p_full : sh.p_half) + (g & 1), g / 2 & 1)) return;
                            tc_fence_after();
                            values(g & 1, half, h, h > 0 || j > 0);
                        }
                        if (half == S::kHalves - 1) tell_done(g & 1, j + 1 == count);
                        mma_commit_elect(sh.kv_empty + st);
                        advance();
                    }
                }
            }
        }
    };
    run();
    __syncwarp();
    mma_commit_elect(sh.drain + stream);  // no product may be under way when TMEM is given back
    mbar_wait(sh.drain + stream, 0);
}

// ------------------------------------------------------------------------------------------------ warps 4..: exponentials, results
template <class E, class S, int kDim, int kStreams>
__device__ void exponentiate(const TcParams& p, Misc<S>& sh, uint32_t tmem, int stream, int warp, int lane, int32_t block) {
    constexpr float kOffset = weight_offset<E>();
    const AttnParams& ap = p.a;
    const int D = ap.c.head_dim;
    int32_t* status = ap.b.device_status;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, &sh.abort, status, p.wait_cycles); };
    const int row = warp * 32 + lane, tile_t = row / ap.group, g = row - tile_t * ap.group, t = stream * p.row_tokens + tile_t;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t o_at = tmem + lanes + S::kTmemO + stream * 128;
    uint32_t count = 0, done = 0, units = 0;  // tiles, and parts with tiles, of this stream so far; parts with tiles of either
    uint32_t k = 0;
    bool ok = true;
    for (; ok; ++k) {
        ok = wait(sh.part_full + k % kParts, k / kParts & 1);
        if (!ok) break;
        const AttnPart a = sh.parts[k % kParts];
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.part_empty + k % kParts);
        if (a.tokens == 0) break;
        const bool mine = tile_t < p.row_tokens && t < a.tokens && g < a.heads;
        if (a.first == a.last) {
            if (mine) fill_row<E>(ap, a, t, g, 0.f, block);
            continue;
        }
        ++units;
        const int64_t pos = static_cast<int64_t>(a.pos0) + t;
        const int32_t hi = ap.causal ? static_cast<int32_t>(min(max(pos + 1, int64_t{0}), static_cast<int64_t>(a.keys))) : a.keys;
        const int32_t lo = ap.window ? static_cast<int32_t>(max(pos - ap.window + 1, int64_t{0})) : 0;
        const bool live = __any_sync(~0u, mine);
        // tiles that every row of this warp sees whole: [clean0, clean1)
        const int32_t clean0 = __reduce_max_sync(~0u, mine ? static_cast<int32_t>((static_cast<int64_t>(lo) + S::kKeys - 1) / S::kKeys) : 0);
        const int32_t clean1 = __reduce_min_sync(~0u, mine ? hi / S::kKeys : 0x7fffffff);
        const int32_t tiles = kStreams == 2 ? stream_end(p, a, stream, S::kKeys) - a.tile0 : a.tile1 - a.tile0;
        float m = -INFINITY, l = 0.f;  // the maximum as used, less the offset; the sum of weights relative to it
        for (int32_t j = 0; j < tiles; ++j, ++count) {
            const uint32_t slot = kStreams == 2 ? stream : count & 1;
            const uint32_t parity = kStreams == 2 ? count & 1 : count / 2 & 1;
            ok = wait(sh.s_full + slot, parity);
            if (!ok) break;
            tc_fence_after();
            if (live) {
                const uint32_t s_at = tmem + lanes + slot * 128;
                uint32_t s[S::kKeys];
#pragma unroll
                for (int c = 0; c < S::kKeys; c += 32) tmem_ld32(s_at + c, s + c);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < S::kKeys; c += 32) tmem_regs_ready32(s + c);
                const uint32_t missing = sh.slot_missing[slot];
                if (a.tile0 + j < clean0 || a.tile0 + j >= clean1) {
                    const int64_t key0 = static_cast<int64_t>(a.tile0 + j) * S::kKeys;
                    const int from = static_cast<int>(max(lo - key0, int64_t{0}));
                    const int upto = static_cast<int>(max(min(hi - key0, static_cast<int64_t>(S::kKeys)), int64_t{0}));
#pragma unroll
                    for (int w = 0; w < S::kKeys; w += 32) {
                        const uint32_t bits = low_bits(upto - w) & ~low_bits(from - w);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(bits >> c & 1)) s[w + c] = 0xff800000u;  // -infinity
                    }
                }
                if (missing) {
#pragma unroll
                    for (int w = 0; w < S::kKeys; w += 32) {
                        const uint32_t bits = reinterpret_cast<const uint32_t*>(sh.slot_keys + slot)[w / 32];
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(bits >> c & 1)) s[w + c] = 0xff800000u;
                    }
                }
                float top[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(s[c]);
#pragma unroll
                for (int c = 4; c < S::kKeys; ++c) top[c % 4] = fmaxf(top[c % 4], __uint_as_float(s[c]));
                const float x = fmaf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), p.scale_log2, -kOffset);
                const bool raise = mine && x > m + kGrowth;
                const bool rescale = __any_sync(~0u, raise);
                float shrink = 1.f;
                if (rescale) {
                    const float now = raise ? x : m;
                    shrink = raise ? exp2_fast(m - now) : 1.f;  // 0 for a row's first keys
                    m = now;
                    l *= shrink;
                    __syncwarp();
                }
                if (j > 0 && rescale) {
                    // With two streams S came after the last product on O; with one it may still be under way.
                    if (kStreams == 1) {
                        ok = wait(sh.pv_done + (count - 1 & 1), (count - 1) / 2 & 1);
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32_wait(o_at + c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
                        tmem_st32(o_at + c, o);
                    }
                }
                const float base = m == -INFINITY ? 0.f : m;
                const uint64_t by = both(p.scale_log2, p.scale_log2), less = both(-base, -base);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        float e[4];
                        split(fma_both(both(__uint_as_float(s[64 * h + c]), __uint_as_float(s[64 * h + c + 1])), by, less), e[0], e[1]);
                        split(fma_both(both(__uint_as_float(s[64 * h + c + 2]), __uint_as_float(s[64 * h + c + 3])), by, less), e[2], e[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) e[i] = exp2_fast(e[i]);
                        sum0 = add_both(sum0, both(e[0], e[1]));
                        sum1 = add_both(sum1, both(e[2], e[3]));
                        w[c / 2] = pack16<E>(e[0], e[1]);
                        w[c / 2 + 1] = pack16<E>(e[2], e[3]);
                    }
                    tmem_st32(s_at + 32 * h, w);
                    if (h == 0) {
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sh.p_half + slot);
                    }
                }
                float s0, s1, s2, s3;
                split(sum0, s0, s1);
                split(sum1, s2, s3);
                l += (s0 + s1) + (s2 + s3);
            }
            if (!ok) break;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (!live) mbar_arrive(sh.p_half + slot);
                mbar_arrive(sh.p_full + slot);
            }
        }
        if (!ok) break;
        if (tiles > 0) {
            // Two streams: a phase a part.  One: a phase a tile, on two barriers in turn: a wait tells a phase only from its neighbours,
            // and the product before the last may be under way, or both may be done.
            ok = kStreams == 1 ? wait(sh.pv_done + (count - 1 & 1), (count - 1) / 2 & 1) : wait(sh.pv_done + stream, done++ & 1);
            if (!ok) break;
            tc_fence_after();
        }
        if (!live) continue;
        const RowOut<E> out = row_out<E>(ap, a, block, t, g);
        const float scale = out.o ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        E* rows4[4]{};             // the rows of this lane's group of four
#pragma unroll
        for (int i = 0; i < 4 && kStreams == 2; ++i)
            rows4[i] = reinterpret_cast<E*>(__shfl_sync(~0u, mine ? reinterpret_cast<unsigned long long>(out.o) : 0ull, (lane & 28) + i));
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            __syncwarp();
            uint32_t o[32];
            if (tiles > 0) {
                tmem_ld32_wait(o_at + c, o);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * scale);
            if (out.o && p.out_vec) {
                uint4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = make_uint4(pack16<E>(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1])),
                                      pack16<E>(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3])),
                                      pack16<E>(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5])),
                                      pack16<E>(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7])));
                if constexpr (kStreams == 1) {  // few rows, most of them nobody's
                    if (mine)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + 8 * i < D) *reinterpret_cast<uint4*>(out.o + c + 8 * i) = x[i];
                    continue;
                }
                // Four lanes swap, so that each writes 16 bytes of the same four rows: 64 bytes of a row at a time (8 prompts: 1494 ->
                // 1445 us).
                swap_quads(x[0], x[1], lane & 1, 1);
                swap_quads(x[2], x[3], lane & 1, 1);
                swap_quads(x[0], x[2], lane & 2, 2);
                swap_quads(x[1], x[3], lane & 2, 2);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rows4[i] && c + 8 * (lane & 3) < D) *reinterpret_cast<uint4*>(rows4[i] + c + 8 * (lane & 3)) = x[i];
            } else if (mine && out.o) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c + i < D) out.o[c + i] = narrow16<E>(__uint_as_float(o[i]));
            } else if (mine && D % 4 == 0) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (c + i < D) *reinterpret_cast<uint4*>(out.part + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            } else if (mine) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c + i < D) out.part[c + i] = __uint_as_float(o[i]);
            }
        }
        __syncwarp();
        tc_fence_before();
        if (mine) {
            if (out.lse) *out.lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            if (out.ml) *out.ml = make_float2(m, l);
        }
        const int2 unfinite = tiles > 0 ? sh.unfinite(stream, units) : make_int2(0, 0);
        if (unfinite.x < unfinite.y) add_unfinite<E, false>(ap, a, mine && l > 0.f, t, g, lo, hi, unfinite, block, lane);
    }
    if (!ok) {  // what a wait that ran out has left undone
        AttnWalk walk;
        walk.begin(sh.scan.start);
        AttnPart a;
        for (uint32_t i = 0; walk.next(ap, a); ++i) {
            if (i < k) continue;
            if (tile_t < p.row_tokens && t < a.tokens && g < a.heads) fill_row<E>(ap, a, t, g, __int_as_float(0x7fffffff), block);
            if (stream == 0 && row == 0) note_cut(ap, a, block, walk);
        }
    }
}

// Few rows: all of a unit's rows lie in every warp's 32 lanes of TMEM, and a warp takes 32 of a tile's 128 keys, with a maximum, a sum
// and a result of its own; the weights of the other keys are zero.  That is a quarter of the work a tile on the one warp that would
// have all rows.  At a part's end the four results are joined in the space of the unit's Q.
template <class E, class S>
__device__ void exponentiate_quarters(const TcParams& p, Misc<S>& sh, uint8_t* q_s, uint32_t tmem, int warp, int lane, int32_t block) {
    constexpr float kOffset = weight_offset<E>();
    const AttnParams& ap = p.a;
    const int D = ap.c.head_dim;
    int32_t* status = ap.b.device_status;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, &sh.abort, status, p.wait_cycles); };
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16, o_at = tmem + lanes + S::kTmemO;
    uint32_t count = 0, qn = 0, mixes = 0, k = 0;
    auto meet = [&]() {  // the four warps
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.mix);
        return wait(&sh.mix, mixes++ & 1);
    };
    // Row r of a part: token, head, and its keys.
    struct Row {
        int t, g;
        int32_t lo, hi;
        bool there;
    };
    auto row_of = [&](const AttnPart& a, int r) {
        Row x;
        x.t = r / ap.group;
        x.g = r - x.t * ap.group;
        x.there = x.t < a.tokens && x.t < p.row_tokens && x.g < a.heads;
        const int64_t pos = static_cast<int64_t>(a.pos0) + x.t;
        x.hi = ap.causal ? static_cast<int32_t>(min(max(pos + 1, int64_t{0}), static_cast<int64_t>(a.keys))) : a.keys;
        x.lo = ap.window ? static_cast<int32_t>(max(pos - ap.window + 1, int64_t{0})) : 0;
        return x;
    };
    bool ok = true;
    for (; ok; ++k) {
        ok = wait(sh.part_full + k % kParts, k / kParts & 1);
        if (!ok) break;
        const AttnPart a = sh.parts[k % kParts];
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.part_empty + k % kParts);
        if (a.tokens == 0) break;
        const Row mine = row_of(a, lane);
        if (a.first == a.last) {
            if (warp == 0 && mine.there) fill_row<E>(ap, a, mine.t, mine.g, 0.f, block);
            continue;
        }
        const int32_t tiles = a.tile1 - a.tile0;
        float m = -INFINITY, l = 0.f;
        for (int32_t j = 0; j < tiles; ++j, ++count) {
            const uint32_t slot = count & 1;
            ok = wait(sh.s_full + slot, count / 2 & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_at = tmem + lanes + slot * 128;
            uint32_t s[32];
            tmem_ld32_wait(s_at + 32 * warp, s);
            const int64_t key0 = static_cast<int64_t>(a.tile0 + j) * S::kKeys + 32 * warp;
            uint32_t bits = ~0u;
            if (mine.there)
                bits = low_bits(static_cast<int>(max(min(mine.hi - key0, int64_t{32}), int64_t{0}))) &
                       ~low_bits(static_cast<int>(min(max(mine.lo - key0, int64_t{0}), int64_t{32})));
            if (sh.slot_missing[slot]) bits &= reinterpret_cast<const uint32_t*>(sh.slot_keys + slot)[warp];
            if (__any_sync(~0u, bits != ~0u))
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (!(bits >> c & 1)) s[c] = 0xff800000u;
            float top[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(s[c]);
#pragma unroll
            for (int c = 4; c < 32; ++c) top[c % 4] = fmaxf(top[c % 4], __uint_as_float(s[c]));
            const float x = fmaf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), p.scale_log2, -kOffset);
            const bool raise = mine.there && x > m + kGrowth;
            if (__any_sync(~0u, raise)) {
                const float now = raise ? x : m, shrink = raise ? exp2_fast(m - now) : 1.f;
                m = now;
                l *= shrink;
                __syncwarp();
                if (j > 0) {
                    ok = wait(sh.pv_done + (count - 1 & 1), (count - 1) / 2 & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32_wait(o_at + c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
                        tmem_st32(o_at + c, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            uint32_t w[16], zero[16];
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[i] = exp2_fast(fmaf(__uint_as_float(s[c + i]), p.scale_log2, -base));
                    sum[i] += e[i];
                    zero[(c + i) / 2] = 0;
                }
                w[c / 2] = pack16<E>(e[0], e[1]);
                w[c / 2 + 1] = pack16<E>(e[2], e[3]);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
            for (int b = 1; b < 4; ++b) tmem_st16(s_at + (warp + b) % 4 * 16, zero);
            tmem_st16(s_at + warp * 16, w);
            if (!ok) break;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(sh.p_half + slot);
                mbar_arrive(sh.p_full + slot);
            }
        }
        ok = ok && wait(sh.pv_done + (count - 1 & 1), (count - 1) / 2 & 1);
        if (!ok) break;
        tc_fence_after();
        // The unit's last scores are done, and with them its Q: its space holds the quarters' maxima and sums, then their results, 32
        // channels at a time.
        const uint32_t q_slot = qn++ % S::kQSlots;
        float* mix = reinterpret_cast<float*>(q_s + q_slot * S::kQBytes);
        reinterpret_cast<float2*>(mix)[warp * 32 + lane] = make_float2(m, l);
        ok = meet();
        if (!ok) break;
        float top = -INFINITY, sum = 0.f;
        float2 ml[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            ml[w] = reinterpret_cast<const float2*>(mix)[w * 32 + lane];
            top = fmaxf(top, ml[w].x);
        }
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum = fmaf(ml[w].y, exp2_fast(ml[w].x - base), sum);
        const bool whole = a.tile0 == a.first && a.tile1 == a.last;
        const float by = exp2_fast(m - base) * (whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f);
        if (warp == 0 && mine.there) {
            const RowOut<E> out = row_out<E>(ap, a, block, mine.t, mine.g);
            if (out.lse) *out.lse = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
            if (out.ml) *out.ml = make_float2(top, sum);
        }
        const int r = 8 * warp + lane / 4;  // the row whose result this lane joins, eight channels of 32
        const Row other = row_of(a, r);
        const RowOut<E> out = row_out<E>(ap, a, block, other.t, other.g);
        bool spoilt = false;
#pragma unroll 1
        for (int c = 0; c < D && ok; c += 32) {
            __syncwarp();
            uint32_t o[32];
            tmem_ld32_wait(o_at + c, o);
            ok = meet();  // what was there has been read
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(mix + (warp * 32 + lane) * 32 + (i ^ (lane & 7)) * 4) =
                    make_float4(__uint_as_float(o[4 * i]) * by, __uint_as_float(o[4 * i + 1]) * by, __uint_as_float(o[4 * i + 2]) * by,
                                __uint_as_float(o[4 * i + 3]) * by);
            ok = meet();
            if (!ok) break;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 v = *reinterpret_cast<const float4*>(mix + (w * 32 + r) * 32 + ((2 * (lane & 3) + h) ^ (r & 7)) * 4);
                    y[4 * h] += v.x, y[4 * h + 1] += v.y, y[4 * h + 2] += v.z, y[4 * h + 3] += v.w;
                }
            const int d = c + 8 * (lane & 3);
            float sum0 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (d + i < D) sum0 = fmaf(y[i], 0.f, sum0);
            // A warp takes the others' keys times zero, so that a value that is not finite makes NaN in the other three.  A single
            // infinite result beside them is the row's: it would be NaN, too, if there were such values among the others' keys.
            if (sum0 != 0.f && other.there) {
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    float kept = 0.f;
                    int infinite = 0;
                    for (int w = 0; w < 4; ++w) {
                        const float v = mix[(w * 32 + r) * 32 + ((2 * (lane & 3) + i / 4) ^ (r & 7)) * 4 + i % 4];
                        if (v == v && v - v != 0.f) kept = v, ++infinite;
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (u == i && infinite == 1 && y[u] != y[u]) y[u] = kept;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) spoilt |= d + i < D && y[i] != y[i];
            }
            if (!other.there) continue;
            if (out.o && p.out_vec) {
                if (d < D) *reinterpret_cast<uint4*>(out.o + d) = make_uint4(pack16<E>(y[0], y[1]), pack16<E>(y[2], y[3]), pack16<E>(y[4], y[5]), pack16<E>(y[6], y[7]));
            } else if (out.part && D % 4 == 0) {
                if (d < D) *reinterpret_cast<float4*>(out.part + d) = make_float4(y[0], y[1], y[2], y[3]);
                if (d + 4 < D) *reinterpret_cast<float4*>(out.part + d + 4) = make_float4(y[4], y[5], y[6], y[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (d + i < D) {
                        if (out.o)
                            out.o[d + i] = narrow16<E>(y[i]);
                        else
                            out.part[d + i] = y[i];
                    }
            }
        }
        if (!ok) break;
        tc_fence_before();
        // Q may come again once all have read; the copies that bring it do not see plain accesses by themselves.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.q_empty + q_slot);
        const float weights = __shfl_sync(~0u, sum, r);
        const bool row = (lane & 3) == 0 && other.there && weights > 0.f;
        const int2 unfinite = sh.unfinite(0, qn);
        if (__any_sync(~0u, spoilt && weights > 0.f))  // the sum of such values that a row sees takes its place
            add_unfinite<E, true>(ap, a, row, other.t, other.g, other.lo, other.hi, make_int2(a.tile0, a.tile1), block, lane);
        else if (unfinite.x < unfinite.y)
            add_unfinite<E, false>(ap, a, row, other.t, other.g, other.lo, other.hi, unfinite, block, lane);
    }
    if (!ok) {  // what a wait that ran out has left undone: the rows whose results this warp joins
        AttnWalk walk;
        walk.begin(sh.scan.start);
        AttnPart a;
        for (uint32_t i = 0; walk.next(ap, a); ++i) {
            if (i < k) continue;
            const Row mine = row_of(a, 8 * warp + lane / 4);
            if ((lane & 3) == 0 && mine.there) fill_row<E>(ap, a, mine.t, mine.g, __int_as_float(0x7fffffff), block);
            if (warp == 0 && lane == 0) note_cut(ap, a, block, walk);
        }
    }
}

template <class E, int kDim, int kStreams>
__global__ void __launch_bounds__(128 + 128 * kStreams, 1)
    attention_tc_kernel(const __grid_constant__ TcParams p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v) {
    using S = Shape<kDim, kStreams>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* q_s = smem;
    uint8_t* kv_s = smem + S::kQTiles * S::kQBytes;
    Misc<S>& sh = *reinterpret_cast<Misc<S>*>(smem + S::kTileBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t block = blockIdx.x;
    griddep_launch_dependents();  // the join's blocks, which wait for this kernel's end
    if (tid == 0) {
        p.a.joins[2 * block] = make_int4(0, 0, 0, 0);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(sh.kv_full + i, p.plain ? 64 : 1);
            mbar_init(sh.kv_empty + i, kStreams);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sh.q_full + i, p.plain ? 64 : 1);
            mbar_init(sh.q_empty + i, p.quarters ? 4 : kStreams);
            mbar_init(sh.s_full + i, 2);     // the product, and the slot's mask
            mbar_init(sh.p_half + i, 4);     // a warpgroup's warps
            mbar_init(sh.p_full + i, 4);
            mbar_init(sh.pv_done + i, 2);     // the product, and what was set apart in its values
        }
        for (int i = 0; i < kParts; ++i) {
            mbar_init(sh.part_full + i, 1);
            mbar_init(sh.part_empty + i, 5 * kStreams);
        }
        mbar_init(&sh.both, 2);
        mbar_init(&sh.mix, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(sh.turn + i, 1);
            mbar_init(sh.drain + i, 1);
        }
        sh.abort = 0;
        fence_mbar_init();
        if (!p.plain) {
            prefetch_tensormap(&map_q);
            prefetch_tensormap(&map_k);
            prefetch_tensormap(&map_v);
        }
    }
    if (warp == 2) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    if (p.plain) {  // channels behind the heads' end are never written: zero once and for all
        for (int i = tid; i < S::kTileBytes / 16; i += S::kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    attn_start<S::kThreads>(p.a, block, gridDim.x, sh.scan);  // and the barriers are there for all
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (warp < 4) {
        if constexpr (kStreams == 2) regs_dec<80>();
        if (warp == 0) {
            if (p.plain)
                produce_plain<E, S, kStreams>(p, sh, q_s, kv_s, 0, lane);
            else
                produce<S, kStreams>(p, &map_q, &map_k, &map_v, sh, q_s, kv_s, lane);
        } else if (warp <= kStreams) {
            multiply<E, S, kStreams>(p, sh, q_s, kv_s, tmem, warp - 1, lane);
        } else if (warp == 3 && p.plain) {
            produce_plain<E, S, kStreams>(p, sh, q_s, kv_s, 1, lane);
        }
    } else {
        if constexpr (kStreams == 2) regs_inc<208>();  // 128 x 80 + 256 x 208 of the 384 x 168 registers that the block has
        if constexpr (kStreams == 1) {
            if (p.quarters)
                exponentiate_quarters<E, S>(p, sh, q_s, tmem, warp & 3, lane, block);
            else
                exponentiate<E, S, kDim, kStreams>(p, sh, tmem, 0, warp & 3, lane, block);
        } else {
            exponentiate<E, S, kDim, kStreams>(p, sh, tmem, (warp - 4) / 4, warp & 3, lane, block);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <class E, int kDim, int kStreams>
cudaError_t launch_shape(const TcParams& p, const CUtensorMap* maps, int32_t blocks, cudaStream_t stream) {
    using S = Shape<kDim, kStreams>;
    static_assert(smem_bytes<S>() <= 227 * 1024, "shared memory");
    auto kernel = attention_tc_kernel<E, kDim, kStreams>;
    constexpr int bytes = static_cast<int>(smem_bytes<S>());
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<blocks, S::kThreads, bytes, stream>>>(p, maps[0], maps[1], maps[2]);
    return cudaGetLastError();
}

template <class E>
cudaError_t launch_typed(const TcParams& p, const CUtensorMap* maps, int streams, int32_t blocks, cudaStream_t stream) {
    const int D = p.a.c.head_dim;
    if (D > 128) return launch_shape<E, 256, 1>(p, maps, blocks, stream);
    if (D > 64)
        return streams == 2 ? launch_shape<E, 128, 2>(p, maps, blocks, stream) : launch_shape<E, 128, 1>(p, maps, blocks, stream);
    return streams == 2 ? launch_shape<E, 64, 2>(p, maps, blocks, stream) : launch_shape<E, 64, 1>(p, maps, blocks, stream);
}

}  // namespace attn_tc

cudaError_t launch_attention_tc_bf16(const attn_tc::TcParams& p, const CUtensorMap* maps, int streams, int32_t blocks, cudaStream_t stream);
cudaError_t launch_attention_tc_f16(const attn_tc::TcParams& p, const CUtensorMap* maps, int streams, int32_t blocks, cudaStream_t stream);

}  // namespace gdn
