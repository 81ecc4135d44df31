// gdn_attention.cuh -- what the kernels of include/gdn_attention.h share: a
// batch's sequences in the cache, and how attention's work is dealt out.  Not
// part of the public C ABI.
#pragma once

#include "../../include/gdn_attention.h"
#include "gdn_internal.cuh"

namespace gdn {

// Sequence i of a batch: its new tokens [start, start + n) of the packed rows, its row of the table (-1: none), its tokens
// with the new ones, and how many of those the table can hold.
struct KvSpan {
    int64_t start;
    int32_t n, row, len, keys;
};

// Never leaves the bounds the host has given, whatever the device data say.  `err` collects status bits.
__device__ __forceinline__ KvSpan kv_span(const gdn_kv_batch& b, int32_t i, uint32_t& err) {
    KvSpan s;
    if (b.cu_seqlens) {
        const int64_t lo = load_index(b.cu_seqlens, b.cu_i64, i), hi = load_index(b.cu_seqlens, b.cu_i64, i + 1);
        if (lo < 0 || hi < lo || hi > b.total_tokens || (i == 0 && lo != 0)) err |= GDN_DEVICE_ERR_CU_SEQLENS;
        const int64_t a = min(max(lo, int64_t{0}), b.total_tokens), e = min(hi, b.total_tokens);
        s.start = a;
        s.n = static_cast<int32_t>(max(e - a, int64_t{0}));
    } else {
        s.start = static_cast<int64_t>(i) * b.tokens_per_seq;
        s.n = b.tokens_per_seq;
    }
    s.row = b.seqs ? b.seqs[i] : i;
    s.len = s.keys = 0;
    if (s.row < 0 || s.row >= b.max_seqs) {
        err |= GDN_PAGES_ERR_SEQ;
        s.row = -1;
        return s;
    }
    s.len = b.lengths[s.row];
    const int64_t room = static_cast<int64_t>(b.max_pages) * b.page_tokens;
    if (s.len < 0 || s.len > room) err |= GDN_PAGES_ERR_PAGE;
    s.len = max(s.len, 0);
    s.keys = static_cast<int32_t>(min(static_cast<int64_t>(s.len), room));
    return s;
}

__device__ __forceinline__ void kv_report(int32_t* status, uint32_t err) {
    if (err && status) atomicOr(status, static_cast<int32_t>(err));
}

// ---------------------------------------------------------------------------------------------------------------------
// Attention's work.  A unit is one sequence's `unit_tokens` successive new tokens of one group of query heads that share a
// key head; its rows are (token, head of the group), token by token.  A unit passes over the tiles of `tile` keys that any
// of its rows sees: that many steps, and `unit_cost` more for what a unit costs beside them.  All units' steps, in the order
// (sequence, group, tokens), are one line that is cut into equal pieces, one a block: any mix of long and short sequences
// fills the GPU evenly, with no list to be written first, and a cut within a unit leaves two partial results to be joined.
// Where a cut falls follows from the lengths alone, so results do not depend on timing.
// ---------------------------------------------------------------------------------------------------------------------
struct AttnParams {
    gdn_kv_batch b;
    gdn_kv_cache c;
    const void* q;
    void* o;
    float* lse;
    int64_t q_stride, o_stride;
    int32_t heads, per_kv;         // query heads; query heads a key head
    int32_t group, pieces;         // heads of a unit; units that a key head's heads make (the last may have fewer)
    int32_t unit_tokens, tile;
    int32_t causal, window;
    float scale_log2;              // scale * log2(e): the kernels' exponentials are powers of two
    int32_t unit_cost;             // steps, about, that a unit's start and end take
    int32_t min_steps;             // a block's least share
    float* part_o;                 // [2 * blocks][unit rows][D], sums of weights times values
    float2* part_ml;               // [2 * blocks][unit rows]: maximum (scaled, log2) and sum of weights
    int4* joins;                   // [2 * blocks]: what a unit that starts in this block and ends in a later one is made of
};

__host__ __device__ inline int32_t attn_units_of(int32_t n, int32_t unit_tokens) { return (n + unit_tokens - 1) / unit_tokens; }

// Tiles [first, last) of the keys that some of the tokens [t0, t1) see.
__device__ __forceinline__ void attn_tiles(const AttnParams& p, const KvSpan& s, int32_t t0, int32_t t1, int32_t& first, int32_t& last) {
    const int64_t at = static_cast<int64_t>(s.len) - s.n, keys = s.keys;
    const int64_t hi = p.causal ? min(max(at + t1, int64_t{0}), keys) : keys;
    const int64_t lo = p.window ? min(max(at + t0 - p.window + 1, int64_t{0}), keys) : 0;
    first = static_cast<int32_t>(lo / p.tile);
    last = static_cast<int32_t>((hi + p.tile - 1) / p.tile);
}

// sum over i < m of floor((clamp(a + step i, 0, cap) + add) / tile), tile a power of two: the clamped ends are constant, in
// between the sum of the quotients is that of the numbers less that of their remainders, which go round with a period of at
// most `tile`.
__device__ __forceinline__ int64_t attn_sum(int64_t a, int64_t step, int64_t m, int64_t cap, int64_t add, int32_t tile) {
    if (m <= 0) return 0;
    int64_t i0 = a >= 0 ? 0 : (-a + step - 1) / step, i1 = a > cap ? 0 : (cap - a) / step + 1;
    i0 = min(i0, m);
    i1 = max(min(i1, m), i0);
    int64_t sum = i0 * (add / tile) + (m - i1) * ((cap + add) / tile);
    const int64_t n = i1 - i0, x = a + step * i0 + add;
    if (n > 0) {
        const int64_t low = step & -step, g = low < tile ? low : tile, period = tile / g, full = n / period, rest = n % period;
        int64_t rem = full * (period * (x & (g - 1)) + g * (period * (period - 1) / 2));
        int64_t r = x & (tile - 1);
        for (int64_t j = 0; j < rest; ++j) {
            rem += r;
            r = (r + step) & (tile - 1);
        }
        sum += (n * x + step * (n * (n - 1) / 2) - rem) / tile;
    }
    return sum;
}

// Steps of the first m units of one group of sequence s.
__device__ __forceinline__ int64_t attn_steps(const AttnParams& p, const KvSpan& s, int32_t m) {
    if (m <= 0) return 0;
    const bool whole = static_cast<int64_t>(m) * p.unit_tokens >= s.n;  // the last unit may be shorter than the others
    const int32_t k = whole ? m - 1 : m;
    int64_t sum = static_cast<int64_t>(m) * p.unit_cost;
    if (k > 0) {
        const int64_t at = static_cast<int64_t>(s.len) - s.n, keys = s.keys, top = (keys + p.tile - 1) / p.tile;
        sum += p.causal ? attn_sum(at + p.unit_tokens, p.unit_tokens, k, keys, p.tile - 1, p.tile) : k * top;
        if (p.window) sum -= attn_sum(at - p.window + 1, p.unit_tokens, k, keys, 0, p.tile);
    }
    if (whole) {
        int32_t first, last;
        attn_tiles(p, s, k * p.unit_tokens, s.n, first, last);
        sum += last - first;
    }
    return sum;
}

// A block's piece of the line.
struct AttnStart {
    int64_t skip;                  // steps of the first unit that belong to earlier blocks
    int64_t left;                  // steps of the piece
    int64_t share;                 // steps of every block's piece (the last one's may be less)
    int32_t seq, group, unit;
};

template <int kThreads>
struct AttnScan {
    int64_t sums[kThreads / 32];
    AttnStart start;
};

// Where this block's piece starts; the whole block calls it.  `blocks` pieces, this one is `block`.
template <int kThreads>
__device__ AttnStart attn_start(const AttnParams& p, int32_t block, int32_t blocks, AttnScan<kThreads>& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t N = p.b.num_seqs, groups = p.c.kv_heads * p.pieces;
    const int32_t each = (N + kThreads - 1) / kThreads, i0 = min(tid * each, N), i1 = min(i0 + each, N);
    uint32_t err = 0;
    int64_t mine = 0;
    for (int32_t i = i0; i < i1; ++i) {
        const KvSpan s = kv_span(p.b, i, err);
        mine += groups * attn_steps(p, s, attn_units_of(s.n, p.unit_tokens));
    }
    if (block == 0) kv_report(p.b.device_status, err);
    int64_t upto = mine;
    for (int d = 1; d < 32; d *= 2) {
        const int64_t o = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) sh.sums[warp] = upto;
    if (tid == 0) sh.start = AttnStart{0, 0, 0, 0, 0, 0};
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before = total;
        total += sh.sums[w];
    }
    const int64_t share = max((total + blocks - 1) / blocks, static_cast<int64_t>(p.min_steps));
    const int64_t begin = share * block;
    before += upto - mine;
    if (begin < total && before <= begin && begin < before + mine) {
        int64_t at = before;
        for (int32_t i = i0; i < i1; ++i) {
            const KvSpan s = kv_span(p.b, i, err);
            const int64_t w = groups * attn_steps(p, s, attn_units_of(s.n, p.unit_tokens));
            if (begin < at + w) {
                sh.start = AttnStart{begin - at, min(share, total - begin), share, i, 0, 0};
                break;
            }
            at += w;
        }
    }
    __syncthreads();
    AttnStart st = sh.start;
    if (warp == 0 && st.left > 0) {
        const KvSpan s = kv_span(p.b, st.seq, err);
        const int32_t units = attn_units_of(s.n, p.unit_tokens);
        const int64_t one = attn_steps(p, s, units);
        st.group = static_cast<int32_t>(st.skip / one);
        st.skip -= st.group * one;
        // the last unit that starts at or before st.skip: 32 candidates at a time
        int32_t lo = 0, hi = units;
        while (hi - lo > 1) {
            const int32_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
            const unsigned vote = __ballot_sync(~0u, at < hi && attn_steps(p, s, at) <= st.skip);
            lo += __popc(vote) * step;
            hi = min(hi, lo + step);
        }
        st.unit = lo;
        st.skip -= attn_steps(p, s, lo);
        if (lane == 0) sh.start = st;
    }
    __syncthreads();
    return sh.start;
}

// One unit's part of a piece: tiles [tile0, tile1) of the unit's [first, last).
struct AttnPart {
    int64_t row0;                  // packed row of the unit's first token
    int32_t tokens, pos0;          // tokens of the unit, the first one's position (may be negative)
    int32_t kv_head, head0, heads; // its query heads
    int32_t table_row, keys;       // keys that the sequence has at most
    int32_t tile0, tile1, first, last;
};

// Walks through a piece unit by unit.  Every thread that calls it gets the same parts.
struct AttnWalk {
    AttnStart at;
    KvSpan span;
    int32_t loaded;                // the sequence that span is of

    __device__ __forceinline__ void begin(const AttnStart& s) {
        at = s;
        loaded = -1;
    }

    // The next part; false at the piece's end.  A unit without any key is a part without tiles (first = last).
    __device__ __forceinline__ bool next(const AttnParams& p, AttnPart& out) {
        uint32_t err = 0;
        while (at.left > 0 && at.seq < p.b.num_seqs) {
            if (loaded != at.seq) {
                span = kv_span(p.b, at.seq, err);
                loaded = at.seq;
            }
            const int32_t units = attn_units_of(span.n, p.unit_tokens);
            if (at.unit >= units) {
                at.unit = 0;
                if (units == 0 || ++at.group >= p.c.kv_heads * p.pieces) {
                    at.group = 0;
                    ++at.seq;
                }
                continue;
            }
            const int32_t t0 = at.unit * p.unit_tokens, t1 = min(t0 + p.unit_tokens, span.n);
            attn_tiles(p, span, t0, t1, out.first, out.last);
            const int64_t take = min(at.left, out.last - out.first + p.unit_cost - at.skip);
            out.tile0 = out.first + static_cast<int32_t>(max(at.skip - p.unit_cost, int64_t{0}));
            out.tile1 = out.first + static_cast<int32_t>(max(at.skip + take - p.unit_cost, int64_t{0}));
            const bool starts = at.skip == 0;
            out.row0 = span.start + t0;
            out.tokens = t1 - t0;
            out.pos0 = static_cast<int32_t>(static_cast<int64_t>(span.len) - span.n + t0);
            const int32_t kv = at.group / p.pieces, piece = at.group % p.pieces;
            out.kv_head = kv;
            out.head0 = kv * p.per_kv + piece * p.group;
            out.heads = min(p.group, p.per_kv - piece * p.group);
            out.table_row = span.row;
            out.keys = span.keys;
            at.left -= take;
            at.skip = 0;
            ++at.unit;
            if (out.first == out.last ? starts : out.tile0 < out.tile1) return true;
        }
        return false;
    }
};

// The slot of partial results of block `block` for a part that is not its whole unit; what starts a unit goes to the odd one.
__device__ __forceinline__ int32_t attn_slot(const AttnPart& a, int32_t block) { return 2 * block + (a.tile0 == a.first ? 1 : 0); }

// Notes a unit that starts here and ends in a later block: {parts, tokens, first head, heads}, {first token (64 bits)}.
__device__ __forceinline__ void attn_note_join(const AttnParams& p, const AttnPart& a, int32_t block, int64_t share) {
    const int32_t later = static_cast<int32_t>((a.last - a.tile1 + share - 1) / share);
    p.joins[2 * block] = make_int4(1 + later, a.tokens, a.head0, a.heads);
    p.joins[2 * block + 1] = make_int4(static_cast<int32_t>(a.row0), static_cast<int32_t>(a.row0 >> 32), 0, 0);
}

// Whether T rows each at x and y, of so many bytes and so many bytes apart, have no byte in common.  Rows of one stride may lie
// between each other (slices of one tensor); of others only the spans are compared.
inline bool rows_apart(const void* x, int64_t x_stride, int64_t x_row, const void* y, int64_t y_stride, int64_t y_row, int64_t T) {
    using wide_t = __int128;
    const wide_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    if (b >= a + static_cast<wide_t>(T - 1) * x_stride + x_row || a >= b + static_cast<wide_t>(T - 1) * y_stride + y_row) return true;
    if (T == 1 || x_stride != y_stride) return false;
    const wide_t off = ((b - a) % x_stride + x_stride) % x_stride;  // from a row of x to the next of y
    return off >= x_row && x_stride - off >= y_row;
}

// What the host can see of a batch and a cache.
gdn_status kv_check(const gdn_kv_batch* batch, const gdn_kv_cache* cache);

size_t attn_workspace(int32_t blocks, int32_t rows, int32_t D);
// Points p's partial results into a workspace.
void attn_place(AttnParams* p, void* workspace, int32_t blocks, int32_t rows);
cudaError_t launch_attention_simple(const AttnParams& p, int32_t blocks, cudaStream_t stream);
cudaError_t launch_attention_join(const AttnParams& p, int32_t blocks, cudaStream_t stream);

}  // namespace gdn
