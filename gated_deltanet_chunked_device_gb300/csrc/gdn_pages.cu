// gdn_pages.cu -- page operators of a cache (include/gdn_pages.h): reserve,
// fork, free, compact and copy, kernels and host side.
//
// The bookkeeping of one call is done by one block of 1024 threads: its size
// is a few bytes a page and a few a table entry, and its time a handful of
// round trips to L2, so what it has to remember between them stays in shared
// memory where it fits (lists of up to 1024 sequences, tables of up to 4096).
// The pages' data are moved by a grid of its own, from lists that the first
// kernel left in the workspace; nothing returns to the host in between.
//
// What bounds them: HBM where pages are large (384 rows of 1 MiB copied in 122
// us, 6.6 TB/s, 0.98 of a measured copy; 1 GB moved by a compaction in 171 us,
// 0.90 with its bookkeeping), the launches and the host else: the bookkeeping
// of a call takes 6 to 9 us of one SM, a fork of 4 sequences 19 us on the host.
#include <climits>

#include "../../include/gdn_pages.h"
#include "gdn_internal.cuh"

namespace {

constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kSmallList = 1024;   // entries of a list that shared memory holds
constexpr int kSmallSeqs = 4096;   // marks of sequences that shared memory holds
constexpr int kSmallFree = 2048;   // free pages that shared memory holds
constexpr int kKept = 8;           // words of a warp's part of the pages that registers hold
constexpr int kCopyThreads = 256;
constexpr int64_t kPiece = 16384;  // bytes of a page that a block copies at a time

struct CopyBuffer {
    const uint8_t* src;
    uint8_t* dst;
    int64_t src_stride, dst_stride, bytes;
    int32_t unit;                  // bytes that source and destination can be copied at a time: 16, 4 or 1
};

// A table to be rewritten by remap.
struct Remap {
    const int32_t* table;
    int32_t* table_out;
    const int32_t* remap;
    int64_t entries;
    int32_t n_pages;
};

// kMax buffers at most: the parameters of a launch are copied whole.
template <int kMax>
struct CopyParams {
    Remap table;                   // entries = 0: none
    CopyBuffer buffers[kMax];
    int32_t n_buffers;
    int32_t src_pages, dst_pages;
    int32_t max_pieces;            // of the largest buffer's row
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;          // pairs, on the device; nullptr: n
    int32_t n;
    int32_t* status;
};

struct BookParams {
    int32_t* table;
    int32_t* refcounts;
    int32_t* lengths;
    int32_t max_seqs, max_pages, n_pages;
    const int32_t* seqs;           // reserve: the sequences; fork: the children
    const int32_t* counts;         // reserve
    const int32_t* parents;        // fork
    int32_t n;
    int32_t page_tokens;
    int32_t* rows;
    int32_t* status;
    // workspace
    int32_t* marks;                // [max_seqs] place in the list of the first entry that names the sequence
    int32_t* need;                 // [n] pages to give, -1: an entry at fault
    int32_t* offset;               // [n] first of them
    int32_t* used;                 // [n] fork: pages in use by the parent
    int32_t* plen;                 // [n] fork: the parent's length
    int32_t* free_list;            // [n_pages]
    int32_t* copy_src;             // [n_pages] pairs of the copy that follows
    int32_t* copy_dst;
    int32_t* copy_count;
    // compact
    int32_t* refcounts_out;
    int32_t* remap;
    int32_t* n_live;
};

__device__ __forceinline__ void report(int32_t* status, int32_t bit) {
    if (status) atomicOr(status, bit);
}

// Numbers the i in [0, n) that pred holds for, in order: emit(rank, i) for each.  Warps own contiguous ranges; they
// count, the block sums the counts, and they go over their ranges again (the first words of them from registers).
// Returns how many there are.
template <class Pred, class Emit>
__device__ __forceinline__ int32_t number_in_order(int32_t n, int32_t* warp_sums, Pred pred, Emit emit) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t seg = ((static_cast<int64_t>(n) + kBookWarps - 1) / kBookWarps + 31) / 32 * 32;
    const int64_t from = warp * seg, to = from + seg < n ? from + seg : n;
    uint32_t kept[kKept];
    int32_t c = 0;
#pragma unroll
    for (int w = 0; w < kKept; ++w) {
        const int64_t i = from + 32 * w + lane;
        kept[w] = __ballot_sync(0xffffffffu, i < to && pred(i));
        c += __popc(kept[w]);
    }
#pragma unroll 4
    for (int64_t i = from + 32 * kKept; i < to; i += 32) c += __popc(__ballot_sync(0xffffffffu, i + lane < to && pred(i + lane)));
    __syncthreads();
    if (lane == 0) warp_sums[warp] = c;
    __syncthreads();
    const int32_t mine = warp_sums[lane];
    const int32_t total = __reduce_add_sync(0xffffffffu, mine);
    int32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
#pragma unroll
    for (int w = 0; w < kKept; ++w) {
        if ((kept[w] >> lane) & 1) emit(before + __popc(kept[w] & ((1u << lane) - 1)), static_cast<int32_t>(from + 32 * w + lane));
        before += __popc(kept[w]);
    }
    for (int64_t i = from + 32 * kKept; i < to; i += 32) {
        const bool on = i + lane < to && pred(i + lane);
        const uint32_t m = __ballot_sync(0xffffffffu, on);
        if (on) emit(before + __popc(m & ((1u << lane) - 1)), static_cast<int32_t>(i + lane));
        before += __popc(m);
    }
    return total;
}
static_assert(kBookWarps == 32, "a lane a warp's sum");

// offset[k] = sum of the positive need[j], j < k; returns the sum of all.
__device__ __forceinline__ int32_t running_sums(int32_t n, const int32_t* need, int32_t* offset, int32_t* warp_sums) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t seg = ((static_cast<int64_t>(n) + kBookWarps - 1) / kBookWarps + 31) / 32 * 32;
    const int64_t from = warp * seg, to = from + seg < n ? from + seg : n;
    int32_t c = 0;
    for (int64_t i = from + lane; i < to; i += 32) c += max(need[i], 0);
    c = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if (lane == 0) warp_sums[warp] = c;
    __syncthreads();
    const int32_t mine = warp_sums[lane];
    const int32_t total = __reduce_add_sync(0xffffffffu, mine);
    int32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
    for (int64_t i = from; i < to; i += 32) {
        const int32_t v = i + lane < to ? max(need[i + lane], 0) : 0;
        int32_t s = v;
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        if (i + lane < to) offset[i + lane] = before + s - v;
        before += __shfl_sync(0xffffffffu, s, 31);
    }
    __syncthreads();
    return total;
}

// Lanes that work on one entry of a list: a power of two, as many as a table row has entries, at most a warp.
struct Lanes {
    int count, lane, first;        // of a group; this thread's place in its group; the group's first lane
    __device__ explicit Lanes(int32_t max_pages) {
        count = 1;
        while (count < 32 && count < max_pages) count *= 2;
        lane = threadIdx.x % count;
        first = threadIdx.x % 32 / count * count;
    }
    __device__ int group() const { return threadIdx.x / count; }
    __device__ int groups() const { return kBookThreads / count; }
    __device__ int32_t sum(int32_t v) const {
        for (int o = count / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    __device__ uint32_t ballot(bool v) const {
        const uint32_t m = __ballot_sync(0xffffffffu, v) >> first;
        return count == 32 ? m : m & ((1u << count) - 1);
    }
    __device__ bool any(bool v) const { return ballot(v) != 0; }
};

// What a list's entries get, in shared memory or in the workspace.
struct BookLists {
    int32_t *marks, *need, *offset, *used, *plen, *free_list;
};

struct BookSmem {
    int32_t warp_sums[kBookWarps];
    int32_t marks[kSmallSeqs];
    int32_t lists[4][kSmallList];
    int32_t free_list[kSmallFree];
};

static_assert(sizeof(BookSmem) <= 48 * 1024, "shared memory that needs no leave");

__device__ __forceinline__ BookLists book_lists(const BookParams& p, BookSmem& sm) {
    BookLists b{p.marks, p.need, p.offset, p.used, p.plen, p.free_list};
    if (p.max_seqs <= kSmallSeqs) b.marks = sm.marks;
    if (p.n <= kSmallList) {
        b.need = sm.lists[0];
        b.offset = sm.lists[1];
        b.used = sm.lists[2];
        b.plen = sm.lists[3];
    }
    return b;
}

// Of the entries of the list that name one sequence, the first one wins.
__device__ __forceinline__ void mark_sequences(const BookParams& p, int32_t* marks) {
    for (int64_t k = threadIdx.x; k < p.n; k += kBookThreads)
        if (p.seqs[k] >= 0 && p.seqs[k] < p.max_seqs) marks[p.seqs[k]] = INT_MAX;
    __syncthreads();
    for (int64_t k = threadIdx.x; k < p.n; k += kBookThreads)
        if (p.seqs[k] >= 0 && p.seqs[k] < p.max_seqs) atomicMin(&marks[p.seqs[k]], static_cast<int32_t>(k));
    __syncthreads();
}

// Lists the first `wanted` free pages; returns how many are free.
__device__ __forceinline__ int32_t list_free_pages(const BookParams& p, int32_t wanted, int32_t* warp_sums, int32_t* list) {
    const int32_t n = number_in_order(
        p.n_pages, warp_sums, [&](int64_t i) { return p.refcounts[i] <= 0; },
        [&](int32_t rank, int32_t page) {
            if (rank < wanted) list[rank] = page;
        });
    __syncthreads();
    return n;
}

__global__ void __launch_bounds__(kBookThreads) gdn_pages_reserve_kernel(BookParams p) {
    extern __shared__ int32_t smem[];
    BookSmem& sm = *reinterpret_cast<BookSmem*>(smem);
    const BookLists b = book_lists(p, sm);
    const Lanes g(p.max_pages);
    mark_sequences(p, b.marks);
    for (int64_t k0 = 0; k0 < p.n; k0 += g.groups()) {
        const int64_t k = k0 + g.group();
        const bool in = k < p.n;
        const int32_t s = in ? p.seqs[k] : -1, want = in ? p.counts[k] : 0;
        const bool seq_ok = s >= 0 && s < p.max_seqs && b.marks[s] == k;
        const bool ok = seq_ok && want >= 0 && want <= p.max_pages;
        int32_t c = 0;
        if (ok)
            for (int32_t j = g.lane; j < want; j += g.count) c += p.table[static_cast<int64_t>(s) * p.max_pages + j] < 0;
        c = g.sum(c);
        if (in && g.lane == 0) {
            b.need[k] = ok ? c : -1;
            if (!ok) report(p.status, seq_ok ? GDN_PAGES_ERR_PAGE : GDN_PAGES_ERR_SEQ);
        }
    }
    __syncthreads();
    const int32_t wanted = running_sums(p.n, b.need, b.offset, sm.warp_sums);
    int32_t* free_list = wanted <= kSmallFree ? sm.free_list : b.free_list;
    const int32_t n_free = list_free_pages(p, wanted, sm.warp_sums, free_list);
    if (wanted > n_free && threadIdx.x == 0) report(p.status, GDN_PAGES_ERR_NO_PAGES);
    for (int64_t k0 = 0; k0 < p.n; k0 += g.groups()) {
        const int64_t k = k0 + g.group();
        const bool in = k < p.n;
        const int32_t need = in ? b.need[k] : -1;
        int32_t at = in ? b.offset[k] : 0;
        const bool served = need >= 0 && at + need <= n_free;
        const int64_t row = need >= 0 ? static_cast<int64_t>(p.seqs[k]) * p.max_pages : 0;
        const int32_t want = served ? p.counts[k] : 0;
        for (int32_t j0 = 0; j0 < p.max_pages; j0 += g.count) {
            const int32_t j = j0 + g.lane;
            int32_t e = need >= 0 && j < p.max_pages ? p.table[row + j] : -1;
            const bool take = j < want && e < 0;
            const uint32_t m = g.ballot(take);
            if (take) {
                e = free_list[at + __popc(m & ((1u << g.lane) - 1))];
                p.table[row + j] = e;
                p.refcounts[e] = 1;
            }
            at += __popc(m);
            if (in && p.rows && j < p.max_pages) p.rows[k * p.max_pages + j] = e;
        }
    }
}

__global__ void __launch_bounds__(kBookThreads) gdn_pages_fork_kernel(BookParams p) {
    extern __shared__ int32_t smem[];
    BookSmem& sm = *reinterpret_cast<BookSmem*>(smem);
    const BookLists b = book_lists(p, sm);
    const Lanes g(p.max_pages);
    mark_sequences(p, b.marks);
    for (int64_t k0 = 0; k0 < p.n; k0 += g.groups()) {
        const int64_t k = k0 + g.group();
        const bool in = k < p.n;
        const int32_t par = in ? p.parents[k] : -1, child = in ? p.seqs[k] : -1;
        int32_t fault = 0, need = 0, used = 0, len = 0;
        if (par < 0 || par >= p.max_seqs || child < 0 || child >= p.max_seqs || par == child || b.marks[child] != k)
            fault = GDN_PAGES_ERR_SEQ;
        bool has = false;
        if (!fault) {
            if (p.lengths) len = p.lengths[par];
            for (int32_t j = g.lane; j < p.max_pages; j += g.count) has |= p.table[static_cast<int64_t>(child) * p.max_pages + j] >= 0;
        }
        if (g.any(has) && !fault) fault = GDN_PAGES_ERR_CHILD;
        bool bad = false;
        int32_t c = 0;
        if (!fault) {
            used = p.max_pages;
            if (p.page_tokens > 0) {
                const int64_t n = len < 0 ? -1 : (static_cast<int64_t>(len) + p.page_tokens - 1) / p.page_tokens;
                bad = n < 0 || n > p.max_pages;
                used = static_cast<int32_t>(bad ? 0 : n);
            }
            for (int32_t j = g.lane; j < used; j += g.count) {
                const int32_t e = p.table[static_cast<int64_t>(par) * p.max_pages + j];
                bad |= e >= p.n_pages || (p.page_tokens > 0 && e < 0);
                c += e >= 0;
            }
        }
        if (g.any(bad) && !fault) fault = GDN_PAGES_ERR_PAGE;
        c = g.sum(c);
        need = p.page_tokens > 0 ? (len % p.page_tokens != 0) : c;
        if (p.page_tokens == 0 && c == 0) used = 0;  // nothing yet, whatever another entry of the list gives this parent
        if (in && g.lane == 0) {
            b.need[k] = fault ? -1 : need;
            b.used[k] = used;
            b.plen[k] = len;
            if (fault) report(p.status, fault);
        }
    }
    __syncthreads();
    const int32_t wanted = running_sums(p.n, b.need, b.offset, sm.warp_sums);
    int32_t* free_list = wanted <= kSmallFree ? sm.free_list : b.free_list;
    const int32_t n_free = list_free_pages(p, wanted, sm.warp_sums, free_list);
    if (wanted > n_free && threadIdx.x == 0) report(p.status, GDN_PAGES_ERR_NO_PAGES);
    int32_t most = 0;  // pairs: the entries served are the first ones
    for (int64_t k0 = 0; k0 < p.n; k0 += g.groups()) {
        const int64_t k = k0 + g.group();
        const bool in = k < p.n;
        const int32_t need = in ? b.need[k] : -1, off = in ? b.offset[k] : 0;
        const bool served = need >= 0 && off + need <= n_free;
        const int64_t child = need >= 0 ? p.seqs[k] : 0, prow = served ? static_cast<int64_t>(p.parents[k]) * p.max_pages : 0;
        const int32_t used = served ? b.used[k] : 0;
        int32_t at = off;
        for (int32_t j0 = 0; j0 < p.max_pages; j0 += g.count) {
            const int32_t j = j0 + g.lane;
            int32_t e = j < used ? p.table[prow + j] : -1;
            const bool copy = e >= 0 && (p.page_tokens == 0 || (need > 0 && j == used - 1));
            const uint32_t m = g.ballot(copy);
            if (copy) {
                const int32_t place = at + __popc(m & ((1u << g.lane) - 1));
                const int32_t fresh = free_list[place];
                p.copy_src[place] = e;
                p.copy_dst[place] = fresh;
                p.refcounts[fresh] = 1;
                e = fresh;
            } else if (e >= 0) {
                atomicAdd(&p.refcounts[e], 1);
            }
            at += __popc(m);
            if (served && j < p.max_pages) p.table[child * p.max_pages + j] = e;
            if (in && p.rows && j < p.max_pages) p.rows[k * p.max_pages + j] = e;
        }
        if (g.lane == 0 && p.lengths && need >= 0) p.lengths[child] = served ? b.plen[k] : 0;
        if (served) most = max(most, off + need);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sm.warp_sums[threadIdx.x / 32] = most;
    __syncthreads();
    if (threadIdx.x < 32) {
        most = __reduce_max_sync(0xffffffffu, sm.warp_sums[threadIdx.x]);
        if (threadIdx.x == 0) *p.copy_count = most;
    }
}

// A warp per sequence.  An entry is taken out of the table by an exchange, so a sequence named twice is freed once.
__global__ void gdn_pages_free_kernel(BookParams p) {
    const int64_t k = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
    const int lane = threadIdx.x % 32;
    if (k >= p.n) return;
    const int32_t s = p.seqs[k];
    if (s < 0 || s >= p.max_seqs) {
        if (lane == 0) report(p.status, GDN_PAGES_ERR_SEQ);
        return;
    }
    for (int32_t j = lane; j < p.max_pages; j += 32) {
        const int32_t e = atomicExch(&p.table[static_cast<int64_t>(s) * p.max_pages + j], -1);
        if (e < 0) continue;
        if (e >= p.n_pages) {
            report(p.status, GDN_PAGES_ERR_PAGE);
        } else if (atomicSub(&p.refcounts[e], 1) <= 0) {
            atomicAdd(&p.refcounts[e], 1);
            report(p.status, GDN_PAGES_ERR_PAGE);
        }
    }
    if (lane == 0 && p.lengths) p.lengths[s] = 0;
}

__global__ void __launch_bounds__(kBookThreads) gdn_pages_compact_kernel(BookParams p) {
    __shared__ int32_t warp_sums[kBookWarps];
    const int32_t L = number_in_order(
        p.n_pages, warp_sums, [&](int64_t i) { return p.refcounts[i] > 0; }, [](int32_t, int32_t) {});
    const int32_t moves = number_in_order(
        p.n_pages, warp_sums, [&](int64_t i) { return i >= L && p.refcounts[i] > 0; },
        [&](int32_t rank, int32_t page) {
            p.copy_src[rank] = page;
            p.free_list[rank] = p.refcounts[page];  // the count that moves with the page
        });
    number_in_order(
        L, warp_sums, [&](int64_t i) { return p.refcounts[i] <= 0; }, [&](int32_t rank, int32_t page) { p.copy_dst[rank] = page; });
    __syncthreads();
    // what stays, then what moves
    for (int64_t i = threadIdx.x; i < p.n_pages; i += kBookThreads) {
        const int32_t r = p.refcounts[i];
        p.remap[i] = r > 0 ? static_cast<int32_t>(i) : -1;
        p.refcounts_out[i] = i < L && r > 0 ? r : 0;
    }
    __syncthreads();
    for (int64_t k = threadIdx.x; k < moves; k += kBookThreads) {
        p.remap[p.copy_src[k]] = p.copy_dst[k];
        p.refcounts_out[p.copy_dst[k]] = p.free_list[k];
    }
    if (threadIdx.x == 0) {
        *p.copy_count = moves;
        *p.n_live = L;
    }
}

// One piece of a row, all loads of a thread before its stores: 64 bytes of a thread in flight, 128 KB of an SM's 8 blocks
// (byte by byte, a load at a time, the same copy takes 5 times as long).
template <class T>
__device__ __forceinline__ void copy_piece(const uint8_t* src, uint8_t* dst, int64_t from, int64_t to) {
    constexpr int kEach = 4;
    const T* s = reinterpret_cast<const T*>(src + from);
    T* d = reinterpret_cast<T*>(dst + from);
    const int n = static_cast<int>((to - from) / sizeof(T));
    for (int i0 = threadIdx.x; i0 < n; i0 += kEach * kCopyThreads) {
        T v[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (i0 + j * kCopyThreads < n) v[j] = __ldcs(s + i0 + j * kCopyThreads);
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (i0 + j * kCopyThreads < n) __stcs(d + i0 + j * kCopyThreads, v[j]);
    }
}

// Copies rows: a unit is one piece of one buffer's row of one pair.  Before that, what there is of a table to rewrite.
template <int kMax>
__global__ void __launch_bounds__(kCopyThreads) gdn_pages_copy_kernel(const __grid_constant__ CopyParams<kMax> p) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; i < p.table.entries;
         i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int32_t e = p.table.table[i];
        if (e < -1 || e >= p.table.n_pages) report(p.status, GDN_PAGES_ERR_PAGE);
        p.table.table_out[i] = e >= 0 && e < p.table.n_pages ? p.table.remap[e] : -1;
    }
    const int64_t units = static_cast<int64_t>(p.count ? *p.count : p.n) * p.n_buffers * p.max_pieces;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        int64_t k;
        int32_t rest;
        const int32_t per_pair = p.n_buffers * p.max_pieces;
        if (unit <= 0xffffffffLL) {  // a division of 32 bits
            k = static_cast<uint32_t>(unit) / static_cast<uint32_t>(per_pair);
            rest = static_cast<int32_t>(unit - k * per_pair);
        } else {
            k = unit / per_pair;
            rest = static_cast<int32_t>(unit % per_pair);
        }
        const int32_t b = rest / p.max_pieces;
        const int64_t from = (rest - b * p.max_pieces) * kPiece;
        const CopyBuffer& f = p.buffers[b];
        if (from >= f.bytes) continue;
        const int32_t s = p.src[k], d = p.dst[k];
        if (s < 0 || d < 0) continue;
        if (s >= p.src_pages || d >= p.dst_pages) {
            if (threadIdx.x == 0) report(p.status, GDN_PAGES_ERR_PAGE);
            continue;
        }
        const int64_t to = from + kPiece < f.bytes ? from + kPiece : f.bytes;
        const uint8_t* src = f.src + s * f.src_stride;
        uint8_t* dst = f.dst + d * f.dst_stride;
        if (f.unit == 16)
            copy_piece<uint4>(src, dst, from, to);
        else if (f.unit == 4)
            copy_piece<uint32_t>(src, dst, from, to);
        else
            copy_piece<uint8_t>(src, dst, from, to);
    }
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

size_t align_up(size_t x) { return (x + 15) / 16 * 16; }

struct Layout {
    size_t marks, need, offset, used, plen, free_list, copy_src, copy_dst, copy_count, total;
};

Layout make_layout(size_t max_seqs, size_t n_pages, size_t list) {
    Layout l{};
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t at = off;
        off = align_up(off + n * sizeof(int32_t));
        return at;
    };
    l.copy_count = take(1);
    l.marks = take(max_seqs);
    l.need = take(list);
    l.offset = take(list);
    l.used = take(list);
    l.plen = take(list);
    l.free_list = take(n_pages);
    l.copy_src = take(n_pages);
    l.copy_dst = take(n_pages);
    l.total = off;
    return l;
}

bool book_ok(const gdn_pages_book* b) {
    return b && b->max_seqs >= 0 && b->max_pages >= 0 && b->n_pages >= 0 && aligned(b->table, 4) && aligned(b->refcounts, 4) &&
           aligned(b->lengths, 4) && (b->table || static_cast<int64_t>(b->max_seqs) * b->max_pages == 0) &&
           (b->refcounts || b->n_pages == 0);
}

bool list_ok(const int32_t* p, int32_t n) { return n >= 0 && aligned(p, 4) && (n == 0 || p); }

// Sums of pages over a list are kept in 32 bits.
bool sums_ok(const gdn_pages_book* b, int32_t n) { return static_cast<int64_t>(b->max_pages) * n <= INT_MAX; }

bool buffers_ok(const gdn_pages_buffer* b, int32_t n) {
    if (n < 0 || n > GDN_PAGES_MAX_BUFFERS || (n > 0 && !b)) return false;
    for (int32_t i = 0; i < n; ++i)
        if (b[i].row_bytes < 0 || b[i].row_stride < b[i].row_bytes || (b[i].row_bytes > 0 && !b[i].base)) return false;
    return true;
}

BookParams make_book(const gdn_pages_book& b, int32_t n, void* workspace) {
    BookParams p{};
    p.table = b.table;
    p.refcounts = b.refcounts;
    p.lengths = b.lengths;
    p.max_seqs = b.max_seqs;
    p.max_pages = b.max_pages;
    p.n_pages = b.n_pages;
    p.n = n;
    if (workspace) {
        const Layout l = make_layout(b.max_seqs, b.n_pages, n);
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        auto at = [&](size_t off) { return reinterpret_cast<int32_t*>(ws + off); };
        p.marks = at(l.marks);
        p.need = at(l.need);
        p.offset = at(l.offset);
        p.used = at(l.used);
        p.plen = at(l.plen);
        p.free_list = at(l.free_list);
        p.copy_src = at(l.copy_src);
        p.copy_dst = at(l.copy_dst);
        p.copy_count = at(l.copy_count);
    }
    return p;
}

// Bytes that rows of both buffers can be copied at a time.
int32_t copy_unit(const gdn_pages_buffer& s, const gdn_pages_buffer& d) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(s.base) | reinterpret_cast<uintptr_t>(d.base) |
                          static_cast<uintptr_t>(s.row_stride | d.row_stride | s.row_bytes);
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
}

// most: an upper bound of the pairs.
template <int kMax>
cudaError_t launch_copy_of(const gdn_pages_buffer* src, int32_t src_pages, const gdn_pages_buffer* dst, int32_t dst_pages,
                           int32_t n_buffers, const int32_t* src_list, const int32_t* dst_list, const int32_t* count, int32_t n,
                           int64_t most, const Remap& table, int32_t* status, cudaStream_t stream) {
    CopyParams<kMax> p;
    int32_t used = 0;
    p.max_pieces = 0;
    for (int32_t i = 0; i < n_buffers; ++i) {
        if (src[i].row_bytes == 0) continue;
        p.buffers[used++] = {static_cast<const uint8_t*>(src[i].base), static_cast<uint8_t*>(dst[i].base), src[i].row_stride,
                             dst[i].row_stride, src[i].row_bytes, copy_unit(src[i], dst[i])};
        const int64_t pieces = (src[i].row_bytes + kPiece - 1) / kPiece;
        if (pieces > INT_MAX / GDN_PAGES_MAX_BUFFERS) return cudaErrorInvalidValue;
        if (pieces > p.max_pieces) p.max_pieces = static_cast<int32_t>(pieces);
    }
    const int64_t rows = most * used * p.max_pieces, entries = (table.entries + kCopyThreads - 1) / kCopyThreads;
    if (rows == 0 && entries == 0) return cudaSuccess;
    p.table = table;
    p.n_buffers = used;
    p.src_pages = src_pages;
    p.dst_pages = dst_pages;
    p.src = src_list;
    p.dst = dst_list;
    p.count = count;
    p.n = n;
    p.status = status;
    const int64_t units = rows > entries ? rows : entries, cap = 8 * gdn::multiprocessors();
    gdn_pages_copy_kernel<kMax><<<static_cast<unsigned>(units < cap ? units : cap), kCopyThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_copy(const gdn_pages_buffer* src, int32_t src_pages, const gdn_pages_buffer* dst, int32_t dst_pages,
                        int32_t n_buffers, const int32_t* src_list, const int32_t* dst_list, const int32_t* count, int32_t n,
                        int64_t most, const Remap& table, int32_t* status, cudaStream_t stream) {
    const auto launch = n_buffers <= 8 ? launch_copy_of<8> : launch_copy_of<GDN_PAGES_MAX_BUFFERS>;
    return launch(src, src_pages, dst, dst_pages, n_buffers, src_list, dst_list, count, n, most, table, status, stream);
}

bool workspace_ok(const gdn_pages_book* b, int32_t n, const void* workspace, size_t bytes) {
    return workspace && aligned(workspace, 16) && bytes >= make_layout(b->max_seqs, b->n_pages, n).total;
}

gdn_status last_launch() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

}  // namespace

extern "C" {

size_t gdn_pages_workspace_bytes(int32_t max_seqs, int32_t max_pages, int32_t n_pages, int32_t list) {
    if (max_seqs < 0 || max_pages < 0 || n_pages < 0 || list < 0) return 0;
    return make_layout(max_seqs, n_pages, list).total;
}

gdn_status gdn_pages_reserve_run(const gdn_pages_book* book, const int32_t* seqs, const int32_t* counts, int32_t n, int32_t* rows,
                                 int32_t* device_status, void* workspace, size_t workspace_bytes, void* stream) {
    if (!book_ok(book) || !list_ok(seqs, n) || !list_ok(counts, n) || !aligned(rows, 4) || !aligned(device_status, 4))
        return GDN_ERR_INVALID_ARG;
    if (!sums_ok(book, n)) return GDN_ERR_UNSUPPORTED;
    if (!workspace_ok(book, n, workspace, workspace_bytes)) return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    BookParams p = make_book(*book, n, workspace);
    p.seqs = seqs;
    p.counts = counts;
    p.rows = rows;
    p.status = device_status;
    gdn_pages_reserve_kernel<<<1, kBookThreads, sizeof(BookSmem), static_cast<cudaStream_t>(stream)>>>(p);
    return last_launch();
}

gdn_status gdn_pages_fork_run(const gdn_pages_book* book, const gdn_pages_buffer* buffers, int32_t n_buffers,
                              const int32_t* parents, const int32_t* children, int32_t n, int32_t page_tokens, int32_t* rows,
                              int32_t* device_status, void* workspace, size_t workspace_bytes, void* stream) {
    if (!book_ok(book) || !list_ok(parents, n) || !list_ok(children, n) || !aligned(rows, 4) || !aligned(device_status, 4) ||
        !buffers_ok(buffers, n_buffers) || page_tokens < 0 || (page_tokens > 0 && !book->lengths && book->max_seqs > 0))
        return GDN_ERR_INVALID_ARG;
    if (!sums_ok(book, n)) return GDN_ERR_UNSUPPORTED;
    if (!workspace_ok(book, n, workspace, workspace_bytes)) return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    BookParams p = make_book(*book, n, workspace);
    p.seqs = children;
    p.parents = parents;
    p.page_tokens = page_tokens;
    p.rows = rows;
    p.status = device_status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    gdn_pages_fork_kernel<<<1, kBookThreads, sizeof(BookSmem), st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    int64_t most = page_tokens > 0 ? n : static_cast<int64_t>(n) * book->max_pages;
    if (most > book->n_pages) most = book->n_pages;
    return launch_copy(buffers, book->n_pages, buffers, book->n_pages, n_buffers, p.copy_src, p.copy_dst, p.copy_count, 0, most,
                       Remap{}, device_status, st) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}

gdn_status gdn_pages_free_run(const gdn_pages_book* book, const int32_t* seqs, int32_t n, int32_t* device_status, void* stream) {
    if (!book_ok(book) || !list_ok(seqs, n) || !aligned(device_status, 4)) return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    BookParams p = make_book(*book, n, nullptr);
    p.seqs = seqs;
    p.status = device_status;
    gdn_pages_free_kernel<<<static_cast<unsigned>((static_cast<int64_t>(n) + 7) / 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return last_launch();
}

gdn_status gdn_pages_compact_run(const gdn_pages_book* book, const gdn_pages_buffer* buffers, int32_t n_buffers, int32_t* table_out,
                                 int32_t* refcounts_out, int32_t* remap, int32_t* n_live, int32_t* device_status, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (!book_ok(book) || !buffers_ok(buffers, n_buffers) || !n_live || !aligned(n_live, 4) || !aligned(table_out, 4) ||
        !aligned(refcounts_out, 4) || !aligned(remap, 4) || !aligned(device_status, 4))
        return GDN_ERR_INVALID_ARG;
    if ((book->n_pages > 0 && (!refcounts_out || !remap)) || (static_cast<int64_t>(book->max_seqs) * book->max_pages > 0 && !table_out))
        return GDN_ERR_INVALID_ARG;
    if (!workspace_ok(book, 0, workspace, workspace_bytes)) return GDN_ERR_INVALID_ARG;
    BookParams p = make_book(*book, 0, workspace);
    p.refcounts_out = refcounts_out;
    p.remap = remap;
    p.n_live = n_live;
    p.status = device_status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    gdn_pages_compact_kernel<<<1, kBookThreads, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    const Remap table{p.table, table_out, remap, static_cast<int64_t>(p.max_seqs) * p.max_pages, p.n_pages};
    return launch_copy(buffers, p.n_pages, buffers, p.n_pages, n_buffers, p.copy_src, p.copy_dst, p.copy_count, 0, p.n_pages / 2, table,
                       device_status, st) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}

gdn_status gdn_pages_copy_run(const gdn_pages_buffer* src_buffers, int32_t src_pages, const gdn_pages_buffer* dst_buffers,
                              int32_t dst_pages, int32_t n_buffers, const int32_t* src, const int32_t* dst, int32_t n,
                              int32_t* device_status, void* stream) {
    if (!buffers_ok(src_buffers, n_buffers) || !buffers_ok(dst_buffers, n_buffers) || src_pages < 0 || dst_pages < 0 ||
        !list_ok(src, n) || !list_ok(dst, n) || !aligned(device_status, 4))
        return GDN_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n_buffers; ++i)
        if (src_buffers[i].row_bytes != dst_buffers[i].row_bytes) return GDN_ERR_INVALID_ARG;
    return launch_copy(src_buffers, src_pages, dst_buffers, dst_pages, n_buffers, src, dst, nullptr, n, n, Remap{}, device_status,
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}

}  // extern "C"
