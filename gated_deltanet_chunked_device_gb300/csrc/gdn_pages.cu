// gdn_pages.cu -- page operators of a cache (include/gdn_pages.h): reserve,
// fork, free, compact and copy, kernels and host side.
//
// The bookkeeping of one call is done by one block of 1024 threads: its size
// is a few bytes a page and a few a table entry.  The pages' data are moved by
// a grid of its own, from lists that the first kernel left in the workspace;
// nothing returns to the host in between.
#include <climits>

#include "../../include/gdn_pages.h"
#include "gdn_internal.cuh"

namespace {

constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int64_t kPiece = 16384;  // bytes of a page that a block copies at a time

struct CopyBuffer {
    const uint8_t* src;
    uint8_t* dst;
    int64_t src_stride, dst_stride, bytes;
};

struct CopyParams {
    CopyBuffer buffers[GDN_PAGES_MAX_BUFFERS];
    int32_t n_buffers;
    int32_t src_pages, dst_pages;
    int64_t max_pieces;            // of the largest buffer's row
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
    int32_t* table_out;
    int32_t* refcounts_out;
    int32_t* remap;
    int32_t* n_live;
};

__device__ __forceinline__ void report(int32_t* status, int32_t bit) {
    if (status) atomicOr(status, bit);
}

// Numbers the i in [0, n) that pred holds for, in order: emit(rank, i) for each.  Warps own contiguous ranges; they
// count, the block sums the counts, and they go over their ranges again.  Returns how many there are.
template <class Pred, class Emit>
__device__ __forceinline__ int32_t number_in_order(int32_t n, int32_t* warp_sums, Pred pred, Emit emit) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t seg = ((static_cast<int64_t>(n) + kBookWarps - 1) / kBookWarps + 31) / 32 * 32;
    const int64_t from = warp * seg, to = from + seg < n ? from + seg : n;
    int32_t c = 0;
    for (int64_t i = from; i < to; i += 32) c += __popc(__ballot_sync(0xffffffffu, i + lane < to && pred(i + lane)));
    __syncthreads();
    if (lane == 0) warp_sums[warp] = c;
    __syncthreads();
    int32_t before = 0, total = 0;
    for (int w = 0; w < kBookWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    for (int64_t i = from; i < to; i += 32) {
        const bool on = i + lane < to && pred(i + lane);
        const uint32_t m = __ballot_sync(0xffffffffu, on);
        if (on) emit(before + __popc(m & ((1u << lane) - 1)), static_cast<int32_t>(i + lane));
        before += __popc(m);
    }
    return total;
}

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
    int32_t before = 0, total = 0;
    for (int w = 0; w < kBookWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
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
    return total;
}

// Of the entries of the list that name one sequence, the first one wins.
__device__ __forceinline__ void mark_sequences(const BookParams& p) {
    for (int64_t k = threadIdx.x; k < p.n; k += kBookThreads)
        if (p.seqs[k] >= 0 && p.seqs[k] < p.max_seqs) p.marks[p.seqs[k]] = INT_MAX;
    __syncthreads();
    for (int64_t k = threadIdx.x; k < p.n; k += kBookThreads)
        if (p.seqs[k] >= 0 && p.seqs[k] < p.max_seqs) atomicMin(&p.marks[p.seqs[k]], static_cast<int32_t>(k));
    __syncthreads();
}

__device__ __forceinline__ int32_t list_free_pages(const BookParams& p, int32_t wanted, int32_t* warp_sums) {
    return number_in_order(
        p.n_pages, warp_sums, [&](int64_t i) { return p.refcounts[i] <= 0; },
        [&](int32_t rank, int32_t page) {
            if (rank < wanted) p.free_list[rank] = page;
        });
}

__global__ void __launch_bounds__(kBookThreads) gdn_pages_reserve_kernel(BookParams p) {
    __shared__ int32_t warp_sums[kBookWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    mark_sequences(p);
    for (int64_t k = warp; k < p.n; k += kBookWarps) {
        const int32_t s = p.seqs[k], want = p.counts[k];
        const bool seq_ok = s >= 0 && s < p.max_seqs && p.marks[s] == k;
        const bool ok = seq_ok && want >= 0 && want <= p.max_pages;
        int32_t c = 0;
        if (ok)
            for (int32_t j = lane; j < want; j += 32) c += p.table[static_cast<int64_t>(s) * p.max_pages + j] < 0;
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) {
            p.need[k] = ok ? c : -1;
            if (!ok) report(p.status, seq_ok ? GDN_PAGES_ERR_PAGE : GDN_PAGES_ERR_SEQ);
        }
    }
    __syncthreads();
    const int32_t wanted = running_sums(p.n, p.need, p.offset, warp_sums);
    const int32_t n_free = list_free_pages(p, wanted, warp_sums);
    __syncthreads();
    if (wanted > n_free && threadIdx.x == 0) report(p.status, GDN_PAGES_ERR_NO_PAGES);
    for (int64_t k = warp; k < p.n; k += kBookWarps) {
        const int32_t need = p.need[k], off = p.offset[k];
        const bool served = need >= 0 && off + need <= n_free;
        const int64_t row = need >= 0 ? static_cast<int64_t>(p.seqs[k]) * p.max_pages : 0;
        const int32_t want = served ? p.counts[k] : 0;
        int32_t at = off;
        for (int32_t j0 = 0; j0 < p.max_pages; j0 += 32) {
            const int32_t j = j0 + lane;
            int32_t e = need >= 0 && j < p.max_pages ? p.table[row + j] : -1;
            const bool take = j < want && e < 0;
            const uint32_t m = __ballot_sync(0xffffffffu, take);
            if (take) {
                e = p.free_list[at + __popc(m & ((1u << lane) - 1))];
                p.table[row + j] = e;
                p.refcounts[e] = 1;
            }
            at += __popc(m);
            if (p.rows && j < p.max_pages) p.rows[k * p.max_pages + j] = e;
        }
    }
}

__global__ void __launch_bounds__(kBookThreads) gdn_pages_fork_kernel(BookParams p) {
    __shared__ int32_t warp_sums[kBookWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    mark_sequences(p);
    for (int64_t k = warp; k < p.n; k += kBookWarps) {
        const int32_t par = p.parents[k], child = p.seqs[k];
        int32_t fault = 0, need = 0, used = 0, len = 0;
        if (par < 0 || par >= p.max_seqs || child < 0 || child >= p.max_seqs || par == child || p.marks[child] != k)
            fault = GDN_PAGES_ERR_SEQ;
        if (!fault) {
            int32_t has = 0;
            for (int32_t j = lane; j < p.max_pages; j += 32) has |= p.table[static_cast<int64_t>(child) * p.max_pages + j] >= 0;
            if (__any_sync(0xffffffffu, has)) fault = GDN_PAGES_ERR_CHILD;
        }
        if (!fault) {
            len = p.lengths ? p.lengths[par] : 0;
            used = p.max_pages;
            if (p.page_tokens > 0) {
                const int64_t n = len < 0 ? -1 : (static_cast<int64_t>(len) + p.page_tokens - 1) / p.page_tokens;
                if (n < 0 || n > p.max_pages) fault = GDN_PAGES_ERR_PAGE;
                used = static_cast<int32_t>(fault ? 0 : n);
            }
            int32_t bad = 0, c = 0;
            for (int32_t j = lane; j < used; j += 32) {
                const int32_t e = p.table[static_cast<int64_t>(par) * p.max_pages + j];
                bad |= e >= p.n_pages || (p.page_tokens > 0 && e < 0);
                c += e >= 0;
            }
            if (__any_sync(0xffffffffu, bad)) fault = GDN_PAGES_ERR_PAGE;
            c = __reduce_add_sync(0xffffffffu, c);
            need = p.page_tokens > 0 ? (len % p.page_tokens != 0) : c;
            if (p.page_tokens == 0 && c == 0) used = 0;  // nothing yet, whatever another entry of the list gives this parent
        }
        if (lane == 0) {
            p.need[k] = fault ? -1 : need;
            p.used[k] = used;
            p.plen[k] = len;
            if (fault) report(p.status, fault);
        }
    }
    __syncthreads();
    const int32_t wanted = running_sums(p.n, p.need, p.offset, warp_sums);
    const int32_t n_free = list_free_pages(p, wanted, warp_sums);
    __syncthreads();
    if (wanted > n_free && threadIdx.x == 0) report(p.status, GDN_PAGES_ERR_NO_PAGES);
    int32_t most = 0;  // pairs: the entries served are the first ones
    for (int64_t k = warp; k < p.n; k += kBookWarps) {
        const int32_t need = p.need[k], off = p.offset[k];
        const bool served = need >= 0 && off + need <= n_free;
        const int32_t child = served || need >= 0 ? p.seqs[k] : 0;
        const int64_t prow = served ? static_cast<int64_t>(p.parents[k]) * p.max_pages : 0;
        const int32_t used = served ? p.used[k] : 0;
        int32_t at = off;
        for (int32_t j0 = 0; j0 < p.max_pages; j0 += 32) {
            const int32_t j = j0 + lane;
            int32_t e = j < used ? p.table[prow + j] : -1;
            const bool copy = e >= 0 && (p.page_tokens == 0 || (need > 0 && j == used - 1));
            const uint32_t m = __ballot_sync(0xffffffffu, copy);
            if (copy) {
                const int32_t place = at + __popc(m & ((1u << lane) - 1));
                const int32_t fresh = p.free_list[place];
                p.copy_src[place] = e;
                p.copy_dst[place] = fresh;
                p.refcounts[fresh] = 1;
                e = fresh;
            } else if (e >= 0) {
                atomicAdd(&p.refcounts[e], 1);
            }
            at += __popc(m);
            if (served && j < p.max_pages) p.table[static_cast<int64_t>(child) * p.max_pages + j] = e;
            if (p.rows && j < p.max_pages) p.rows[k * p.max_pages + j] = e;
        }
        if (lane == 0 && p.lengths && need >= 0) p.lengths[child] = served ? p.plen[k] : 0;
        if (served) most = max(most, off + need);
    }
    __syncthreads();
    if (lane == 0) warp_sums[warp] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kBookWarps; ++w) most = max(most, warp_sums[w]);
        *p.copy_count = most;
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
        [&](int32_t rank, int32_t page) { p.copy_src[rank] = page; });
    number_in_order(
        p.n_pages, warp_sums, [&](int64_t i) { return i < L && p.refcounts[i] <= 0; },
        [&](int32_t rank, int32_t page) { p.copy_dst[rank] = page; });
    __syncthreads();
    for (int64_t i = threadIdx.x; i < p.n_pages; i += kBookThreads) p.remap[i] = p.refcounts[i] > 0 ? static_cast<int32_t>(i) : -1;
    __syncthreads();
    for (int64_t k = threadIdx.x; k < moves; k += kBookThreads) {
        p.remap[p.copy_src[k]] = p.copy_dst[k];
        p.free_list[k] = p.refcounts[p.copy_src[k]];  // the count that moves with the page
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < p.n_pages; i += kBookThreads) p.refcounts_out[i] = i < L ? p.refcounts[i] : 0;
    __syncthreads();
    for (int64_t k = threadIdx.x; k < moves; k += kBookThreads) p.refcounts_out[p.copy_dst[k]] = p.free_list[k];
    if (threadIdx.x == 0) {
        *p.copy_count = moves;
        *p.n_live = L;
    }
}

__global__ void gdn_pages_remap_kernel(BookParams p) {
    const int64_t n = static_cast<int64_t>(p.max_seqs) * p.max_pages;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int32_t e = p.table[i];
        if (e < -1 || e >= p.n_pages) report(p.status, GDN_PAGES_ERR_PAGE);
        p.table_out[i] = e >= 0 && e < p.n_pages ? p.remap[e] : -1;
    }
}

// Copies rows: a unit is one piece of one buffer's row of one pair.
__global__ void __launch_bounds__(kCopyThreads) gdn_pages_copy_kernel(const __grid_constant__ CopyParams p) {
    const int64_t pairs = p.count ? *p.count : p.n;
    const int64_t units = pairs * p.n_buffers * p.max_pieces;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t piece = unit % p.max_pieces, b = unit / p.max_pieces % p.n_buffers, k = unit / p.max_pieces / p.n_buffers;
        const int32_t s = p.src[k], d = p.dst[k];
        if (s < 0 || d < 0) continue;
        if (s >= p.src_pages || d >= p.dst_pages) {
            if (threadIdx.x == 0) report(p.status, GDN_PAGES_ERR_PAGE);
            continue;
        }
        const CopyBuffer& f = p.buffers[b];
        const int64_t from = piece * kPiece, to = from + kPiece < f.bytes ? from + kPiece : f.bytes;
        const uint8_t* src = f.src + s * f.src_stride;
        uint8_t* dst = f.dst + d * f.dst_stride;
        for (int64_t i = from + threadIdx.x; i < to; i += kCopyThreads) dst[i] = src[i];
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

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    return n > 0 ? n : 1;
}

// most: an upper bound of the pairs.
cudaError_t launch_copy(const gdn_pages_buffer* src, int32_t src_pages, const gdn_pages_buffer* dst, int32_t dst_pages,
                        int32_t n_buffers, const int32_t* src_list, const int32_t* dst_list, const int32_t* count, int32_t n,
                        int64_t most, int32_t* status, cudaStream_t stream) {
    CopyParams p{};
    int32_t used = 0;
    for (int32_t i = 0; i < n_buffers; ++i) {
        if (src[i].row_bytes == 0) continue;
        p.buffers[used++] = {static_cast<const uint8_t*>(src[i].base), static_cast<uint8_t*>(dst[i].base), src[i].row_stride,
                             dst[i].row_stride, src[i].row_bytes};
        const int64_t pieces = (src[i].row_bytes + kPiece - 1) / kPiece;
        if (pieces > p.max_pieces) p.max_pieces = pieces;
    }
    if (used == 0 || most == 0) return cudaSuccess;
    p.n_buffers = used;
    p.src_pages = src_pages;
    p.dst_pages = dst_pages;
    p.src = src_list;
    p.dst = dst_list;
    p.count = count;
    p.n = n;
    p.status = status;
    const int64_t units = most * used * p.max_pieces, cap = 8 * sm_count();
    gdn_pages_copy_kernel<<<static_cast<unsigned>(units < cap ? units : cap), kCopyThreads, 0, stream>>>(p);
    return cudaGetLastError();
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
    gdn_pages_reserve_kernel<<<1, kBookThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
    gdn_pages_fork_kernel<<<1, kBookThreads, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    int64_t most = page_tokens > 0 ? n : static_cast<int64_t>(n) * book->max_pages;
    if (most > book->n_pages) most = book->n_pages;
    return launch_copy(buffers, book->n_pages, buffers, book->n_pages, n_buffers, p.copy_src, p.copy_dst, p.copy_count, 0, most,
                       device_status, st) == cudaSuccess
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
    p.table_out = table_out;
    p.refcounts_out = refcounts_out;
    p.remap = remap;
    p.n_live = n_live;
    p.status = device_status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    gdn_pages_compact_kernel<<<1, kBookThreads, 0, st>>>(p);
    const int64_t entries = static_cast<int64_t>(p.max_seqs) * p.max_pages;
    if (entries > 0) {
        const int64_t blocks = (entries + 255) / 256, cap = 8 * sm_count();
        gdn_pages_remap_kernel<<<static_cast<unsigned>(blocks < cap ? blocks : cap), 256, 0, st>>>(p);
    }
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    return launch_copy(buffers, p.n_pages, buffers, p.n_pages, n_buffers, p.copy_src, p.copy_dst, p.copy_count, 0, p.n_pages / 2,
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
    return launch_copy(src_buffers, src_pages, dst_buffers, dst_pages, n_buffers, src, dst, nullptr, n, n, device_status,
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}

}  // extern "C"
