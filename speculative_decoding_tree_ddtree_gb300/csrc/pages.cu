// pages.cu -- sequences that share, take over, give back and close up the pages
// of the KV pool: lucetree_reorder_pages, lucetree_trim_pages and
// lucetree_compact_pages work on page tables and reference counts (integers,
// a few launches, bound by launch and memory latency);
// lucetree_copy_pages and lucetree_reorder_states move the data they ask for
// (bound by HBM: every byte is read once and written once; 652 MB in 97 us).
//
// Free pages are found by rank, not by search: the pool is cut into chunks of
// kChunk pages, each with a bit mask of its free (or used) pages and their
// count, so the k-th one is a short scan of the counts, one popcount scan of 32
// words and a bit select.  Every result depends on the inputs alone: ranks
// follow page and row numbers, and the only atomics are integer additions.
#include "internal.cuh"
#include "pages.h"

namespace lucetree {

namespace {

constexpr int kChunk = 1024;            // pages per chunk: one thread each, 32 mask words
constexpr int kCols = 1024;             // table columns per CTA
constexpr int kThreads = 256;
constexpr int kMaxTail = 64;            // tail pages of a row (one 64-bit mask)
// Up to these sizes one CTA does the whole of a call: a launch more costs as much as its
// pass over a few pages and rows, a warp to a row.  One CTA against several launches, us of
// GPU time (rows in and out alike x columns, pages of the pool):
//   reorder   4 x 16, 1,500  6.6 / 7.2   16 x 64, 1,500  7.0 / 7.5   16 x 96, 1,500  7.2 / 7.4
//             16 x 64, 4,096 7.8 / 7.4   24 x 32, 1,500  7.9 / 7.3   1 x 512, 412    7.9 / 6.5
//   trim      4 x 16, 1,500  2.4 / 3.2   16 x 64, 1,500  3.1 / 3.1   32 x 16, 1,500  2.6 / 3.1
//             15 x 60, 4,096 3.5 / 3.3   48 x 16, 1,500  3.1 / 3.1   16 x 96, 1,500  3.8 / 3.1
//             counts in place (one launch either way)  4 x 16  2.0 / 1.9   16 x 64  2.7 / 1.8
//   compact   16 x 64, 1,500 4.7 / 6.7   32 x 64, 1,793  4.9 / 6.2   1 x 2,048, 2,028 4.9 / 5.9
//             16 x 64, 4,096 8.1 / 6.6   64 x 64, 3,546  8.5 / 6.7
constexpr int kSmallPages = 2048, kSmallRows = 32, kSmallCols = 96, kSmallTrimCols = 64, kSmallEntries = 2048;
constexpr int kMaxPages = 1 << 30;      // chunk and page numbers stay within an int
// ... and so do row and column numbers with one more step of a kernel's loop (65,535 rows, kCols columns)
constexpr int kMaxRows = 0x7fffffff - 65535, kMaxCols = 0x7fffffff - kCols;

int chunks_of(int num_pages) { return (num_pages + kChunk - 1) / kChunk; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// ---------------------------------------------------------------- reorder

// What the rows' plan leaves for the apply kernel.
struct ReorderPlan {
    int32_t* children;   // [rows_in] rows that take this one
    int32_t* first;      // [rows_in] the lowest of them
    uint64_t* kept;      // [rows_in] bit k: tail page full + k stays with the first of them
    int32_t* base;       // [rows_out] rank of the row's first new page among the free ones
    uint32_t* free_bits;  // [chunks][32]
    int32_t* free_count;  // [chunks]
};

struct ReorderLaunch {
    lucetree_reorder_args a;
    ReorderPlan w;
    int chunks;
};

struct RowSpan {
    int L, full, end;  // committed length, whole pages, pages with the reserve
    bool ok;
};

// The pages that row b's length and the reserve take.  `goes_on`: some new row maps the reserve.
__device__ inline RowSpan row_span(const lucetree_reorder_args& a, int b, uint32_t* status, bool goes_on = false) {
    RowSpan s{a.ctx_in[b], 0, 0, true};
    if (s.L < 0 || (long long)s.L > (long long)a.max_pages_per_seq * kPage) {
        if (status) atomicOr(status, LUCETREE_DEV_BAD_CTX);
        s.ok = false;
        s.L = 0;
        return s;
    }
    s.full = s.L / kPage;
    const long long end = ((long long)s.L + a.reserve + kPage - 1) / kPage;
    if (end > a.max_pages_per_seq && goes_on) atomicOr(status, LUCETREE_DEV_BAD_CTX);
    s.end = (int)(end < a.max_pages_per_seq ? end : a.max_pages_per_seq);
    return s;
}

// Source row of out row r, -1 when it stays empty (none, out of range, or a bad length).
__device__ inline int source_row(const lucetree_reorder_args& a, int r, uint32_t* status) {
    const int b = a.src[r];
    if (b < -1 || b >= a.rows_in) {
        if (status) atomicOr(status, LUCETREE_DEV_BAD_ROW);
        return -1;
    }
    return b;
}

__device__ inline bool page_ok(int page, int num_pages) { return page >= 0 && page < num_pages; }

// Inclusive sum over the CTA (kChunk threads); s_warp: one int per warp.
__device__ inline int block_scan(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
        const int x = s_warp[w];
        before += w < warp ? x : 0;
        all += x;
    }
    *total = all;
    return v + before;
}

// Pages [chunk kChunk, (chunk + 1) kChunk): free mask, count, and the copy of the
// reference counts (kChunk threads).
__device__ inline void scan_pages(const ReorderLaunch& R, int chunk, int* s_warp) {
    const lucetree_reorder_args& a = R.a;
    const int t = threadIdx.x, page = chunk * kChunk + t;
    const int ref = page < a.num_pages ? a.ref_in[page] : -1;
    if (page < a.num_pages && a.ref_out != a.ref_in) a.ref_out[page] = ref;
    const unsigned free = __ballot_sync(0xffffffffu, ref == 0);
    if ((t & 31) == 0) {
        R.w.free_bits[chunk * 32 + (t >> 5)] = free;
        s_warp[t >> 5] = __popc(free);
    }
    __syncthreads();
    if (t == 0) {
        int n = 0;
        for (int w = 0; w < 32; ++w) n += s_warp[w];
        R.w.free_count[chunk] = n;
    }
    __syncthreads();
}

// (the plan's counters are updated by atomics: read past the L1 cache, or from shared memory)
__device__ inline int now(const int32_t* p) { return *(const volatile int32_t*)p; }

// Who takes which row, what stays with it, and where its new pages start (kChunk threads).
__device__ inline void plan_rows(const ReorderLaunch& R, int* s_warp) {
    const lucetree_reorder_args& a = R.a;
    const int t = threadIdx.x;
    for (int b = t; b < a.rows_in; b += kChunk) {
        R.w.children[b] = 0;
        R.w.first[b] = 0x7fffffff;
    }
    __syncthreads();
    for (int r = t; r < a.rows_out; r += kChunk) {
        const int b = source_row(a, r, a.status);
        if (b < 0) continue;
        atomicAdd(&R.w.children[b], 1);
        atomicMin(&R.w.first[b], r);
    }
    __syncthreads();
    // tail pages that no other row holds stay with the first row that takes the parent
    for (int b = t; b < a.rows_in; b += kChunk) {
        uint64_t kept = 0;
        const bool goes_on = now(&R.w.children[b]) > 0;
        const RowSpan s = row_span(a, b, a.status, goes_on);
        if (goes_on)
            for (int c = s.full; c < s.end; ++c) {
                const int page = a.table_in[(size_t)b * a.max_pages_per_seq + c];
                if (page_ok(page, a.num_pages) && a.ref_in[page] == 1) kept |= 1ull << (c - s.full);
            }
        R.w.kept[b] = kept;
    }
    __syncthreads();
    // new pages in the order of rows
    int before = 0;
    for (int r0 = 0; r0 < a.rows_out; r0 += kChunk) {
        const int r = r0 + t;
        int need = 0;
        if (r < a.rows_out) {
            const int b = source_row(a, r, nullptr);
            if (b >= 0) {
                const RowSpan s = row_span(a, b, nullptr);
                need = s.end - s.full;
                if (now(&R.w.first[b]) == r) need -= __popcll(R.w.kept[b]);
            }
        }
        int all;
        const int upto = block_scan(need, s_warp, &all);
        if (r < a.rows_out) R.w.base[r] = before + upto - need;
        before += all;
    }
}

// The page with rank k among the free ones (-1: there are not so many), by the whole warp.
__device__ inline int free_page(const ReorderPlan& w, int chunks, int k) {
    const int lane = threadIdx.x & 31;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
        const int n = c0 + lane < chunks ? w.free_count[c0 + lane] : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const unsigned has = __ballot_sync(0xffffffffu, k < incl);
        if (!has) {
            k -= __shfl_sync(0xffffffffu, incl, 31);
            continue;
        }
        const int l = __ffs(has) - 1;
        k -= __shfl_sync(0xffffffffu, incl - n, l);
        const int chunk = c0 + l;
        const uint32_t bits = w.free_bits[chunk * 32 + lane];
        int upto = __popc(bits);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const int wl = __ffs(__ballot_sync(0xffffffffu, k < upto)) - 1;
        const int left = k - __shfl_sync(0xffffffffu, upto - __popc(bits), wl);
        const uint32_t word = __shfl_sync(0xffffffffu, bits, wl);
        return chunk * kChunk + wl * 32 + (int)__fns(word, 0, left + 1);
    }
    return -1;
}

// Whether table entry `page` names a page that has a holder.  A free one may be handed to a
// new row in this very call, so it is read as if it were missing.
__device__ inline bool held_page(const ReorderLaunch& R, int page) {
    return page_ok(page, R.a.num_pages) && !((R.w.free_bits[page >> 5] >> (page & 31)) & 1u);
}

// Columns [c0, c1) of row y: y < rows_out: the new rows; behind them the old ones, whose
// pages gain a holder for each row that takes them and lose the old one.  The
// thread is number t of n, whole warps.
__device__ inline void apply_row(const ReorderLaunch& R, int y, int c0, int c1, int t, int n) {
    const lucetree_reorder_args& a = R.a;
    const int P = a.max_pages_per_seq;
    if (y >= a.rows_out) {
        const int b = y - a.rows_out;
        const RowSpan s = row_span(a, b, nullptr);
        if (!s.ok) return;  // a row of unknown length keeps its pages
        const int children = now(&R.w.children[b]);
        const uint64_t kept = R.w.kept[b];
        for (int c = c0 + t; c < c1; c += n) {
            const int page = a.table_in[(size_t)b * P + c];
            if (page == -1) continue;
            if (!held_page(R, page)) {
                atomicOr(a.status, LUCETREE_DEV_BAD_PAGE);
                continue;
            }
            int delta = -1;
            if (c < s.full) delta = children - 1;
            else if (c < s.end && ((kept >> (c - s.full)) & 1)) delta = 0;
            if (delta != 0 && atomicAdd(a.ref_out + page, delta) + delta < 0) atomicOr(a.status, LUCETREE_DEV_BAD_PAGE);
        }
        return;
    }
    const int r = y;
    int b = source_row(a, r, nullptr);
    RowSpan s{0, 0, 0, false};
    if (b >= 0) s = row_span(a, b, nullptr);
    if (!s.ok) b = -1;
    int32_t* out = a.table_out + (size_t)r * P;
    const int32_t* in = a.table_in + (size_t)(b < 0 ? 0 : b) * P;
    for (int c = c0 + t; c < c1; c += n) {
        if (c >= s.full && c < s.end) continue;
        int page = -1;
        if (b >= 0 && c < s.full) {
            page = in[c];
            if (!held_page(R, page)) page = -1;
        }
        out[c] = page;
    }
    if (c0 > 0) return;
    // the tail, a warp to a page
    const int warp = t >> 5, lane = t & 31;
    const uint64_t kept = b >= 0 && now(&R.w.first[b]) == r ? R.w.kept[b] : 0;
    for (int c = s.full + warp; c < s.end; c += n / 32) {
        const int k = c - s.full, old = in[c];
        if ((kept >> k) & 1) {
            if (lane == 0) out[c] = old;
            continue;
        }
        const int rank = R.w.base[r] + k - __popcll(kept & ((1ull << k) - 1));
        const int page = free_page(R.w, R.chunks, rank);
        if (lane == 0) {
            out[c] = page;
            if (page < 0) atomicOr(a.status, LUCETREE_DEV_NO_PAGE);
            else a.ref_out[page] = 1;
            if (k == 0) {
                const bool copy = s.L % kPage != 0 && page >= 0 && held_page(R, old);
                a.copy_src[r] = copy ? old : -1;
                a.copy_dst[r] = copy ? page : -1;
            }
        }
    }
    if (t == 0) {
        a.ctx_out[r] = s.L;
        if (s.full >= s.end || (kept & 1)) a.copy_src[r] = a.copy_dst[r] = -1;
    }
}

// CTA 0 plans the rows, CTA 1 + i takes chunk i of the pages.
__global__ void __launch_bounds__(kChunk) reorder_plan_kernel(ReorderLaunch R) {
    __shared__ int s_warp[kChunk / 32];
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    if (blockIdx.x == 0) plan_rows(R, s_warp);
    else scan_pages(R, blockIdx.x - 1, s_warp);
}

__global__ void __launch_bounds__(kThreads) reorder_apply_kernel(ReorderLaunch R) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int c0 = blockIdx.x * kCols, c1 = min(R.a.max_pages_per_seq, c0 + kCols);
    for (int y = blockIdx.y; y < R.a.rows_in + R.a.rows_out; y += gridDim.y) apply_row(R, y, c0, c1, threadIdx.x, kThreads);
}

// Both in one CTA, with the plan in shared memory: a warp to a row.
__global__ void __launch_bounds__(kChunk) reorder_small_kernel(ReorderLaunch R) {
    __shared__ int s_warp[kChunk / 32];
    __shared__ int32_t s_children[kSmallRows], s_first[kSmallRows], s_base[kSmallRows];
    __shared__ uint64_t s_kept[kSmallRows];
    __shared__ uint32_t s_bits[kSmallPages / 32];
    __shared__ int32_t s_count[kSmallPages / kChunk];
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    R.w = ReorderPlan{s_children, s_first, s_kept, s_base, s_bits, s_count};
    for (int c = 0; c < R.chunks; ++c) scan_pages(R, c, s_warp);
    plan_rows(R, s_warp);
    __syncthreads();
    for (int y = threadIdx.x >> 5; y < R.a.rows_in + R.a.rows_out; y += kChunk / 32)
        apply_row(R, y, 0, R.a.max_pages_per_seq, threadIdx.x & 31, 32);
}

// ---------------------------------------------------------------- trim

// Columns [c0, c1) of row b, by thread t of n.
__device__ inline void trim_row(const lucetree_trim_args& a, int b, int c0, int c1, int t, int n) {
    const int P = a.max_pages_per_seq;
    int L = a.ctx_len[b];
    if (L < 0 || (long long)L > (long long)P * kPage) {
        if (t == 0 && c0 == 0) atomicOr(a.status, LUCETREE_DEV_BAD_CTX);
        L = 0;  // nothing of it is known to lie behind the window
    }
    // pages [sp, wp) hold no sink and nothing that the window of the next token reaches
    const int lo = max(L - a.window + 1, 0);
    const int sp = a.sinks / kPage + (a.sinks % kPage != 0), wp = lo / kPage;
    for (int c = c0 + t; c < c1; c += n) {
        const int page = a.table_in[(size_t)b * P + c];
        const bool gone = c >= sp && c < wp;
        if (gone && page != -1) {
            if (!page_ok(page, a.num_pages) || atomicSub(a.ref_out + page, 1) <= 0)
                atomicOr(a.status, LUCETREE_DEV_BAD_PAGE);
        }
        if (gone || a.table_out != a.table_in) a.table_out[(size_t)b * P + c] = gone ? -1 : page;
    }
}

__global__ void __launch_bounds__(kThreads) trim_kernel(lucetree_trim_args a) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int c0 = blockIdx.x * kCols, c1 = min(a.max_pages_per_seq, c0 + kCols);
    for (int b = blockIdx.y; b < a.rows; b += gridDim.y) trim_row(a, b, c0, c1, threadIdx.x, kThreads);
}

__global__ void __launch_bounds__(kThreads) copy_counts_kernel(const int32_t* from, int32_t* to, int n) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const long long i = ((long long)blockIdx.x * 4 + k) * kThreads + threadIdx.x;
        if (i < n) to[i] = from[i];
    }
}

// The same in one CTA, counts copied first.
__global__ void __launch_bounds__(kChunk) trim_small_kernel(lucetree_trim_args a) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    for (int p = threadIdx.x; p < a.num_pages; p += kChunk) a.ref_out[p] = a.ref_in[p];
    __syncthreads();
    for (int b = threadIdx.x >> 5; b < a.rows; b += kChunk / 32)
        trim_row(a, b, 0, a.max_pages_per_seq, threadIdx.x & 31, 32);
}

// ---------------------------------------------------------------- compact

struct CompactLaunch {
    lucetree_compact_args a;
    int32_t* used_count;  // [chunks]
    int32_t* rank;        // [num_pages] -1: free; else of a page at or past the live count: its place among the movers
    int chunks;
};

__global__ void __launch_bounds__(kChunk) compact_count_kernel(CompactLaunch C) {
    __shared__ int s_warp[kChunk / 32];
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int page = blockIdx.x * kChunk + threadIdx.x;
    const bool used = page < C.a.num_pages && C.a.ref_in[page] > 0;
    const int n = __popc(__ballot_sync(0xffffffffu, used));
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        int all = 0;
        for (int w = 0; w < kChunk / 32; ++w) all += s_warp[w];
        C.used_count[blockIdx.x] = all;
    }
}

// Ranks: with `live` used pages, the used ones at or past `live` move, in order,
// to the free ones before it.
__global__ void __launch_bounds__(kChunk) compact_rank_kernel(CompactLaunch C) {
    const lucetree_compact_args& a = C.a;
    __shared__ int s_warp[kChunk / 32];
    __shared__ int s_sum[3];
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int t = threadIdx.x, chunk = blockIdx.x;
    if (t < 3) s_sum[t] = 0;
    __syncthreads();
    int before = 0, all = 0;
    for (int c = t; c < C.chunks; c += kChunk) {
        const int n = C.used_count[c];
        all += n;
        before += c < chunk ? n : 0;
    }
    atomicAdd(&s_sum[0], before);
    atomicAdd(&s_sum[1], all);
    __syncthreads();
    const int live = s_sum[1], first = s_sum[0];
    // used pages before page `live`: whole chunks, and the part of the chunk it lies in
    const int lc = live / kChunk;
    int low = 0;
    for (int c = t; c < lc; c += kChunk) low += C.used_count[c];
    const int p = lc * kChunk + t;
    if (p < live && p < a.num_pages && a.ref_in[p] > 0) ++low;
    atomicAdd(&s_sum[2], low);
    __syncthreads();
    const int low_used = s_sum[2], movers = live - low_used;
    const int page = chunk * kChunk + t;
    const bool used = page < a.num_pages && a.ref_in[page] > 0;
    int n;
    const int used_before = first + block_scan(used ? 1 : 0, s_warp, &n) - (used ? 1 : 0);
    if (page < a.num_pages) {
        if (page >= live) {
            const int k = used ? used_before - low_used : -1;
            C.rank[page] = k;
            if (used) a.copy_src[k] = page;
        } else {
            C.rank[page] = used ? 0 : -1;
            if (!used) a.copy_dst[page - used_before] = page;
        }
    }
    const int cap = a.num_pages / 2;  // no more pages can move
    for (int i = movers + chunk * kChunk + t; i < cap; i += C.chunks * kChunk) a.copy_src[i] = a.copy_dst[i] = -1;
    if (chunk == 0 && t == 0) {
        *a.live = live;
        *a.copy_n = movers;
    }
}

// Tables and reference counts under the new names; every table entry and every
// count is touched by one thread, so outputs may be the inputs.
__global__ void __launch_bounds__(kThreads) compact_apply_kernel(CompactLaunch C) {
    const lucetree_compact_args& a = C.a;
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int live = *a.live;
    const long long step = (long long)gridDim.x * kThreads, at = (long long)blockIdx.x * kThreads + threadIdx.x;
    for (long long p = at; p < a.num_pages; p += step) {
        const int ref = a.ref_in[p];
        if (p < live) {
            if (ref > 0) a.ref_out[p] = ref;  // a free one gets its count from the page that moves there
        } else if (ref > 0) {
            a.ref_out[a.copy_dst[C.rank[p]]] = ref;
            a.ref_out[p] = 0;
        } else {
            a.ref_out[p] = ref;
        }
    }
    const long long n = (long long)a.rows * a.max_pages_per_seq;
    for (long long e = at; e < n; e += step) {
        int page = a.table_in[e];
        if (page != -1) {
            if (!page_ok(page, a.num_pages) || C.rank[page] < 0) {
                atomicOr(a.status, LUCETREE_DEV_BAD_PAGE);
                page = -1;
            } else if (page >= live) {
                page = a.copy_dst[C.rank[page]];
            }
        }
        a.table_out[e] = page;
    }
}

// All of it in one CTA: each thread keeps the counts of its pages, and the new names
// stay in shared memory.
__global__ void __launch_bounds__(kChunk) compact_small_kernel(CompactLaunch C) {
    constexpr int kMine = kSmallPages / kChunk;
    const lucetree_compact_args& a = C.a;
    __shared__ int s_warp[kChunk / 32];
    __shared__ int16_t s_name[kSmallPages];      // new number of a page, -1 if free
    __shared__ int16_t s_hole[kSmallPages / 2];  // free pages before it
    static_assert(kSmallPages <= 32767 + 1, "page numbers in 16 bits");
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int t = threadIdx.x;
    int ref[kMine], used_before[kMine], live = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int p = i * kChunk + t;
        ref[i] = p < a.num_pages ? a.ref_in[p] : 0;
        used_before[i] = 0;
        if (i >= C.chunks) continue;  // the same for all threads
        int n;
        used_before[i] = live + block_scan(ref[i] > 0 ? 1 : 0, s_warp, &n) - (ref[i] > 0 ? 1 : 0);
        live += n;
    }
    int low = 0, low_used;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int p = i * kChunk + t;
        low += p < live && ref[i] > 0;
        if (p < live && ref[i] <= 0) s_hole[p - used_before[i]] = (int16_t)p;
    }
    block_scan(low, s_warp, &low_used);  // (and every hole is written)
    const int movers = live - low_used;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int p = i * kChunk + t;
        if (p >= a.num_pages) continue;
        if (p < live) {
            s_name[p] = ref[i] > 0 ? (int16_t)p : (int16_t)-1;
            if (ref[i] > 0 && a.ref_out != a.ref_in) a.ref_out[p] = ref[i];
        } else if (ref[i] > 0) {
            const int k = used_before[i] - low_used, to = s_hole[k];
            s_name[p] = (int16_t)to;
            a.copy_src[k] = p;
            a.copy_dst[k] = to;
            a.ref_out[to] = ref[i];
            a.ref_out[p] = 0;
        } else {
            s_name[p] = -1;
            a.ref_out[p] = ref[i];
        }
    }
    for (int i = movers + t; i < a.num_pages / 2; i += kChunk) a.copy_src[i] = a.copy_dst[i] = -1;
    if (t == 0) {
        *a.live = live;
        *a.copy_n = movers;
    }
    __syncthreads();
    const int n = a.rows * a.max_pages_per_seq;
    for (int e = t; e < n; e += kChunk) {
        int page = a.table_in[e];
        if (page != -1) {
            const int name = page_ok(page, a.num_pages) ? s_name[page] : -1;
            if (name < 0) atomicOr(a.status, LUCETREE_DEV_BAD_PAGE);
            page = name;
        }
        a.table_out[e] = page;
    }
}

// ---------------------------------------------------------------- copies

// Copies of rows of 16-byte units: pair i copies row src[i] of `from` to row
// dst[i] (dst null: row i) of `to`, for up to two arrays with the same pairs.
// A work item is a slice of one row, kUnroll units a thread with all loads
// issued before the first store.
struct CopyLaunch {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;  // pairs in use (null: n)
    int n;
    int rows_from, rows_to;
    const uint4* from[2];
    uint4* to[2];
    long long units[2];   // of one row
    long long slices[2];  // per row
    uint32_t bad;         // flag of an index out of range
    uint32_t* status;
};

constexpr int kUnroll = 8;
constexpr int kSlice = kThreads * kUnroll;  // 16-byte units: 32 KB

__global__ void __launch_bounds__(kThreads) copy_rows_kernel(CopyLaunch C) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    int n = C.n;
    if (C.count) n = max(0, min(n, *C.count));
    const long long per = C.slices[0] + C.slices[1];
    for (long long item = blockIdx.x; item < n * per; item += gridDim.x) {
        const int i = (int)(item / per);
        const long long s = item % per;
        const int which = s >= C.slices[0];
        const long long u0 = (which ? s - C.slices[0] : s) * kSlice + threadIdx.x;
        const int from = C.src[i], to = C.dst ? C.dst[i] : (from == -1 ? -1 : i);
        if (from == -1 && to == -1) continue;
        if (from < 0 || from >= C.rows_from || to < 0 || to >= C.rows_to) {
            if (s == 0 && threadIdx.x == 0) atomicOr(C.status, C.bad);
            continue;
        }
        const long long units = which ? C.units[1] : C.units[0];
        const uint4* x = (which ? C.from[1] : C.from[0]) + (long long)from * units;
        uint4* y = (which ? C.to[1] : C.to[0]) + (long long)to * units;
        uint4 v[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (u0 + k * kThreads < units) v[k] = __ldcs(x + u0 + k * kThreads);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (u0 + k * kThreads < units) y[u0 + k * kThreads] = v[k];
    }
}

cudaError_t launch_copy(CopyLaunch& C, cudaStream_t stream) {
    for (int w = 0; w < 2; ++w) C.slices[w] = (C.units[w] + kSlice - 1) / kSlice;
    int dev = 0;
    cudaGetDevice(&dev);
    const long long items = C.n * (C.slices[0] + C.slices[1]), cap = 8ll * device_sm_count(dev);
    if (items == 0) return cudaSuccess;
    return launch_pdl(copy_rows_kernel, dim3((unsigned)(items < cap ? items : cap)), dim3(kThreads), 0, stream, C);
}

dim3 table_grid(int max_pages, long long rows) {
    return dim3((unsigned)((max_pages + kCols - 1) / kCols), (unsigned)(rows < 65535 ? rows : 65535));
}

}  // namespace

size_t reorder_workspace_bytes(int rows_in, int rows_out, int num_pages) {
    const size_t ch = chunks_of(num_pages);
    return align256(8 * (size_t)rows_in) + 2 * align256(4 * (size_t)rows_in) + align256(4 * (size_t)rows_out) +
           align256(ch * 128) + align256(ch * 4);
}

cudaError_t launch_reorder_pages(const lucetree_reorder_args& a, void* workspace, cudaStream_t stream) {
    ReorderLaunch R;
    R.a = a;
    R.chunks = chunks_of(a.num_pages);
    char* w = reinterpret_cast<char*>(workspace);
    auto take = [&](size_t bytes) {
        char* p = w;
        w += align256(bytes);
        return p;
    };
    R.w.kept = reinterpret_cast<uint64_t*>(take(8 * (size_t)a.rows_in));
    R.w.children = reinterpret_cast<int32_t*>(take(4 * (size_t)a.rows_in));
    R.w.first = reinterpret_cast<int32_t*>(take(4 * (size_t)a.rows_in));
    R.w.base = reinterpret_cast<int32_t*>(take(4 * (size_t)a.rows_out));
    R.w.free_bits = reinterpret_cast<uint32_t*>(take((size_t)R.chunks * 128));
    R.w.free_count = reinterpret_cast<int32_t*>(take((size_t)R.chunks * 4));
    const long long all = (long long)a.rows_in + a.rows_out;
    if (a.num_pages <= kSmallPages && all <= kSmallRows && a.max_pages_per_seq <= kSmallCols)
        return launch_pdl(reorder_small_kernel, dim3(1), dim3(kChunk), 0, stream, R);
    cudaError_t e = launch_pdl(reorder_plan_kernel, dim3(1 + R.chunks), dim3(kChunk), 0, stream, R);
    if (e != cudaSuccess) return e;
    return launch_pdl(reorder_apply_kernel, table_grid(a.max_pages_per_seq, all),
                      dim3(kThreads), 0, stream, R);
}

cudaError_t launch_trim_pages(const lucetree_trim_args& a, cudaStream_t stream) {
    if (a.ref_out != a.ref_in && a.num_pages <= kSmallPages && a.rows <= kSmallRows && a.max_pages_per_seq <= kSmallTrimCols)
        return launch_pdl(trim_small_kernel, dim3(1), dim3(kChunk), 0, stream, a);
    if (a.ref_out != a.ref_in) {
        const unsigned ctas = (unsigned)((a.num_pages + 4ll * kThreads - 1) / (4 * kThreads));
        cudaError_t e = launch_pdl(copy_counts_kernel, dim3(ctas), dim3(kThreads), 0, stream, a.ref_in, a.ref_out, a.num_pages);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(trim_kernel, table_grid(a.max_pages_per_seq, a.rows), dim3(kThreads), 0, stream, a);
}

size_t compact_workspace_bytes(int num_pages) {
    return align256(4 * (size_t)chunks_of(num_pages)) + align256(4 * (size_t)num_pages);
}

cudaError_t launch_compact_pages(const lucetree_compact_args& a, void* workspace, cudaStream_t stream) {
    CompactLaunch C;
    C.a = a;
    C.chunks = chunks_of(a.num_pages);
    C.used_count = reinterpret_cast<int32_t*>(workspace);
    C.rank = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(workspace) + align256(4 * (size_t)C.chunks));
    if (a.num_pages <= kSmallPages && (long long)a.rows * a.max_pages_per_seq <= kSmallEntries)
        return launch_pdl(compact_small_kernel, dim3(1), dim3(kChunk), 0, stream, C);
    cudaError_t e = launch_pdl(compact_count_kernel, dim3(C.chunks), dim3(kChunk), 0, stream, C);
    if (e != cudaSuccess) return e;
    e = launch_pdl(compact_rank_kernel, dim3(C.chunks), dim3(kChunk), 0, stream, C);
    if (e != cudaSuccess) return e;
    int dev = 0;
    cudaGetDevice(&dev);
    const long long n = (long long)a.rows * a.max_pages_per_seq, most = n > a.num_pages ? n : a.num_pages;
    const long long want = (most + kThreads - 1) / kThreads, cap = 8ll * device_sm_count(dev);
    return launch_pdl(compact_apply_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(kThreads), 0, stream, C);
}

cudaError_t launch_copy_pages(const lucetree_copy_pages_args& a, cudaStream_t stream) {
    CopyLaunch C = {};
    C.src = a.src;
    C.dst = a.dst;
    C.count = a.count;
    C.n = a.n;
    C.rows_from = C.rows_to = a.num_pages;
    C.from[0] = reinterpret_cast<const uint4*>(a.k_pool);
    C.from[1] = reinterpret_cast<const uint4*>(a.v_pool);
    C.to[0] = reinterpret_cast<uint4*>(a.k_pool);
    C.to[1] = reinterpret_cast<uint4*>(a.v_pool);
    C.units[0] = a.k_page_bytes / 16;
    C.units[1] = a.v_pool ? a.v_page_bytes / 16 : 0;
    C.bad = LUCETREE_DEV_BAD_PAGE;
    C.status = a.status;
    return launch_copy(C, stream);
}

cudaError_t launch_reorder_states(const lucetree_reorder_states_args& a, cudaStream_t stream) {
    CopyLaunch C = {};
    C.src = a.src;
    C.n = a.rows_out;
    C.rows_from = a.rows_in;
    C.rows_to = a.rows_out;
    C.from[0] = reinterpret_cast<const uint4*>(a.state_in);
    C.to[0] = reinterpret_cast<uint4*>(a.state_out);
    C.units[0] = a.row_bytes / 16;
    C.bad = LUCETREE_DEV_BAD_ROW;
    C.status = a.status;
    return launch_copy(C, stream);
}

}  // namespace lucetree

using namespace lucetree;

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// `b` may be `a` itself, not a part of it
bool crosses(const void* a, const void* b, long long n) { return a != b && bytes_overlap(a, n, b, n); }

lucetree_status ws_check(const void* workspace, size_t have, size_t want) {
    if (!workspace || have < want || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LUCETREE_ERR_WORKSPACE;
    return LUCETREE_OK;
}

lucetree_status done(cudaError_t e) { return e == cudaSuccess ? LUCETREE_OK : LUCETREE_ERR_CUDA; }

}  // namespace

extern "C" {

lucetree_status lucetree_reorder_pages_workspace(int rows_in, int rows_out, int num_pages, size_t* bytes) {
    if (!bytes || rows_in < 1 || rows_out < 1 || num_pages < 1) return LUCETREE_ERR_INVALID_ARG;
    if (num_pages > kMaxPages) return LUCETREE_ERR_UNSUPPORTED;
    *bytes = reorder_workspace_bytes(rows_in, rows_out, num_pages);
    return LUCETREE_OK;
}

lucetree_status lucetree_reorder_pages(const lucetree_reorder_args* a, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    if (a->rows_in < 1 || a->rows_out < 1 || a->max_pages_per_seq < 1 || a->num_pages < 1 || a->reserve < 0)
        return LUCETREE_ERR_INVALID_ARG;
    if (!a->table_in || !a->ctx_in || !a->src || !a->ref_in || !a->table_out || !a->ctx_out || !a->ref_out ||
        !a->copy_src || !a->copy_dst || !a->status)
        return LUCETREE_ERR_INVALID_ARG;
    if (a->reserve > LUCETREE_MAX_RESERVE || a->num_pages > kMaxPages || a->max_pages_per_seq > kMaxCols ||
        (long long)a->rows_in + a->rows_out > kMaxRows ||
        (long long)a->rows_out * ((a->reserve + 2ll * kPage - 2) / kPage) > 0x7fffffffll)  // ranks of new pages
        return LUCETREE_ERR_UNSUPPORTED;
    static_assert(LUCETREE_MAX_RESERVE / kPage + 1 <= kMaxTail, "a row's tail pages fit one 64-bit mask");
    const long long row = 4ll * a->max_pages_per_seq;
    if (bytes_overlap(a->table_in, row * a->rows_in, a->table_out, row * a->rows_out) ||
        bytes_overlap(a->ctx_in, 4ll * a->rows_in, a->ctx_out, 4ll * a->rows_out) ||
        crosses(a->ref_in, a->ref_out, 4ll * a->num_pages))
        return LUCETREE_ERR_INVALID_ARG;
    const long long src_bytes = 4ll * a->rows_out;
    for (const int32_t* out : {a->ctx_out, a->copy_src, a->copy_dst})
        if (bytes_overlap(a->src, src_bytes, out, src_bytes)) return LUCETREE_ERR_INVALID_ARG;
    if (bytes_overlap(a->src, src_bytes, a->table_out, row * a->rows_out) ||
        bytes_overlap(a->src, src_bytes, a->ref_out, 4ll * a->num_pages))
        return LUCETREE_ERR_INVALID_ARG;
    const lucetree_status st =
        ws_check(workspace, workspace_bytes, reorder_workspace_bytes(a->rows_in, a->rows_out, a->num_pages));
    if (st != LUCETREE_OK) return st;
    return done(launch_reorder_pages(*a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

lucetree_status lucetree_trim_pages(const lucetree_trim_args* a, void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    if (a->rows < 1 || a->max_pages_per_seq < 1 || a->num_pages < 1 || a->window < 1 || a->sinks < 0)
        return LUCETREE_ERR_INVALID_ARG;
    if (!a->table_in || !a->ctx_len || !a->ref_in || !a->table_out || !a->ref_out || !a->status)
        return LUCETREE_ERR_INVALID_ARG;
    if (a->rows > kMaxRows || a->max_pages_per_seq > kMaxCols) return LUCETREE_ERR_UNSUPPORTED;
    if (crosses(a->table_in, a->table_out, 4ll * a->max_pages_per_seq * a->rows) ||
        crosses(a->ref_in, a->ref_out, 4ll * a->num_pages))
        return LUCETREE_ERR_INVALID_ARG;
    return done(launch_trim_pages(*a, reinterpret_cast<cudaStream_t>(stream)));
}

lucetree_status lucetree_compact_pages_workspace(int num_pages, size_t* bytes) {
    if (!bytes || num_pages < 1) return LUCETREE_ERR_INVALID_ARG;
    if (num_pages > kMaxPages) return LUCETREE_ERR_UNSUPPORTED;
    *bytes = compact_workspace_bytes(num_pages);
    return LUCETREE_OK;
}

lucetree_status lucetree_compact_pages(const lucetree_compact_args* a, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    if (a->rows < 1 || a->max_pages_per_seq < 1 || a->num_pages < 1) return LUCETREE_ERR_INVALID_ARG;
    if (!a->table_in || !a->ref_in || !a->table_out || !a->ref_out || !a->copy_n || !a->live || !a->status ||
        (a->num_pages > 1 && (!a->copy_src || !a->copy_dst)))
        return LUCETREE_ERR_INVALID_ARG;
    if (a->num_pages > kMaxPages) return LUCETREE_ERR_UNSUPPORTED;
    if (crosses(a->table_in, a->table_out, 4ll * a->max_pages_per_seq * a->rows) ||
        crosses(a->ref_in, a->ref_out, 4ll * a->num_pages))
        return LUCETREE_ERR_INVALID_ARG;
    const lucetree_status st = ws_check(workspace, workspace_bytes, compact_workspace_bytes(a->num_pages));
    if (st != LUCETREE_OK) return st;
    return done(launch_compact_pages(*a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

lucetree_status lucetree_copy_pages(const lucetree_copy_pages_args* a, void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    if (a->n < 0 || a->num_pages < 1 || a->k_page_bytes < 16 || a->k_page_bytes % 16 != 0 ||
        (a->v_pool && (a->v_page_bytes < 16 || a->v_page_bytes % 16 != 0)))
        return LUCETREE_ERR_INVALID_ARG;
    if (a->n == 0) return LUCETREE_OK;
    if (!a->src || !a->dst || !a->k_pool || !a->status || !al16(a->k_pool) || !al16(a->v_pool))
        return LUCETREE_ERR_INVALID_ARG;
    return done(launch_copy_pages(*a, reinterpret_cast<cudaStream_t>(stream)));
}

lucetree_status lucetree_reorder_states(const lucetree_reorder_states_args* a, void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    if (a->rows_in < 1 || a->rows_out < 1 || a->row_bytes < 16 || a->row_bytes % 16 != 0) return LUCETREE_ERR_INVALID_ARG;
    if (!a->state_in || !a->state_out || !a->src || !a->status || !al16(a->state_in) || !al16(a->state_out))
        return LUCETREE_ERR_INVALID_ARG;
    if (bytes_overlap(a->state_in, a->row_bytes * a->rows_in, a->state_out, a->row_bytes * a->rows_out))
        return LUCETREE_ERR_INVALID_ARG;
    return done(launch_reorder_states(*a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
