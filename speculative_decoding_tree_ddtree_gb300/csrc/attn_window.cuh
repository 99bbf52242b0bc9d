// attn_window.cuh -- key lists and split plan of windowed tree-verify attention.
//
// A node at depth d of the tree is at position L + d and sees the committed
// positions p with p < sinks or L + d - p < window, and its ancestors under the
// same rule.  The key list of a (sequence, KV head) segment is made of 64-key
// pages: the sink pages, the pages from the window of a depth-0 node on (deeper
// nodes see less), and last one page that holds the N tree nodes.  These
// "virtual" pages are numbered without the gap between sinks and window, and two
// consecutive ones make a key tile.  As for the whole prefix, the
// segments' tiles form one flat list that is cut evenly over the CTAs of a
// row group; a segment that one CTA has to itself needs no partial sums.
#pragma once

#include "internal.cuh"

namespace lucetree {
namespace win {

struct WinLaunch {
    AttnLaunch L;   // a.out is not used
    int window, sinks;
    int out_dtype;  // LUCETREE_F32 or a.dtype
    void* out;
    bool alone;     // CTA c of a row group has segment c to itself: no partial sums
};

struct Span {
    int lo;    // first position that the window of a depth-0 node reaches
    int sp;    // sink pages
    int skip;  // pages between the last sink page and the window's first
    int vp;    // virtual pages without the tree's, which has number vp
};

__host__ __device__ inline Span span_of(int L, int window, int sinks) {
    Span w;
    const int n = L / kPage + (L % kPage != 0);
    const int sp = sinks / kPage + (sinks % kPage != 0);
    w.lo = L - window + 1 > 0 ? L - window + 1 : 0;  // window >= 1: no overflow
    w.sp = sp < n ? sp : n;
    const int wp = w.lo >= L ? n : w.lo / kPage;
    w.skip = wp > w.sp ? wp - w.sp : 0;
    w.vp = n - w.skip;
    return w;
}

// Tiles of a segment: its pages and the tree's, two to a tile.
__host__ __device__ inline int tiles_of(const Span& w) { return (w.vp + 2) / 2; }

// The page of the sequence that virtual page v < vp stands for.
__host__ __device__ inline int page_of(const Span& w, int v) { return v < w.sp ? v : v + w.skip; }

__device__ inline int seq_tiles(const WinLaunch& W, int b) {
    return tiles_of(span_of(seq_len_quiet(W.L.a.ctx_len, b, W.L.plan.max_pages), W.window, W.sinks));
}

// Flat tiles of all segments, and of those before sequence b, by the whole warp
// (the host refuses shapes whose flat tile count reaches 2^31).
__device__ inline int flat_tiles(const WinLaunch& W, int b, int* before) {
    int all = 0, pre = 0;
    for (int i = threadIdx.x & 31; i < W.L.plan.B; i += 32) {
        const int t = seq_tiles(W, i);
        all += t;
        pre += i < b ? t : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        pre += __shfl_xor_sync(0xffffffffu, pre, o);
    }
    *before = pre * W.L.plan.Hkv;
    return all * W.L.plan.Hkv;
}

// The cut of T flat tiles over the CTAs of a row group: CTA c < n has the tiles
// [begin(c), begin(c + 1)), at least one; CTAs from n on have none.  (floor(c T / n)
// by 32-bit divisions.)
struct Cut {
    int T, n, q, r;
    __device__ Cut(int tiles, int ctas) : T(tiles), n(tiles < ctas ? tiles : ctas) {
        q = T / n;
        r = T % n;
    }
    __device__ int begin(int c) const { return c * q + c * r / n; }
    __device__ int cta_of(int tile) const { return cta_of_tile(tile, T, n); }
};

// Tiles of a segment at most, whatever its length.
inline int most_tiles(int window, int sinks, int max_pages) {
    // the window - 1 positions before a depth-0 node, wherever they begin in a page
    const int wp = window > 1 ? (window - 2) / kPage + 2 : 0, sp = sinks / kPage + (sinks % kPage != 0);
    return wp >= max_pages || sp >= max_pages - wp ? (max_pages + 2) / 2 : (wp + sp + 2) / 2;
}

// Where a CTA starts: its tile range and the segment of its first tile, found by
// the whole warp from one read of the lengths.
struct Start {
    int t0, t1;  // tile range, empty when t0 == t1
    int b, g;    // sequence and KV head of tile t0
    int off;     // flat offset of that segment's first tile
    int L;       // committed length of sequence b
};

__device__ inline Start start_of(const WinLaunch& W, int cta) {
    const PlanDims& p = W.L.plan;
    const int lane = threadIdx.x & 31;
    Start s = {0, 0, 0, 0, 0, 0};
    if (W.alone) {
        s.b = cta / p.Hkv;
        s.g = cta % p.Hkv;
        s.L = seq_len_quiet(W.L.a.ctx_len, s.b, p.max_pages);
        s.t1 = tiles_of(span_of(s.L, W.window, W.sinks));
        return s;
    }
    int before, nT = p.B > 32 ? flat_tiles(W, 0, &before) : 0, off = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int L = b0 + lane < p.B ? seq_len_quiet(W.L.a.ctx_len, b0 + lane, p.max_pages) : 0;
        const int tiles = tiles_of(span_of(L, W.window, W.sinks));
        const int mine = b0 + lane < p.B ? tiles * p.Hkv : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const int all = __shfl_sync(0xffffffffu, incl, 31);
        if (b0 == 0) {
            if (p.B <= 32) nT = all;
            const Cut cut(nT, p.Cg);
            if (cta >= cut.n) return s;
            s.t0 = cut.begin(cta);
            s.t1 = cut.begin(cta + 1);
        }
        const unsigned in = __ballot_sync(0xffffffffu, s.t0 < off + incl);
        if (in) {
            const int l = __ffs(in) - 1, per = __shfl_sync(0xffffffffu, tiles, l);
            s.b = b0 + l;
            s.off = off + __shfl_sync(0xffffffffu, incl - mine, l);
            s.L = __shfl_sync(0xffffffffu, L, l);
            s.g = (s.t0 - s.off) / per;
            s.off += s.g * per;
            return s;
        }
        off += all;
    }
    return s;
}

// A segment's share of this CTA's tiles.
struct Piece {
    int b, g, L;  // sequence, KV head, committed length
    int ta, te;   // tile range within the segment
    Span w;
    __device__ bool whole() const { return ta == 0 && te == tiles_of(w); }
};

// The CTA's tiles in order: piece and tile within the segment.  step() goes to
// the first tile, then to each next one; a length is read only when a sequence
// begins.
struct Cursor {
    int t0, t1, off, b, g, L;  // of the segment after the current piece
    Piece pc;
    int t;
    int piece_no;
    bool live;
    __device__ void start(const Start& s) {
        t0 = s.t0;
        t1 = s.t1;
        off = s.off;
        b = s.b;
        g = s.g;
        L = s.L;
        piece_no = -1;
        t = -1;
        pc.te = 0;
        live = true;
    }
    __device__ void next_piece(const WinLaunch& W) {
        live = b < W.L.plan.B && off < t1;
        if (!live) return;
        pc.b = b;
        pc.g = g;
        pc.L = L;
        pc.w = span_of(L, W.window, W.sinks);
        const int s0 = off, s1 = off + tiles_of(pc.w);
        pc.ta = (t0 > s0 ? t0 : s0) - s0;
        pc.te = (t1 < s1 ? t1 : s1) - s0;
        off = s1;
        if (++g == W.L.plan.Hkv) {
            g = 0;
            if (++b < W.L.plan.B) L = seq_len_quiet(W.L.a.ctx_len, b, W.L.plan.max_pages);
        }
        t = pc.ta;
        ++piece_no;
    }
    __device__ bool first() const { return t == pc.ta; }
    __device__ bool last() const { return t == pc.te - 1; }
    __device__ void step(const WinLaunch& W) {
        if (++t >= pc.te) next_piece(W);
    }
};

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

cudaError_t launch_merge(const WinLaunch& W, cudaStream_t stream);

}  // namespace win
}  // namespace lucetree
