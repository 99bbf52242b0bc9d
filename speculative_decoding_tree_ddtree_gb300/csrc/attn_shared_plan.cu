// attn_shared_plan.cu -- lucetree_shared_plan: what a batch's page tables have in
// common, and the cut of the attention's work over the CTAs.
//
// One launch.  The CTAs of a cluster compare table rows with their group's first row (a
// warp a row); then the first CTA lays out blocks of rows and their key lists and cuts
// the flat list of tiles evenly over the CTAs, with an allowance for each segment's
// queries and output.  Bound by its chain of dependent steps (about a dozen); it
// runs once for all layers of a decoding step.
#include "attn_shared.cuh"
#include "tc_ptx.cuh"

namespace lucetree {
namespace shr {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterMax = 8;
// Batches that are laid out in shared memory (each trip to the plan in global memory costs its latency).
constexpr int kSmallSeqs = 256, kSmallBlocks = 512;
constexpr int kPieceCost = 2;  // tiles' time that a segment's queries, first tile and output take

struct PlanLaunch {
    Dims d;
    Plan plan;
    const int32_t* table;
    int max_pages;
    int num_pages;
    const int32_t* ctx_len;
    const int32_t* group_start;
    int32_t* shared_pages;
    uint32_t* status;
};

// (Functions of their own, not inlined: the kernel runs through its code once, and the fetch of
// its instructions is much of what it takes: 47 KB of them 9.9 to 13.4 us, 26 KB 8.4 to 12.3.)

// Sum of v over the block and of the threads before this one.
__device__ __noinline__ int block_scan(int v, int* s_warp, int* before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    const int mine = lane < kWarps ? s_warp[lane] : 0;
    *before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0) + incl - v;
    return __reduce_add_sync(0xffffffffu, mine);
}

// The last of n records (a number in each that grows, the first one's at most x) whose number is at most x.
__device__ __noinline__ int last_at_most(const int* number, int stride, int n, int x) {
    int lo = 0, hi = n - 1;
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (number[mid * stride] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __noinline__ int2 div_mod(int a, int b) { return make_int2(a / b, a % b); }

__device__ __forceinline__ int pages_of(int L) { return (L + kPage - 1) / kPage; }
__device__ __forceinline__ int tiles_of(const Block& b) { return (b.vp + 1) / 2; }

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanLaunch A) {
    __shared__ int s_warp[kWarps];
    __shared__ int s_seg[kMaxCtas + 1], s_tile[kMaxCtas + 1];  // where each CTA that has tiles begins
    __shared__ int s_first[kMaxCtas];
    __shared__ Seq s_seq[kSmallSeqs + 1];
    __shared__ Group s_grp[kSmallSeqs + 1];
    __shared__ Block s_blk[kSmallBlocks + 1];
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const Dims& d = A.d;
    const Plan& P = A.plan;
    Seq* const seqs = d.B <= kSmallSeqs ? s_seq : P.seq;
    Group* const grps = d.groups <= kSmallSeqs ? s_grp : P.grp;
    Block* const blks = d.max_blocks() <= kSmallBlocks ? s_blk : P.blk;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool lead = blockIdx.x == 0;

    // ---------------------------------------------------- groups
    bool bad = false;
#pragma unroll 1
    for (int g = t; g <= d.groups; g += kThreads) {
        const int a = A.group_start[g], z = g < d.groups ? A.group_start[g + 1] : d.B;
        bad |= a < 0 || z < a || z > d.B || (g == 0 && a != 0) || (g == d.groups && a != d.B);
    }
    bad = __syncthreads_or(bad);  // then every sequence is alone
    if (bad && lead && t == 0) atomicOr(A.status, LUCETREE_DEV_BAD_ROW);

    // ---------------------------------------------------- rows against their group's first
#pragma unroll 1
    for (int b = blockIdx.x * kWarps + warp; b < d.B; b += gridDim.x * kWarps) {
        const int L = seq_len_quiet(A.ctx_len, b, A.max_pages);
        const int g = bad ? 0 : last_at_most(A.group_start, 1, d.groups, b);
        const int first = bad ? b : A.group_start[g];
        int n = L / kPage;
        if (first != b) {
            const int32_t* x = A.table + (size_t)b * A.max_pages;
            const int32_t* y = A.table + (size_t)first * A.max_pages;
            constexpr int kU = 8;
#pragma unroll 1
            for (int c0 = 0; c0 < n; c0 += 32 * kU) {
                int v[kU], w[kU], mine = 0x7fffffff;
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int c = c0 + 32 * u + lane;
                    v[u] = w[u] = 0;
                    if (c < n) {
                        v[u] = x[c];
                        w[u] = y[c];
                    }
                }
#pragma unroll
                for (int u = kU - 1; u >= 0; --u)
                    if (v[u] != w[u] || (unsigned)v[u] >= (unsigned)A.num_pages) mine = c0 + 32 * u + lane;
                mine = __reduce_min_sync(0xffffffffu, mine);
                if (mine < n) n = mine;  // (and the loop ends)
            }
        }
        if (lane == 0) {
            if (A.ctx_len[b] != L) atomicOr(A.status, LUCETREE_DEV_BAD_CTX);
            // (`used`: for now, the pages that it has in common with its group's first)
            (gridDim.x > 1 ? P.seq : seqs)[b] = Seq{g, first, L, n, 0, 0};
        }
    }
    if (gridDim.x > 1) tc::cluster_sync();
    else __syncthreads();
    if (!lead) return;
    if (gridDim.x > 1 && seqs != P.seq) {
        for (int b = t; b < d.B; b += kThreads) seqs[b] = P.seq[b];
        __syncthreads();
    }

    // ---------------------------------------------------- what the groups have in common, and use
#pragma unroll 1
    for (int g = warp; g < d.groups; g += kWarps) {
        const int a = bad ? 0 : A.group_start[g], z = bad ? 0 : A.group_start[g + 1];
        int n = 0x7fffffff;
#pragma unroll 1
        for (int b = a + lane; b < z; b += 32) n = min(n, seqs[b].used);
        n = __reduce_min_sync(0xffffffffu, n);
        if (z - a < 2) n = 0;
        if (lane == 0) {
            A.shared_pages[g] = n;
            // pages are read once for a block: fewer blocks than without
            const int blocks = div_mod((z - a) * d.N + d.NPG - 1, d.NPG).x;
            if (blocks >= (z - a) * d.NG) n = 0;
            grps[g] = Group{n, 0, n > 0 ? blocks : (z - a) * d.NG, a, z - a};
        }
    }
    __syncthreads();
    const int groups = bad ? 1 : d.groups;
    if (bad && t == 0) grps[0] = Group{0, 0, d.B * d.NG, 0, d.B};
    if (bad) __syncthreads();
    int blocks = 0;
#pragma unroll 1
    for (int g0 = 0; g0 < groups; g0 += kThreads) {
        const int g = g0 + t;
        int before;
        const int all = block_scan(g < groups ? grps[g].blocks : 0, s_warp, &before);
        if (g < groups) grps[g].block0 = blocks + before;
        blocks += all;
    }
    if (t == 0) grps[groups] = Group{0, blocks, 0, d.B, 0};
    int off = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < d.B; b0 += kThreads) {
        const int b = b0 + t;
        int n = 0, before, used = 0;
        if (b < d.B) {
            used = grps[seqs[b].group].used;
            n = pages_of(seqs[b].L) - used;
        }
        const int all = block_scan(n, s_warp, &before);
        if (b < d.B) {
            seqs[b].used = used;
            seqs[b].off = off + before;
        }
        off += all;
    }
    if (t == 0) seqs[d.B] = Seq{-1, 0, 0, 0, off, 0};
    __syncthreads();

    // ---------------------------------------------------- blocks
    int weight = 0;
#pragma unroll 1
    for (int x0 = 0; x0 < blocks; x0 += kThreads) {
        const int x = x0 + t;
        Block k = {};
        int n = 0, before;
        if (x < blocks) {
            k.group = last_at_most(&grps[0].block0, sizeof(Group) / 4, groups, x);
            const Group q = grps[k.group];
            k.used = q.used;
            if (q.used > 0) {
                k.node0 = q.seq0 * d.N + (x - q.block0) * d.NPG;
                k.nodes = min(d.NPG, (q.seq0 + q.n) * d.N - k.node0);
            } else {
                const int2 at = div_mod(x - q.block0, d.NG);
                k.node0 = (q.seq0 + at.x) * d.N + at.y * d.NPGo;
                k.nodes = min(d.NPGo, d.N - at.y * d.NPGo);
            }
            k.b0 = div_mod(k.node0, d.N).x;
            k.seqs = div_mod(k.node0 + k.nodes - 1, d.N).x - k.b0 + 1;
            k.vp = k.used + seqs[k.b0 + k.seqs].off - seqs[k.b0].off + pages_of(k.seqs * d.N);
            n = tiles_of(k) + kPieceCost;
        }
        const int all = block_scan(n, s_warp, &before);
        if (x < blocks) {
            k.pre = weight + before;
            blks[x] = k;
        }
        weight += all;
    }
    if (t == 0) {
        Block end = {};
        end.pre = weight;
        blks[blocks] = end;
    }
    __syncthreads();

    // ---------------------------------------------------- the cut
    // Groups' weights follow each other in the flat list, a group's KV heads, a head's
    // blocks; a block's first kPieceCost units are no tiles.
    const int segs = blocks * d.Hkv;
    const int2 fair = div_mod(weight * d.Hkv, d.C);
#pragma unroll 1
    for (int c = t; c <= d.C; c += kThreads) {
        // the segment and tile where CTA c begins
        const int w = fair.x * c + fair.y * c / d.C;
        int seg = segs, tile = 0;
        if (c < d.C) {
            const int head = div_mod(w, d.Hkv).x;  // (a block's weight comes once for each KV head)
            const int k = last_at_most(&blks[0].pre, sizeof(Block) / 4, blocks, head);
            const Group* q = &grps[blks[k].group];
            const int k0 = q->block0, n = q->blocks, base = blks[k0].pre;
            const int2 at = div_mod(w - base * d.Hkv, blks[k0 + n].pre - base);
            const int x = at.y + base, kk = k0 + last_at_most(&blks[k0].pre, sizeof(Block) / 4, n, x);
            seg = k0 * d.Hkv + at.x * n + (kk - k0);
            tile = x - blks[kk].pre - kPieceCost;
            if (tile <= 1) {  // no piece of a tile next to the segment's border
                tile = 0;
            } else if (tile >= tiles_of(blks[kk]) - 1) {
                tile = 0;
                ++seg;
            }
        }
        s_seg[c] = seg;
        s_tile[c] = tile;
    }
    __syncthreads();
    // CTAs without tiles go last
    int n = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < d.C; c0 += kThreads) {
        const int c = c0 + t;
        int seg = 0, tile = 0, before;
        bool has = false;
        if (c < d.C) {
            seg = s_seg[c];
            tile = s_tile[c];
            has = seg != s_seg[c + 1] || tile != s_tile[c + 1];
        }
        const int all = block_scan(has ? 1 : 0, s_warp, &before);  // (its barriers: all have read)
        if (has) {
            s_seg[n + before] = seg;
            s_tile[n + before] = tile;
        }
        n += all;
    }
    __syncthreads();
    if (t == 0) {
        s_seg[n] = segs;
        s_tile[n] = 0;
    }
    __syncthreads();

    // ---------------------------------------------------- pieces
    // Piece x = r + s is CTA r's of segment s; s_first: each CTA's first one.
#pragma unroll 1
    for (int r = t; r < d.C; r += kThreads) {
        Cta c = {0, 0, 0, 0};
        if (r < n) {
            c.first = s_first[r] = r + s_seg[r];
            c.pieces = s_seg[r + 1] - s_seg[r] + (s_tile[r + 1] > 0);
        }
        P.cta[r] = c;
        P.split[r] = Split{};
    }
    __syncthreads();
#pragma unroll 1
    for (int x = t; x < n + segs; x += kThreads) {
        const int r = last_at_most(s_first, 1, n, x), s = x - r;
        if (s > s_seg[r + 1] || (s == s_seg[r + 1] && s_tile[r + 1] == 0)) continue;  // a number that no piece has
        const Group q = grps[last_at_most(&grps[0].block0, sizeof(Group) / 4, groups, div_mod(s, d.Hkv).x)];
        const int2 at = div_mod(s - q.block0 * d.Hkv, q.blocks);
        const int k = q.block0 + at.y, tiles = tiles_of(blks[k]);
        const Block& b = blks[k];
        Piece p;
        p.b0 = b.b0;
        p.seqs = b.seqs;
        p.node0 = b.node0;
        p.nodes = b.nodes;
        p.used = b.used;
        p.vp = b.vp;
        p.ta = s == s_seg[r] ? s_tile[r] : 0;
        p.te = s == s_seg[r + 1] ? s_tile[r + 1] : tiles;
        p.g = at.x;
        p.slot = p.ta == 0 && p.te == tiles ? -1 : row0_of(d, q.seq0, q.n, at.x, b.node0) + d.block_rows() * r;
        p.own = q.used == 0;
        p.reread = (q.used > 0 ? q.blocks : d.NG) > 1;
        P.piece[x] = p;
        if (p.ta == 0 && p.te < tiles)
            P.split[r] = Split{last_at_most(s_seg, 1, n, s) - r + 1, p.slot, b.node0, b.nodes * d.G, at.x, {}};
        atomicAdd(&P.cta[r].tiles, p.te - p.ta);
    }
    // what was laid out in shared memory
    if (seqs != P.seq)
        for (int b = t; b <= d.B; b += kThreads) P.seq[b] = seqs[b];
    if (grps != P.grp)
        for (int g = t; g <= groups; g += kThreads) P.grp[g] = grps[g];
    if (blks != P.blk)
        for (int k = t; k <= blocks; k += kThreads) P.blk[k] = blks[k];
    if (t == 0) {
        Head h = {};
        h.magic = kMagic;
        h.B = d.B; h.N = d.N; h.Hq = d.Hq; h.Hkv = d.Hkv; h.D = d.D; h.groups = d.groups; h.C = d.C;
        h.max_pages = A.max_pages;
        h.num_pages = A.num_pages;
        h.blocks = blocks;
        *P.head = h;
    }
}

}  // namespace

cudaError_t launch_shared_plan(const lucetree_shared_plan_args& a, const Dims& d, cudaStream_t stream) {
    PlanLaunch A;
    A.d = d;
    plan_bytes(d, &A.plan, a.plan);
    A.table = a.page_table;
    A.max_pages = a.max_pages_per_seq;
    A.num_pages = a.num_pages;
    A.ctx_len = a.ctx_len;
    A.group_start = a.group_start;
    A.shared_pages = a.shared_pages;
    A.status = a.status;
    // a CTA for every 16 rows to compare, as far as a cluster goes
    int ctas = 1;
    while (ctas < kClusterMax && ctas * kWarps < a.B) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, plan_kernel, static_cast<const PlanLaunch>(A));
}

}  // namespace shr
}  // namespace lucetree
