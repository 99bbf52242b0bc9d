// attn_shared_plan.cu -- lucetree_shared_plan: what a batch's page tables have in
// common, and the cut of the attention's work over the CTAs.
//
// One launch.  The CTAs of a cluster compare table rows with their group's first row (a
// warp a row, or fewer lanes where that leaves rows for a second turn); then the first CTA lays
// out blocks of rows and their key lists and cuts the flat list of tiles evenly over the CTAs,
// with an allowance for each segment's queries and output.  A thread finds where its CTA begins
// by searches in the running sums and goes through that CTA's pieces one after the other: no
// search and no division for each piece, and no counting of them.  Bound by its chain of
// dependent steps, 900 to 2,000 cycles each, most of that the fetch of instructions which run
// once (20 KB), and for long rows by the trips to the page table: 4.7 us for 4 sequences, 5.0
// for 8 under 16,384 tokens, 7.2 for 32 under 32,768, 8.0 for 24 groups of 8.  It runs once for
// all layers of a decoding step.
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
constexpr int kLoads = 8;      // table entries of a lane in flight
constexpr int kFewPages = 60;
constexpr int kPieceCost = 2;  // tiles' time that a segment's queries, first tile and output take

// n / d for 0 <= n < 2^31: n m >> s with m = ceil(2^s / d), s = 31 + ceil(log2 d); m d - 2^s < d,
// and n (m d - 2^s) / d 2^s < 2^(31 - s) <= 1 / d.
struct Quick {
    uint32_t m;
    int s, d;
    __device__ __forceinline__ int div(int n) const { return (int)((uint64_t)(uint32_t)n * m >> s); }
};
Quick quick(int d) {
    int l = 0;
    while ((1ll << l) < d) ++l;
    return {(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l, d};
}

struct PlanLaunch {
    Dims d;
    Plan plan;
    Quick N, NPG, cap, NG, Hkv;
    int lane_bits;  // 2^lane_bits lanes compare a row
    const int32_t* table;
    int max_pages;
    int num_pages;
    const int32_t* ctx_len;
    const int32_t* group_start;
    int32_t* shared_pages;
    uint32_t* status;
};

// (Functions of their own, not inlined: the kernel runs through its code once, and the fetch of
// its instructions is much of what it takes.)

// Sums of v over the block and of the threads before this one.
__device__ __noinline__ int2 block_scan(int2 v, int2* s_warp, int2* before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 incl = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
        if (lane >= o) {
            incl.x += x;
            incl.y += y;
        }
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    const int2 mine = lane < kWarps ? s_warp[lane] : make_int2(0, 0);
    before->x = __reduce_add_sync(0xffffffffu, lane < warp ? mine.x : 0) + incl.x - v.x;
    before->y = __reduce_add_sync(0xffffffffu, lane < warp ? mine.y : 0) + incl.y - v.y;
    return make_int2(__reduce_add_sync(0xffffffffu, mine.x), __reduce_add_sync(0xffffffffu, mine.y));
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

// Blocks of a group of n sequences that share `common` pages: by the mean group's size, or (*large) by its own where its
// rows then go through kFewPages fewer common pages, or without any in common through so many more.  By the mean,
// 32 sequences under 256 common pages beside 32 alone took 169 us instead of 46.5 with one token each (16 blocks
// instead of 2) and 492 instead of 282 with 22 (nothing shared), 24 groups of 12 and 4 under 64 pages 101 instead of 88.
// Its own size is faster below kFewPages too (under 16 pages 45 us instead of 54), but there the checks of plans in
// tests/shared_cases.py hold blocks to the mean group's size.
__device__ __forceinline__ int blocks_of(const PlanLaunch& A, int n, int common, bool* large) {
    const int nodes = n * A.d.N, mean = A.NPG.div(nodes + A.d.NPG - 1), least = A.cap.div(nodes + A.d.cap - 1);
    *large = (min(mean, n * A.d.NG) - least) * common >= kFewPages;
    return *large ? least : mean;
}
// Nodes of each of them, by its own size: as block_nodes.
__device__ __noinline__ int large_nodes(int nodes, int blocks, int N, int cap) {
    const int per = (nodes + blocks - 1) / blocks, whole = (per + N - 1) / N * N;
    if (whole <= cap) return whole;
    const int most = cap / N * N;
    return most > 0 && (nodes + most - 1) / most <= blocks ? most : per;
}

__device__ __forceinline__ int pages_of(int L) { return (L + kPage - 1) / kPage; }
__device__ __forceinline__ int tiles_of(int vp) { return (vp + 1) / 2; }

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanLaunch A) {
    __shared__ int2 s_warp[kWarps];
    // where each CTA begins: segment, tile, block, KV head, and the tiles before it
    __shared__ int s_seg[kMaxCtas + 1], s_tile[kMaxCtas + 1], s_blk_no[kMaxCtas + 1], s_head[kMaxCtas + 1], s_done[kMaxCtas + 1];
    __shared__ int s_start[kSmallSeqs + 1];
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
    const int* const starts = d.groups <= kSmallSeqs ? s_start : A.group_start;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool lead = blockIdx.x == 0;

    // ---------------------------------------------------- groups
    bool bad = false;
#pragma unroll 1
    for (int g = t; g <= d.groups; g += kThreads) {
        const int a = A.group_start[g], z = g < d.groups ? A.group_start[g + 1] : d.B;
        bad |= a < 0 || z < a || z > d.B || (g == 0 && a != 0) || (g == d.groups && a != d.B);
        if (starts == s_start) s_start[g] = a;
        if (lead) grps[g].used = 0x7fffffff;  // for now, the fewest pages that a row has in common with its group's first
    }
    bad = __syncthreads_or(bad);  // then every sequence is alone
    if (bad && lead && t == 0) atomicOr(A.status, LUCETREE_DEV_BAD_ROW);

    // ---------------------------------------------------- rows against their group's first
    const int lanes = 1 << A.lane_bits, rows = kThreads >> A.lane_bits;  // of a row; rows at a time
#pragma unroll 1
    for (int b = blockIdx.x * rows + (t >> A.lane_bits); b < d.B; b += gridDim.x * rows) {
        const int in_row = t & (lanes - 1);
        const uint32_t row_mask = (0xffffffffu >> (32 - lanes)) << (lane - in_row);
        int L = A.ctx_len[b];
        const int g = bad ? 0 : last_at_most(starts, 1, d.groups, b);
        const int first = bad ? b : starts[g];
        if (L < 0 || (long long)L > (long long)A.max_pages * kPage) {
            if (in_row == 0) atomicOr(A.status, LUCETREE_DEV_BAD_CTX);
            L = 0;
        }
        int n = L / kPage;
        if (first != b) {
            const int32_t* x = A.table + (size_t)b * A.max_pages;
            const int32_t* y = A.table + (size_t)first * A.max_pages;
            constexpr int kU = kLoads;
#pragma unroll 1
            for (int c0 = in_row; c0 - in_row < n; c0 += lanes * kU) {
                int v[kU], w[kU], mine = 0x7fffffff;
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int c = c0 + lanes * u;
                    v[u] = w[u] = 0;
                    if (c < n) {
                        v[u] = x[c];
                        w[u] = y[c];
                    }
                }
#pragma unroll
                for (int u = kU - 1; u >= 0; --u)
                    if (v[u] != w[u] || (unsigned)v[u] >= (unsigned)A.num_pages) mine = c0 + lanes * u;
                mine = __reduce_min_sync(row_mask, mine);
                if (mine < n) n = mine;  // (and the loop ends)
            }
        }
        if (in_row == 0) {
            // (`used`: for now, the pages that it has in common with its group's first)
            (gridDim.x > 1 ? P.seq : seqs)[b] = Seq{g, first, L, n, 0, 0};
            if (gridDim.x == 1) atomicMin(&grps[g].used, n);
        }
    }
    if (gridDim.x > 1) {
        __syncwarp();  // (rows of a warp end at different turns; the cluster's barrier wants whole warps)
        tc::cluster_sync();
        if (!lead) return;
#pragma unroll 1
        for (int b = t; b < d.B; b += kThreads) {
            const Seq q = P.seq[b];
            if (seqs != P.seq) seqs[b] = q;
            atomicMin(&grps[q.group].used, q.used);
        }
    }
    __syncthreads();

    // ---------------------------------------------------- what the groups have in common, and use
    const int groups = bad ? 1 : d.groups;
    struct Use {
        int a, n;    // sequences
        int common;  // pages
        int used;
        int blocks;
    };
    // (`used` of a group is read as the common pages, or as what this made of them: both give the same)
    auto use = [&](int g) {
        Use r;
        r.a = bad ? 0 : starts[g];
        r.n = (bad ? d.B : starts[g + 1]) - r.a;
        r.common = bad || r.n < 2 ? 0 : grps[g].used;
        // pages are read once for a block: fewer blocks than without
        bool large;
        const int blocks = blocks_of(A, r.n, r.common, &large);
        r.used = blocks < r.n * d.NG ? r.common : 0;
        r.blocks = r.used > 0 ? blocks : r.n * d.NG;
        return r;
    };
    int blocks = 0, off = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < max(d.groups, d.B); i0 += kThreads) {
        const int i = i0 + t;
        Use u = {};
        int used = 0;
        int2 n = {0, 0}, before;  // blocks of group i, own pages of sequence i
        if (i < groups) {
            u = use(i);
            n.x = u.blocks;
        }
        if (i < d.B) {
            used = use(seqs[i].group).used;
            n.y = pages_of(seqs[i].L) - used;
        }
        const int2 all = block_scan(n, s_warp, &before);
        if (i < d.groups) A.shared_pages[i] = u.common;
        if (i < groups) grps[i] = Group{u.used, blocks + before.x, u.blocks, u.a, u.n};
        if (i < d.B) {
            seqs[i].used = used;
            seqs[i].off = off + before.y;
        }
        blocks += all.x;
        off += all.y;
    }
    if (t == 0) {
        grps[groups] = Group{0, blocks, 0, d.B, 0};
        seqs[d.B] = Seq{-1, 0, 0, 0, off, 0};
    }
    __syncthreads();

    // ---------------------------------------------------- blocks
    int weight = 0;
#pragma unroll 1
    for (int x0 = 0; x0 < blocks; x0 += kThreads) {
        const int x = x0 + t;
        Block k = {};
        int2 n = {0, 0}, before;
        if (x < blocks) {
            k.group = last_at_most(&grps[0].block0, sizeof(Group) / 4, groups, x);
            const Group q = grps[k.group];
            k.used = q.used;
            if (q.used > 0) {
                bool large;
                blocks_of(A, q.n, q.used, &large);
                const int per = large ? large_nodes(q.n * d.N, q.blocks, d.N, d.cap) : d.NPG;
                k.node0 = q.seq0 * d.N + (x - q.block0) * per;
                k.nodes = min(per, (q.seq0 + q.n) * d.N - k.node0);
            } else {
                const int b = A.NG.div(x - q.block0), part = x - q.block0 - b * d.NG;
                k.node0 = (q.seq0 + b) * d.N + part * d.NPGo;
                k.nodes = min(d.NPGo, d.N - part * d.NPGo);
            }
            k.b0 = A.N.div(k.node0);
            k.seqs = A.N.div(k.node0 + k.nodes - 1) - k.b0 + 1;
            k.vp = k.used + seqs[k.b0 + k.seqs].off - seqs[k.b0].off + pages_of(k.seqs * d.N);
            n.x = tiles_of(k.vp) + kPieceCost;
        }
        const int2 all = block_scan(n, s_warp, &before);
        if (x < blocks) {
            k.pre = weight + before.x;
            blks[x] = k;
        }
        weight += all.x;
    }
    if (t == 0) {
        Block end = {};
        end.pre = weight;
        blks[blocks] = end;
    }
    __syncthreads();

    // ---------------------------------------------------- the cut
    // Groups' weights follow each other in the flat list, a group's KV heads, a head's
    // blocks; a block's first kPieceCost units are no tiles.  Every CTA gets one unit at least, so
    // those without a tile lie between segments, and a segment's CTAs follow each other.
    const int segs = blocks * d.Hkv, ctas = min(d.C, weight * d.Hkv);
    const int2 fair = div_mod(weight * d.Hkv, ctas);
#pragma unroll 1
    for (int c = t; c <= d.C; c += kThreads) {
        int seg = segs, tile = 0, kk = blocks, hd = 0, done = (weight - kPieceCost * blocks) * d.Hkv;
        if (c < ctas) {
            const int w = fair.x * c + min(fair.y, c);
            const int k = last_at_most(&blks[0].pre, sizeof(Block) / 4, blocks, A.Hkv.div(w));  // (a block's weight comes once for each KV head)
            const Group* q = &grps[blks[k].group];
            const int k0 = q->block0, n = q->blocks, base = blks[k0].pre, span = blks[k0 + n].pre - base;
            const int2 at = div_mod(w - base * d.Hkv, span);
            const int x = at.y + base;
            kk = k0 + last_at_most(&blks[k0].pre, sizeof(Block) / 4, n, x);
            hd = at.x;
            seg = k0 * d.Hkv + hd * n + (kk - k0);
            const int pre = blks[kk].pre, tiles = tiles_of(blks[kk].vp);
            tile = x - pre - kPieceCost;
            if (tile <= 1) tile = 0;  // no piece of a tile next to the segment's border
            else if (tile >= tiles - 1) tile = tiles;
            done = (base - kPieceCost * k0) * d.Hkv + hd * (span - kPieceCost * n) + pre - base - kPieceCost * (kk - k0) + tile;
            if (tile == tiles) {
                tile = 0;
                ++seg;
                if (++kk == k0 + n && hd + 1 < d.Hkv) {  // the next block, or the next head's first one
                    kk = k0;
                    ++hd;
                } else if (kk == k0 + n) {
                    hd = 0;
                }
            }
        }
        s_seg[c] = seg;
        s_tile[c] = tile;
        s_blk_no[c] = kk;
        s_head[c] = hd;
        s_done[c] = done;
    }
    __syncthreads();

    // ---------------------------------------------------- pieces, by the first warps
    constexpr int kCopyWarps = 3;
    constexpr int kPieceThreads = kThreads - 32 * kCopyWarps;
    if (t < kPieceThreads) {
#pragma unroll 1
        for (int r = t; r < d.C; r += kPieceThreads) {
            const int s0 = s_seg[r], s1 = s_seg[r + 1], t1 = s_tile[r + 1];
            const int n = s1 - s0 + (t1 > 0);
            *reinterpret_cast<int4*>(P.cta + r) = make_int4(d.C + s0 + 1, n, s_done[r + 1] - s_done[r], 0);
            int kk = s_blk_no[r], hd = s_head[r], ta = s_tile[r];
            int4 split[2] = {};
#pragma unroll 1
            for (int s = s0; s < s0 + n; ++s) {
                const Block b = blks[kk];
                const Group q = grps[b.group];
                const int tiles = tiles_of(b.vp), te = s == s1 ? t1 : tiles;
                const bool whole = ta == 0 && te == tiles;
                const int slot = whole ? -1 : row0_of(d, q.seq0, q.n, hd, b.node0) + d.block_rows() * r;
                int4* const p = reinterpret_cast<int4*>(P.piece + (s == s0 ? r : d.C + s));
                p[0] = make_int4(b.b0, b.seqs, b.node0, b.nodes);
                p[1] = make_int4(b.used, b.vp, ta, te);
                bool large;
                blocks_of(A, q.n, q.used, &large);
                p[2] = make_int4(hd, slot, q.used == 0, (int)((q.used > 0 ? q.blocks : d.NG) > 1) | (int)large << 1);
                if (ta == 0 && !whole) {  // (the CTA's last piece)
                    split[0] = make_int4(last_at_most(s_seg, 1, ctas, s) - r + 1, slot, b.node0, b.nodes * d.G);
                    split[1] = make_int4(hd, 0, 0, 0);
                }
                ta = 0;
                if (++kk == q.block0 + q.blocks) {
                    if (++hd < d.Hkv) kk = q.block0;
                    else hd = 0;
                }
            }
            int4* const sp = reinterpret_cast<int4*>(P.split + r);
            sp[0] = split[0];
            sp[1] = split[1];
        }
        return;
    }
    // ---------------------------------------------------- what was laid out in shared memory, by the last ones
    const int u = t - kPieceThreads;
    if (u == 0) {
        Head h = {};
        h.magic = kMagic;
        h.B = d.B; h.N = d.N; h.Hq = d.Hq; h.Hkv = d.Hkv; h.D = d.D; h.groups = d.groups; h.C = d.C;
        h.max_pages = A.max_pages;
        h.num_pages = A.num_pages;
        h.blocks = blocks;
        *P.head = h;
    }
    auto copy = [&](void* to, const void* from, int words) {
        if (to == from) return;
#pragma unroll 1
        for (int x = u; x < words; x += 32 * kCopyWarps) reinterpret_cast<int*>(to)[x] = reinterpret_cast<const int*>(from)[x];
    };
    copy(P.seq, seqs, (d.B + 1) * (int)(sizeof(Seq) / 4));
    copy(P.grp, grps, (groups + 1) * (int)(sizeof(Group) / 4));
    copy(P.blk, blks, (blocks + 1) * (int)(sizeof(Block) / 4));
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
    A.N = quick(d.N);
    A.NPG = quick(d.NPG);
    A.cap = quick(d.cap);
    A.NG = quick(d.NG);
    A.Hkv = quick(d.Hkv);
    // One CTA where it compares all rows at once, with eight lanes or more to a row that go through
    // the table's columns in four turns at most: no barrier of a cluster, whose results come through
    // memory (21 rows of 55 pages 6.2 us instead of 7.1, 24 4.9 instead of 5.7; but 32 of 530, nine
    // turns, 10.0 instead of 7.2, and 64 of 36 in two turns of rows 7.2 instead of 6.8).  Otherwise a
    // CTA for every 8 rows, as far as a cluster goes, then fewer lanes to a row.
    int ctas = 1;
    A.lane_bits = 5;
    while (A.lane_bits > 3 && (kThreads >> A.lane_bits) < a.B) --A.lane_bits;
    const int cols = kLoads << A.lane_bits;
    if (a.B > kWarps && (a.B > (kThreads >> A.lane_bits) || (a.max_pages_per_seq + cols - 1) / cols > 4)) {
        while (ctas < kClusterMax && ctas * kWarps < a.B) ctas *= 2;
        A.lane_bits = 5;
        while (A.lane_bits > 3 && ctas * (kThreads >> A.lane_bits) < a.B) --A.lane_bits;
    }
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
