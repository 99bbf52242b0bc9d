// attn_shared_plan.cu -- lucetree_shared_plan: what a batch's page tables have in
// common, and the cut of the attention's work over the CTAs.
//
// One launch.  The CTAs of a cluster compare table rows with their group's first row (a
// warp a row); then the first CTA lays out blocks of rows and their key lists and cuts
// the flat list of tiles evenly over the CTAs, with an allowance for each segment's
// queries and output.  Bound by its chain of dependent steps (about a dozen); it
// runs once for all layers of a decoding step.
#include "attn_shared.cuh"

namespace lucetree {
namespace shr {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterMax = 8;
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

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sum of v over the block and of the threads before this one.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int pre = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        pre += w < warp ? s_warp[w] : 0;
        all += s_warp[w];
    }
    *before = pre + incl - v;
    return all;
}

__device__ __forceinline__ int pages_of(int L) { return L / kPage + (L % kPage != 0); }
__device__ __forceinline__ int tiles_of(const Block& b) { return (b.vp + 1) / 2; }

// The last of n numbers that grow (at(0) <= x) which is at most x.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, long long x, F at) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (at(mid) <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanLaunch A) {
    __shared__ int s_warp[kWarps];
    __shared__ int s_seg[kMaxCtas + 1], s_tile[kMaxCtas + 1];  // where each CTA that has tiles begins
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const Dims& d = A.d;
    const Plan& P = A.plan;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool lead = blockIdx.x == 0;

    // ---------------------------------------------------- groups
    bool bad = false;
    for (int g = t; g <= d.groups; g += kThreads) {
        const int a = A.group_start[g];
        bad |= a < 0 || a > d.B || (g == 0 && a != 0) || (g == d.groups ? a != d.B : A.group_start[g + 1] < a);
    }
    bad = __syncthreads_or(bad);  // then every sequence is alone
    if (bad && lead && t == 0) atomicOr(A.status, LUCETREE_DEV_BAD_ROW);

    // ---------------------------------------------------- rows against their group's first
    for (int b = blockIdx.x * kWarps + warp; b < d.B; b += gridDim.x * kWarps) {
        int g = -1;
        for (int g0 = 0; g0 < d.groups && !bad; g0 += 32) {
            const unsigned in = __ballot_sync(0xffffffffu, g0 + lane < d.groups && A.group_start[g0 + lane] <= b);
            g += __popc(in);
            if (in != 0xffffffffu) break;
        }
        const int first = bad ? b : A.group_start[g];
        const int L = seq_len_quiet(A.ctx_len, b, A.max_pages);
        int n = L / kPage;
        if (first != b) {
            const int32_t* x = A.table + (size_t)b * A.max_pages;
            const int32_t* y = A.table + (size_t)first * A.max_pages;
            constexpr int kU = 8;
            bool done = false;
            for (int c0 = 0; c0 < n && !done; c0 += 32 * kU) {
                int v[kU], w[kU];
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
                for (int u = 0; u < kU; ++u) {
                    const unsigned off = __ballot_sync(0xffffffffu, v[u] != w[u] || v[u] < 0 || v[u] >= A.num_pages);
                    if (off && !done) {
                        n = min(n, c0 + 32 * u + __ffs(off) - 1);
                        done = true;
                    }
                }
            }
        }
        if (lane == 0) {
            if (A.ctx_len[b] != L) atomicOr(A.status, LUCETREE_DEV_BAD_CTX);
            P.lcp[b] = n;
            P.seq[b] = Seq{g, first, L, 0, 0, 0};
        }
    }
    if (gridDim.x > 1) cluster_sync();
    else __syncthreads();
    if (!lead) return;

    // ---------------------------------------------------- what the groups have in common, and use
    for (int g = warp; g < d.groups; g += kWarps) {
        const int a = bad ? 0 : A.group_start[g], z = bad ? 0 : A.group_start[g + 1];
        int n = 0x7fffffff;
        for (int b = a + lane; b < z; b += 32) n = min(n, b == a ? P.seq[a].L / kPage : P.lcp[b]);
        n = __reduce_min_sync(0xffffffffu, n);
        if (z - a < 2) n = 0;
        if (lane == 0) {
            A.shared_pages[g] = n;
            // pages are read once for a block: fewer blocks than without
            const long long blocks = ((long long)(z - a) * d.N + d.NPG - 1) / d.NPG;
            if (blocks >= (long long)(z - a) * d.NG) n = 0;
            P.grp[g] = Group{n, 0, n > 0 ? (int)blocks : (z - a) * d.NG, a, z - a};
        }
    }
    __syncthreads();
    int blocks = 0;
    for (int g0 = 0; g0 < d.groups; g0 += kThreads) {
        const int g = g0 + t;
        int before;
        const int all = block_scan(g < d.groups ? P.grp[g].blocks : 0, s_warp, &before);
        if (g < d.groups) P.grp[g].block0 = blocks + before;
        blocks += all;
    }
    if (bad) blocks = d.B * d.NG;
    int off = 0;
    for (int b0 = 0; b0 < d.B; b0 += kThreads) {
        const int b = b0 + t;
        Seq s = {0, 0, 0, 0, 0, 0};
        int n = 0, before;
        if (b < d.B) {
            s = P.seq[b];
            s.used = s.group >= 0 ? P.grp[s.group].used : 0;
            n = pages_of(s.L) - s.used + 1;
        }
        const int all = block_scan(n, s_warp, &before);
        if (b < d.B) {
            s.off = off + before;
            P.seq[b] = s;
        }
        off += all;
    }
    if (t == 0) P.seq[d.B] = Seq{-1, 0, 0, 0, off, 0};
    __syncthreads();

    // ---------------------------------------------------- blocks
    int weight = 0;
    for (int x0 = 0; x0 < blocks; x0 += kThreads) {
        const int x = x0 + t;
        Block k = {};
        int n = 0, before;
        if (x < blocks) {
            Group q = {0, 0, blocks, 0, d.B};
            k.group = -1;
            if (!bad) {
                k.group = last_at_most(d.groups, x, [&](int g) { return P.grp[g].block0; });
                q = P.grp[k.group];
            }
            k.used = q.used;
            if (q.used > 0) {
                k.node0 = q.seq0 * d.N + (x - q.block0) * d.NPG;
                k.nodes = min(d.NPG, (q.seq0 + q.n) * d.N - k.node0);
            } else {
                const int b = q.seq0 + (x - q.block0) / d.NG, i = (x - q.block0) % d.NG * d.NPGo;
                k.node0 = b * d.N + i;
                k.nodes = min(d.NPGo, d.N - i);
            }
            k.b0 = k.node0 / d.N;
            k.seqs = (k.node0 + k.nodes - 1) / d.N - k.b0 + 1;
            k.vp = k.used + P.seq[k.b0 + k.seqs].off - P.seq[k.b0].off;
            n = tiles_of(k) + kPieceCost;
        }
        const int all = block_scan(n, s_warp, &before);
        if (x < blocks) {
            k.pre = weight + before;
            P.blk[x] = k;
        }
        weight += all;
    }
    if (t == 0) {
        Block end = {};
        end.pre = weight;
        P.blk[blocks] = end;
    }
    __syncthreads();

    // ---------------------------------------------------- the cut
    // Groups' weights follow each other in the flat list, a group's KV heads, a head's
    // blocks; a block's first kPieceCost units are no tiles.
    const long long total = (long long)weight * d.Hkv;
    const int groups = bad ? 1 : d.groups;
    auto first_block = [&](int g) { return g >= groups ? blocks : bad ? 0 : P.grp[g].block0; };
    int n = 0;
    for (int c0 = 0; c0 < d.C; c0 += kThreads) {
        const int c = c0 + t;
        // the segment and tile where CTA x begins
        auto begin = [&](int x, int& seg, int& tile) {
            long long w = total / d.C * x + total % d.C * x / d.C;
            if (w >= total) {
                seg = blocks * d.Hkv;
                tile = 0;
                return;
            }
            const int g = last_at_most(groups, w, [&](int y) { return (long long)P.blk[first_block(y)].pre * d.Hkv; });
            const int k0 = first_block(g), k1 = first_block(g + 1), base = P.blk[k0].pre, per = P.blk[k1].pre - base;
            w -= (long long)base * d.Hkv;
            const int h = (int)(w / per), rest = (int)(w % per);
            const int k = k0 + last_at_most(k1 - k0, rest + base, [&](int y) { return P.blk[k0 + y].pre; });
            seg = k0 * d.Hkv + h * (k1 - k0) + (k - k0);
            const int tiles = tiles_of(P.blk[k]);
            tile = rest + base - P.blk[k].pre - kPieceCost;
            if (tile <= 1) tile = 0;  // no piece of a tile next to the segment's border
            else if (tile >= tiles - 1) {
                tile = 0;
                ++seg;
            }
        };
        int seg = 0, tile = 0, seg1 = 0, tile1 = 0, before;
        if (c < d.C) {
            begin(c, seg, tile);
            begin(c + 1, seg1, tile1);
        }
        const bool has = c < d.C && (seg != seg1 || tile != tile1);
        const int all = block_scan(has ? 1 : 0, s_warp, &before);
        if (has) {
            s_seg[n + before] = seg;
            s_tile[n + before] = tile;
        }
        n += all;
    }
    const int segs = blocks * d.Hkv;
    if (t == 0) {
        s_seg[n] = segs;
        s_tile[n] = 0;
    }
    __syncthreads();

    // ---------------------------------------------------- pieces
    // the block and KV head of a segment
    auto block_of = [&](int s, int& g) {
        const int q = last_at_most(groups, s / d.Hkv, [&](int y) { return first_block(y); });
        const int k0 = first_block(q), per = first_block(q + 1) - k0, rest = s - k0 * d.Hkv;
        g = rest / per;
        return k0 + rest % per;
    };
    for (int r = t; r < d.C; r += kThreads) {
        Cta c = {0, 0, 0, 0};
        if (r < n) {
            c.first = r + s_seg[r];
            c.pieces = s_seg[r + 1] - s_seg[r] + (s_tile[r + 1] > 0);
        }
        P.cta[r] = c;
    }
    __syncthreads();
    for (int s = t; s < segs; s += kThreads) {
        int g;
        const int k = block_of(s, g);
        const Block b = P.blk[k];
        const int tiles = tiles_of(b);
        // the CTAs that have its first and its last tile: the last ones that begin at or before them
        auto cta_of = [&](int tile) {
            int lo = 0, hi = n - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (s_seg[mid] < s || (s_seg[mid] == s && s_tile[mid] <= tile)) lo = mid;
                else hi = mid - 1;
            }
            return lo;
        };
        const int r0 = cta_of(0), r1 = cta_of(tiles - 1);
        P.seg[s] = Seg{r0, r1 - r0 + 1};
        Group q = {0, 0, blocks, 0, d.B};
        if (!bad) q = P.grp[b.group];
        const int alike = q.used > 0 ? q.blocks : d.NG, row0 = r0 != r1 ? row0_of(d, q.seq0, q.n, g, b.node0) : 0;
        for (int r = r0; r <= r1; ++r) {
            Piece p;
            p.block = k;
            p.g = g;
            p.ta = r == r0 ? 0 : s_tile[r];
            p.te = r == r1 ? tiles : s_tile[r + 1];
            p.slot = r0 == r1 ? -1 : row0 + kBlockRows * r;
            p.own = b.used == 0;
            p.reread = alike > 1;
            p.pad = 0;
            P.piece[r + s] = p;
            atomicAdd(&P.cta[r].tiles, p.te - p.ta);
        }
    }
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
