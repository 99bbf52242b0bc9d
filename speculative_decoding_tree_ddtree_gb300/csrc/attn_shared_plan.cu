// attn_shared_plan.cu -- lucetree_shared_plan: what a batch's page tables have in
// common, and the cut of the attention's work over the CTAs.
//
// One launch.  The CTAs of a cluster compare table rows with their group's first row (a
// warp a row); then the first CTA lays the work out:
//   - a group uses its common pages if that saves tiles: one pass over them for its row
//     blocks instead of one for each sequence's row groups;
//   - with T tiles a CTA's fair share, the common pages of a row block are cut into
//     parts of at most X = T / m tiles, m = 1 .. kMaxParts chosen by the rounds that the
//     CTAs then need; part after part, row blocks side by side, so that CTAs
//     that read the same keys do it at the same time and the second finds them in L2;
//   - own tiles fill the CTAs up to a common level: one flat list, cut in CTA order.
// Bound by its chain of dependent steps (about a dozen); it runs once for all layers of
// a decoding step.
#include "attn_shared.cuh"

namespace lucetree {
namespace shr {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterMax = 8;
constexpr int kPieceCost = 2;  // tiles' time that a piece's queries and partial sums take

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
__device__ __forceinline__ int own_tiles(int L, int used) { return (pages_of(L) - used + 2) / 2; }

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanLaunch A) {
    __shared__ int s_warp[kWarps];
    __shared__ int s_sum[kMaxParts + 1];
    __shared__ int s_load[kMaxCtas];
    __shared__ int s_begin[kMaxCtas + 1];  // own tiles of the CTAs that have some
    __shared__ int s_cta[kMaxCtas];        // which those are
    __shared__ int s_n;
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
            P.seq[b] = Seq{g, first, L, 0, 0};
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
            const long long blocks = ((long long)(z - a) * d.N + d.NPG - 1) / d.NPG, tiles = (n + 1) / 2;
            const long long saved = (long long)(z - a) * d.own.NG * n / 2 - blocks * (tiles + kPieceCost);
            P.grp[g] = Group{saved > 0 ? n : 0, 0, 0, (int)blocks};
        }
    }
    if (t <= kMaxParts) s_sum[t] = 0;
    __syncthreads();

    // ---------------------------------------------------- tiles
    int own_all = 0;
    for (int b0 = 0; b0 < d.B; b0 += kThreads) {
        const int b = b0 + t;
        int n = 0, before;
        Seq s = {0, 0, 0, 0, 0};
        if (b < d.B) {
            s = P.seq[b];
            s.used = s.group >= 0 ? P.grp[s.group].used : 0;
            n = own_tiles(s.L, s.used) * d.Hkv * d.own.NG;
        }
        const int all = block_scan(n, s_warp, &before);
        if (b < d.B) {
            s.off = own_all + before;
            P.seq[b] = s;
        }
        own_all += all;
    }
    int mine = 0;
    for (int g = t; g < d.groups; g += kThreads) mine += (P.grp[g].used + 1) / 2 * P.grp[g].blocks * d.Hkv;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0 && mine) atomicAdd(&s_sum[0], mine);
    __syncthreads();
    const int shared_all = s_sum[0];
    const int fair = max(1, (int)(((long long)shared_all + own_all + d.C - 1) / d.C));

    // ---------------------------------------------------- parts of the shared tiles
    int x = 1;
    if (shared_all > 0) {
        int n[kMaxParts] = {};
        for (int g = t; g < d.groups; g += kThreads) {
            const Group q = P.grp[g];
            if (q.used == 0) continue;
            const int tiles = (q.used + 1) / 2;
#pragma unroll
            for (int m = 1; m <= kMaxParts; ++m) {
                const int len = (fair + m - 1) / m;
                n[m - 1] += (tiles + len - 1) / len * q.blocks * d.Hkv;
            }
        }
#pragma unroll
        for (int m = 0; m < kMaxParts; ++m) {
            const int all = __reduce_add_sync(0xffffffffu, n[m]);
            if (lane == 0 && all) atomicAdd(&s_sum[m + 1], all);
        }
        __syncthreads();
        int best = 0x7fffffff;
#pragma unroll
        for (int m = 1; m <= kMaxParts; ++m) {
            const int len = (fair + m - 1) / m, rounds = (s_sum[m] + d.C - 1) / d.C;
            // the fullest CTA, or all with the pieces' own cost
            const int cost = max(rounds * (len + kPieceCost), fair + (int)((long long)s_sum[m] * kPieceCost / d.C));
            if (cost < best) {
                best = cost;
                x = len;
            }
        }
    }
    int items = 0;
    for (int g0 = 0; g0 < d.groups; g0 += kThreads) {
        const int g = g0 + t;
        Group q = {0, 0, 0, 0};
        int n = 0, before;
        if (g < d.groups) {
            q = P.grp[g];
            q.parts = ((q.used + 1) / 2 + x - 1) / x;
            n = q.parts * q.blocks * d.Hkv;
        }
        const int all = block_scan(n, s_warp, &before);
        if (g < d.groups) {
            q.base = items + before;
            P.grp[g] = q;
        }
        items += all;
    }
    __syncthreads();

    // ---------------------------------------------------- shared pieces
    for (int c = t; c < d.C; c += kThreads) s_load[c] = 0;
    __syncthreads();
    for (int i = t; i < items; i += kThreads) {
        int lo = 0, hi = d.groups - 1;  // the last group that begins at or before it (empty ones begin where the next does)
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (P.grp[mid].base <= i) lo = mid;
            else hi = mid - 1;
        }
        const Group q = P.grp[lo];
        const int rest = i - q.base, block = rest % q.blocks, part = rest / q.blocks % q.parts, g = rest / q.blocks / q.parts;
        const int a = A.group_start[lo], z = A.group_start[lo + 1], tiles = (q.used + 1) / 2;
        const int node = block * d.NPG;
        Piece p;
        p.b = a;
        p.g = g;
        p.node0 = a * d.N + node;
        p.nodes = min(d.NPG, (z - a) * d.N - node);
        p.page0 = 0;
        p.vp = q.used;
        p.ta = (int)((long long)tiles * part / q.parts);
        p.te = (int)((long long)tiles * (part + 1) / q.parts);
        p.keys = q.used * kPage;
        p.slot = i;
        p.own = 0;
        p.reread = q.blocks > 1;
        P.item[i] = p;
        atomicAdd(&s_load[i % d.C], p.te - p.ta + kPieceCost);
    }
    __syncthreads();

    // ---------------------------------------------------- own tiles fill up to a level
    if (warp == 0) {
        const int least = fair >= 8 ? 2 : 1;  // no room for less
        auto room = [&](int level, int c) {
            const int r = c < d.C ? level - s_load[c] : 0;
            return r >= least ? r : 0;
        };
        int top = 0;
        for (int c = lane; c < d.C; c += 32) top = max(top, s_load[c]);
        top = __reduce_max_sync(0xffffffffu, top);
        int lo = 0, hi = top + least + own_all / d.C + 1;  // the lowest level with room for all is in (lo, hi]
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            long long sum = 0;
            for (int c = lane; c < d.C; c += 32) sum += room(mid, c);
            // (a lane's sum stays below 2^31: stop counting at what is needed)
            const unsigned part = (unsigned)(sum > own_all ? own_all : sum);
            unsigned long long all = part;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            if (all >= (unsigned long long)own_all) hi = mid;
            else lo = mid;
        }
        int n = 0, at = 0;
        for (int c0 = 0; c0 < d.C; c0 += 32) {
            const int c = c0 + lane, r = min(room(hi, c), own_all);
            long long incl = r;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const long long from = at + incl - r;
            const bool has = r > 0 && from < own_all;
            const unsigned who = __ballot_sync(0xffffffffu, has);
            if (has) {
                const int k = n + __popc(who & ((1u << lane) - 1u));
                s_begin[k] = (int)from;
                s_cta[k] = c;
            }
            n += __popc(who);
            const long long end = at + __shfl_sync(0xffffffffu, incl, 31);
            at = (int)(end < own_all ? end : own_all);
        }
        if (lane == 0) {
            s_begin[n] = own_all;
            s_n = n;
        }
    }
    __syncthreads();
    const int n = s_n, per_seq = d.Hkv * d.own.NG;
    // the segment that an own tile is in
    auto seg_of = [&](int tile) {
        int lo = 0, hi = d.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (P.seq[mid].off <= tile) lo = mid;
            else hi = mid - 1;
        }
        const Seq s = P.seq[lo];
        return lo * per_seq + (tile - s.off) / own_tiles(s.L, s.used);
    };
    for (int c = t; c < d.C; c += kThreads) {
        const int its = (items - c + d.C - 1) / d.C;
        P.cta[c] = Cta{0, 0, s_load[c] - max(its, 0) * kPieceCost, max(its, 0)};
    }
    __syncthreads();
    for (int k = t; k < n; k += kThreads) {
        const int from = s_begin[k], to = s_begin[k + 1], s0 = seg_of(from), s1 = seg_of(to - 1);
        Cta& c = P.cta[s_cta[k]];
        c.own0 = k + s0;
        c.owns = s1 - s0 + 1;
        c.tiles += to - from;
    }
    // a segment's pieces: one in each CTA that has some of its tiles, numbered by CTA and segment
    for (int s = t; s < d.B * per_seq; s += kThreads) {
        const int b = s / per_seq, rest = s % per_seq, g = rest / d.own.NG, rg = rest % d.own.NG;
        const Seq q = P.seq[b];
        const int tiles = own_tiles(q.L, q.used), from = q.off + rest * tiles;
        auto cta_of = [&](int tile) {
            int lo = 0, hi = n - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (s_begin[mid] <= tile) lo = mid;
                else hi = mid - 1;
            }
            return lo;
        };
        const int k0 = cta_of(from), k1 = cta_of(from + tiles - 1);
        P.seg[s] = Seg{k0 + s, k0 == k1 && q.used == 0 ? -1 : k1 - k0 + 1};
        for (int k = k0; k <= k1; ++k) {
            Piece p;
            p.b = b;
            p.g = g;
            p.node0 = b * d.N + rg * d.own.NPG;
            p.nodes = min(d.own.NPG, d.N - rg * d.own.NPG);
            p.page0 = q.used;
            p.vp = pages_of(q.L) - q.used;
            p.ta = max(s_begin[k] - from, 0);
            p.te = min(s_begin[k + 1] - from, tiles);
            p.keys = q.L - q.used * kPage;
            p.slot = k0 == k1 && q.used == 0 ? -1 : k + s;
            p.own = 1;
            p.reread = d.own.NG > 1;
            P.piece[k + s] = p;
        }
    }
    if (t == 0) {
        Head h = {};
        h.magic = kMagic;
        h.B = d.B; h.N = d.N; h.Hq = d.Hq; h.Hkv = d.Hkv; h.D = d.D; h.groups = d.groups; h.C = d.C;
        h.max_pages = A.max_pages;
        h.num_pages = A.num_pages;
        h.parts = items;
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
