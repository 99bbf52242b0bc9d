// attn_window_merge.cu -- joins the partial sums of segments that several CTAs of
// the windowed attention kernel share.
//
// With weights w_k = 2^(m_k - max m), out = sum w_k O_k / sum w_k l_k.  Only a
// segment with a CTA boundary inside it has partial sums, so every CTA first lists
// those segments (at most one for each boundary).  Then one to eight warps take a
// row at a time: its partials' maxima and sums in one load of the lanes, their O rows a
// few at a time.  Bound by those trips to L2, so few rows are spread over many warps
// (528 rows of 33 partials: one warp a row 28 us for the whole call, up to eight 24;
// with the list made before the wait and O loaded with its weights 22).
#include "attn_window.cuh"

namespace lucetree {
namespace win {

namespace {

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kSeqs = 1024;    // sequences whose tile offsets are held at a time
constexpr int kMaxSplit = 1024;  // CTAs of a row group (a GPU has fewer SMs)
constexpr int kCtasPerSm = 2;

struct Split {
    int b, g, c0, count;  // a segment and the CTAs [c0, c0 + count) that have its tiles
};

template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&v)[N]) {
#pragma unroll
    for (int x = 0; x < N; x += 4) {
        const float4 f = *reinterpret_cast<const float4*>(p + x);
        v[x] = f.x;
        v[x + 1] = f.y;
        v[x + 2] = f.z;
        v[x + 3] = f.w;
    }
}

template <int N, typename TO>
__device__ __forceinline__ void store_row(TO* p, const float (&v)[N]) {
    if constexpr (sizeof(TO) == 4) {
#pragma unroll
        for (int x = 0; x < N; x += 4) *reinterpret_cast<float4*>(p + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
    } else {
        alignas(16) TO t[N];
#pragma unroll
        for (int x = 0; x < N; ++x) store_out(t + x, v[x]);
        if constexpr (N == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
        else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(t);
    }
}

template <typename TO, int D>
__global__ void __launch_bounds__(kMergeThreads, kCtasPerSm) merge_kernel(WinLaunch W) {
    constexpr int kV = D / 32;  // output dims of a lane
    constexpr int kU = 32 / kV;  // partials in flight
    __shared__ int s_off[kSeqs + 1];
    __shared__ int s_warp[kMergeWarps];
    __shared__ Split s_split[kMaxSplit];
    __shared__ float s_o[kMergeWarps][D];
    __shared__ float2 s_ml[kMergeWarps];
    const lucetree_attn_args& a = W.L.a;
    const PlanDims& p = W.L.plan;
    if (threadIdx.x == 0) pdl_trigger();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    int before, tiles = p.B > kSeqs ? flat_tiles(W, 0, &before) : 0;
    // ---- segments with a CTA boundary inside, by the sequences' tile offsets.  This
    // reads the lengths before the wait below: the attention kernel lets this
    // one start only after its own wait, so its inputs are final.
    int base = 0, n_split = 0;
    for (int b0 = 0; b0 < p.B; b0 += kSeqs) {
        const int nb = min(p.B - b0, kSeqs);
        if (b0 > 0) __syncthreads();
        int run = base;
        for (int i0 = 0; i0 < nb; i0 += kMergeThreads) {
            const int i = i0 + t, n = i < nb ? seq_tiles(W, b0 + i) * p.Hkv : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            if (i0 > 0) __syncthreads();
            if (lane == 31) s_warp[warp] = incl;
            __syncthreads();
            int pre = 0, all = 0;
#pragma unroll
            for (int w = 0; w < kMergeWarps; ++w) {
                pre += w < warp ? s_warp[w] : 0;
                all += s_warp[w];
            }
            if (i < nb) s_off[i] = run + pre + incl - n;
            run += all;
        }
        if (t == 0) s_off[nb] = run;
        if (p.B <= kSeqs) tiles = run;
        const Cut cut(tiles, p.Cg);
        __syncthreads();
        for (int cb = 1; cb < cut.n; cb += kMergeThreads) {
            const int c = cb + t;
            Split sp = {0, 0, 0, 0};
            const int tile = c < cut.n ? cut.begin(c) : cut.T;  // the first of CTA c
            if (tile >= base && tile < run) {
                int lo = 0, hi = nb - 1;  // the last sequence that starts at or before it
                while (lo < hi) {
                    const int mid = (lo + hi + 1) / 2;
                    if (s_off[mid] <= tile) lo = mid;
                    else hi = mid - 1;
                }
                const int per = (s_off[lo + 1] - s_off[lo]) / p.Hkv, g = (tile - s_off[lo]) / per;
                const int first = s_off[lo] + g * per;
                // the segment's first boundary speaks for it: the CTA before has its first tile
                if (tile != first && cut.begin(c - 1) <= first)
                    sp = Split{b0 + lo, g, c - 1, cut.cta_of(first + per - 1) - c + 2};
            }
            // in the order of boundaries: every CTA makes the same list
            const unsigned who = __ballot_sync(0xffffffffu, sp.count > 0);
            if (cb > 1) __syncthreads();
            if (lane == 0) s_warp[warp] = __popc(who);
            __syncthreads();
            int at = n_split + __popc(who & ((1u << lane) - 1u));
#pragma unroll
            for (int w = 0; w < kMergeWarps; ++w) {
                at += w < warp ? s_warp[w] : 0;
                n_split += s_warp[w];
            }
            if (sp.count > 0) s_split[at] = sp;
        }
        base = run;
    }
    __syncthreads();
    pdl_wait();  // the partial sums
    const size_t sf = slot_floats(p);
    const int R = p.N * p.G;  // rows of a segment
    const long long rows = (long long)n_split * R, warps = (long long)gridDim.x * kMergeWarps;
    // warps to a row: as many as keep every row in flight
    int G = kMergeWarps;
    while (G > 1 && rows * G > warps) G >>= 1;
    const int member = warp % G;
    for (long long x0 = (long long)blockIdx.x * (kMergeWarps / G); x0 < rows; x0 += warps / G) {
        const long long x = x0 + warp / G;
        const bool has_row = x < rows;
        const Split sp = s_split[has_row ? x / R : 0];
        const int r = (int)(x % R), i = r / p.G, h = sp.g * p.G + r % p.G;
        const int rg = i / p.rg.NPG, rl = r - rg * p.rg.NPG * p.G;
        const float* ws = W.L.ws + slot_index(p, rg, sp.c0, sp.b * p.Hkv + sp.g) * sf;
        const float* parts = ws + (size_t)rl * D + lane * kV;
        float m = -INFINITY, l = 0.f, o[kV] = {};
        // this warp's partials are member, member + G, ..
        const int mine = has_row ? (sp.count - member + G - 1) / G : 0;
        for (int k0 = 0; k0 < mine; k0 += 32) {
            const int n = min(32, mine - k0), k = member + (k0 + lane) * G;
            // rows u0 .. u0 + kU - 1 of this round
            float v[kU][kV];
            auto load = [&](int u0) {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    if (u0 + u < n) {
                        load_row<kV>(parts + (size_t)(member + (k0 + u0 + u) * G) * sf, v[u]);
                    } else {
#pragma unroll
                        for (int y = 0; y < kV; ++y) v[u][y] = 0.f;
                    }
                }
            };
            load(0);  // with the maxima and sums, not after them
            float mk = -INFINITY, lk = 0.f;
            if (lane < n) {
                const float* s = ws + (size_t)k * sf + (size_t)p.rg.RG * D + rl;
                mk = s[0];
                lk = s[p.rg.RG];
            }
            float top = fmaxf(m, mk);
#pragma unroll
            for (int y = 16; y > 0; y >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
            const float w = mk > -INFINITY ? exp2f(mk - top) : 0.f;  // (0 past n)
            float sum = w * lk;
#pragma unroll
            for (int y = 16; y > 0; y >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
            const float keep = m > -INFINITY ? exp2f(m - top) : 0.f;
            l = fmaf(l, keep, sum);
            m = top;
#pragma unroll
            for (int y = 0; y < kV; ++y) o[y] *= keep;
            for (int u0 = 0; u0 < n; u0 += kU) {
                if (u0 > 0) load(u0);
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const float wu = __shfl_sync(0xffffffffu, w, u0 + u);
#pragma unroll
                    for (int y = 0; y < kV; ++y) o[y] = fmaf(wu, v[u][y], o[y]);
                }
            }
        }
        if (G > 1) {
            // the members' parts on their common shift; the first member adds them up
            __syncthreads();
            if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
            for (int y = 0; y < kV; ++y) s_o[warp][y * 32 + lane] = o[y];
            __syncthreads();
            if (member != 0) continue;
            float top = m;
            for (int w = 1; w < G; ++w) top = fmaxf(top, s_ml[warp + w].x);
            const float keep = m > -INFINITY ? exp2f(m - top) : 0.f;
            l *= keep;
#pragma unroll
            for (int y = 0; y < kV; ++y) o[y] *= keep;
            for (int w = 1; w < G; ++w) {
                const float2 ml = s_ml[warp + w];
                const float wt = ml.x > -INFINITY ? exp2f(ml.x - top) : 0.f;
                l = fmaf(wt, ml.y, l);
#pragma unroll
                for (int y = 0; y < kV; ++y) o[y] = fmaf(wt, s_o[warp + w][y * 32 + lane], o[y]);
            }
            m = top;
        }
        if (!has_row) continue;
        const float inv = l != 0.f ? 1.f / l : 0.f;  // (0: no key; NaN stays, and is flagged)
        bool finite = true;
#pragma unroll
        for (int y = 0; y < kV; ++y) {
            o[y] *= inv;
            finite = finite && isfinite(o[y]);
        }
        const size_t row = ((size_t)sp.b * p.N + i) * p.Hq + h;
        store_row<kV>(reinterpret_cast<TO*>(W.out) + row * D + lane * kV, o);
        if (!finite) atomicOr(a.status, LUCETREE_DEV_NONFINITE);
        if (a.lse && lane == 0) a.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
}

template <typename TO>
cudaError_t launch(const WinLaunch& W, cudaStream_t stream) {
    const PlanDims& p = W.L.plan;
    if (p.Cg > kMaxSplit) return cudaErrorInvalidConfiguration;
    // a CTA for every row that may have to be joined, as long as all run at once
    int dev = 0;
    cudaGetDevice(&dev);
    const long long most = p.Cg - 1 < p.S ? p.Cg - 1 : p.S, rows = most * p.N * p.G;
    const long long cap = (long long)kCtasPerSm * device_sm_count(dev);
    const dim3 grid((unsigned)(rows < cap ? rows : cap)), block(kMergeThreads);
    if (W.L.a.D == 256) return launch_pdl(merge_kernel<TO, 256>, grid, block, 0, stream, W);
    return launch_pdl(merge_kernel<TO, 128>, grid, block, 0, stream, W);
}

}  // namespace

cudaError_t launch_merge(const WinLaunch& W, cudaStream_t stream) {
    if (W.L.plan.Cg < 2) return cudaSuccess;  // one CTA for a row group: nothing is shared
    if (W.out_dtype == LUCETREE_F32) return launch<float>(W, stream);
    return W.out_dtype == LUCETREE_BF16 ? launch<__nv_bfloat16>(W, stream) : launch<__half>(W, stream);
}

}  // namespace win
}  // namespace lucetree
