// attn_shared_merge.cu -- joins the partial sums of rows whose segment several CTAs share.
//
// With weights w_k = 2^(m_k - max m), out = sum w_k O_k / sum w_k l_k.  One to eight
// warps take a row at a time: its partials' maxima and sums in one load of the
// lanes, their O rows a few at a time.  Bound by those trips to L2, so few rows are spread
// over many warps.  Rows whose segment lies in one CTA are left alone.
#include "attn_shared.cuh"
#include "attn_window.cuh"

namespace lucetree {
namespace shr {

namespace {

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kCtasPerSm = 2;

using win::store_out;

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
__global__ void __launch_bounds__(kMergeThreads, kCtasPerSm) merge_kernel(const __grid_constant__ Launch W) {
    constexpr int kV = D / 32;   // output dims of a lane
    constexpr int kU = 32 / kV;  // partials in flight
    __shared__ float s_o[kMergeWarps][D];
    __shared__ float2 s_ml[kMergeWarps];
    __shared__ int s_warp[kMergeWarps];
    __shared__ Split s_split[kMaxCtas];
    __shared__ int s_row[kMaxCtas + 1];  // rows of the split segments before each
    const lucetree_attn_args& a = W.a;
    const Dims& d = W.d;
    if (threadIdx.x == 0) pdl_trigger();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    // ---- the split segments.  This reads the plan before the wait below: the attention
    // kernel lets this one start only after its own wait, so the plan is final.
    auto split_of = [&](int c) {
        Split sp = {};
        if (c < d.C) {
            const int4* x = reinterpret_cast<const int4*>(W.plan.split + c);
            int4* y = reinterpret_cast<int4*>(&sp);
            y[0] = x[0];
            y[1] = x[1];
        }
        return sp;
    };
    Split sp = split_of(t);  // (with the head, not after it)
    if (!plan_fits(W)) {
        pdl_wait();  // (no launch completes before the one it follows)
        return;
    }
    int n = 0, total = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < d.C; c0 += kMergeThreads) {
        if (c0 > 0) sp = split_of(c0 + t);
        // how many come before it, and their rows (in the low 20 bits), by one scan
        const int mine = sp.count > 0 ? 1 << 20 | sp.rows : 0;
        int incl = mine;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, y);
            if (lane >= y) incl += x;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        int all = 0, pre = incl - mine;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            pre += w < warp ? s_warp[w] : 0;
            all += s_warp[w];
        }
        if (mine) {
            s_split[n + (pre >> 20)] = sp;
            s_row[n + (pre >> 20)] = total + (pre & 0xFFFFF);
        }
        n += all >> 20;
        total += all & 0xFFFFF;
    }
    if (t == 0) s_row[n] = total;
    __syncthreads();
    pdl_wait();  // the partial sums
    const size_t pr = partial_rows(d);
    const int rows = total, warps = (int)gridDim.x * kMergeWarps;  // (rows: at most 512 segments' 256)
    // warps to a row: as many as keep every row in flight, a power of two
    int bits = 3;
#pragma unroll 1
    while (bits > 0 && rows > warps >> bits) --bits;
    static_assert(kMergeWarps == 8, "2^3");
    const int G = 1 << bits, member = warp & (G - 1);
#pragma unroll 1
    for (int x0 = (int)blockIdx.x << (3 - bits); x0 < rows; x0 += warps >> bits) {
        const int x = x0 + (warp >> bits);
        const bool has_row = x < rows;
        int at = 0;
        if (has_row) {
            int hi = n - 1;
#pragma unroll 1
            while (at < hi) {
                const int mid = (at + hi + 1) / 2;
                if (s_row[mid] <= x) at = mid;
                else hi = mid - 1;
            }
        }
        const Split& sp = s_split[at];
        const int r = has_row ? x - s_row[at] : 0;
        const int count = has_row ? sp.count : 0;
        const size_t first = has_row ? (size_t)sp.row + r : 0;
        // partial j's O row
        auto o_at = [&](int j) { return W.ws + (first + (size_t)d.block_rows() * j) * D; };
        float m = -INFINITY, l = 0.f, o[kV] = {};
        // this warp's partials are member, member + G, ..
        const int mine = has_row ? (count - member + G - 1) >> bits : 0;
#pragma unroll 1
        for (int k0 = 0; k0 < mine; k0 += 32) {
            const int n = min(32, mine - k0);
            float mk = -INFINITY, lk = 0.f, w = 0.f;
            if (lane < n) {
                const float* s = W.ws + pr * D + first + (size_t)d.block_rows() * (member + (k0 + lane) * G);
                mk = s[0];
                lk = s[pr];
            }
#pragma unroll 1
            for (int u0 = 0; u0 < n; u0 += kU) {
                float v[kU][kV];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    if (u0 + u < n) {
                        load_row<kV>(o_at(member + (k0 + u0 + u) * G) + lane * kV, v[u]);
                    } else {
#pragma unroll
                        for (int y = 0; y < kV; ++y) v[u][y] = 0.f;
                    }
                }
                if (u0 == 0) {  // (the maxima and sums come with the first rows, not before them)
                    float top = fmaxf(m, mk);
#pragma unroll 1
                    for (int y = 16; y > 0; y >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
                    w = mk > -INFINITY ? exp2f(mk - top) : 0.f;  // (0 past n)
                    float sum = w * lk;
#pragma unroll 1
                    for (int y = 16; y > 0; y >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
                    const float keep = m > -INFINITY ? exp2f(m - top) : 0.f;
                    l = fmaf(l, keep, sum);
                    m = top;
#pragma unroll
                    for (int y = 0; y < kV; ++y) o[y] *= keep;
                }
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
#pragma unroll 1
            for (int w = 1; w < G; ++w) top = fmaxf(top, s_ml[warp + w].x);
            const float keep = m > -INFINITY ? exp2f(m - top) : 0.f;
            l *= keep;
#pragma unroll
            for (int y = 0; y < kV; ++y) o[y] *= keep;
#pragma unroll 1
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
        finite = __all_sync(0xffffffffu, finite);
        if (!finite) {  // (all of the row and its lse, as in the attention's epilogue)
            l = __int_as_float(0x7FFFFFFF);
#pragma unroll
            for (int y = 0; y < kV; ++y) o[y] = l;
        }
        const size_t row = (size_t)(sp.node0 + r / d.G) * d.Hq + sp.g * d.G + r % d.G;
        store_row<kV>(reinterpret_cast<TO*>(W.out) + row * D + lane * kV, o);
        if (!finite && lane == 0) atomicOr(a.status, LUCETREE_DEV_NONFINITE);
        if (a.lse && lane == 0) a.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
}

template <typename TO>
cudaError_t launch(const Launch& W, cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    // a CTA for every row that may have to be joined, as long as all run at once
    const long long all = (long long)W.d.B * W.d.N * W.d.Hq, most = (long long)W.d.C * W.d.block_rows();
    const long long rows = all < most ? all : most, cap = (long long)kCtasPerSm * device_sm_count(dev);
    const dim3 grid((unsigned)(rows < cap ? rows : cap)), block(kMergeThreads);
    if (W.d.D == 256) return launch_pdl(merge_kernel<TO, 256>, grid, block, 0, stream, W);
    return launch_pdl(merge_kernel<TO, 128>, grid, block, 0, stream, W);
}

}  // namespace

cudaError_t launch_shared_merge(const Launch& W, cudaStream_t stream) {
    if (W.out_dtype == LUCETREE_F32) return launch<float>(W, stream);
    return W.out_dtype == LUCETREE_BF16 ? launch<__nv_bfloat16>(W, stream) : launch<__half>(W, stream);
}

}  // namespace shr
}  // namespace lucetree
