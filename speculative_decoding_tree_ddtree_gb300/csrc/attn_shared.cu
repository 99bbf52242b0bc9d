// attn_shared.cu -- lucetree_shared_plan and lucetree_verify_attn_shared: tree-verify
// attention of a batch in which groups of sequences share their first pages.
// Argument checks, TMA tensor maps and the launches (attn_shared_plan.cu,
// attn_shared_tc.cuh, attn_shared_merge.cu).
#include <cuda.h>

#include "attn_shared_tc.cuh"

namespace lucetree {

lucetree_status verify_attn_check(const lucetree_attn_args* a, bool need_mask, int v_format, AttnLaunch* L);

namespace shr {

namespace {

// Sizes that the kernels take; the plan of a batch for the current device.
lucetree_status dims_of(int B, int N, int Hq, int Hkv, int D, int groups, Dims* d) {
    if (B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || groups <= 0 || groups > B) return LUCETREE_ERR_INVALID_ARG;
    if (N > LUCETREE_MAX_NODES || Hq % Hkv != 0 || (D != 128 && D != 256) || Hq / Hkv > kRows)
        return LUCETREE_ERR_UNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const int ctas = prefix_grid_ctas(dev);
    // 32-bit numbers of rows, pieces and words of the plan
    if ((long long)B * N * Hq > 0x7ff00000ll || (long long)B * Hkv * LUCETREE_MAX_NODES > 0x7ffffffll || ctas > kMaxCtas)
        return LUCETREE_ERR_UNSUPPORTED;
    *d = make_dims(B, N, Hq, Hkv, D, groups, ctas);
    return LUCETREE_OK;
}

// 32-bit numbers of pages and tiles: every segment's, as if nothing were shared.
bool tiles_fit(const Dims& d, int max_pages) {
    return (long long)d.B * d.NG * d.Hkv * (max_pages + 8ll) < 0x7fffffffll;
}

cudaError_t launch_shared(const Launch& W, cudaStream_t stream) {
    const lucetree_attn_args& a = W.a;
    const Dims& p = W.d;
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const CUtensorMapDataType dt =
        a.dtype == LUCETREE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint32_t ones[3] = {1, 1, 1};
    auto map = [&](CUtensorMap* m, int rank, const void* at, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
        return enc(m, dt, rank, const_cast<void*>(at), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t D = a.D, row = D * 2;
    Maps m;
    // pools as [num_pages * Hkv * 64 rows][D]; box = one 64-token page x 64 dims
    const cuuint64_t pool_dims[2] = {D, (cuuint64_t)a.num_pages * a.Hkv * kPage}, pool_strides[1] = {row};
    const cuuint32_t pool_box[2] = {64, (cuuint32_t)kPage};
    // V (K of a pair): the same as [D / 64][rows][64], box = 128 dims, 64 after the other 64 (K of a pair: all
    // dims; V of a pair with D = 128: half of them)
    const cuuint64_t v_dims[3] = {64, pool_dims[1], D / 64}, v_strides[2] = {row, 128};
    const cuuint32_t w_box[3] = {64, (cuuint32_t)kPage, (cuuint32_t)(D / 64)}, v_box[3] = {64, (cuuint32_t)kPage, p.pair == 2 && D == 128 ? 1u : 2u};
    // queries as [B*N nodes][Hq heads][D]; box = 64 dims x G heads x a CTA's nodes of a block of each kind
    const cuuint64_t q_dims[3] = {D, (cuuint64_t)a.Hq, (cuuint64_t)a.B * a.N}, q_strides[2] = {row, (cuuint64_t)a.Hq * row};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.half(kMeanCut)}, o_box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.half(kOwnCut)},
                     l_box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.half(kLargeCut)};
    // tree K/V as [B*N nodes][Hkv][D]; box = 64 dims of one head of 64 nodes
    const cuuint64_t t_dims[3] = {D, (cuuint64_t)a.Hkv, (cuuint64_t)a.B * a.N}, t_strides[2] = {row, (cuuint64_t)a.Hkv * row};
    const cuuint32_t t_box[3] = {64, 1, (cuuint32_t)kPage};
    const bool k_ok = p.pair == 2 ? map(&m.k, 3, a.k_pool, v_dims, v_strides, w_box)
                                  : map(&m.k, 2, a.k_pool, pool_dims, pool_strides, pool_box);
    if (!k_ok || !map(&m.v, 3, a.v_pool, v_dims, v_strides, v_box) ||
        !map(&m.q, 3, a.q, q_dims, q_strides, q_box) || !map(&m.qown, 3, a.q, q_dims, q_strides, o_box) ||
        !map(&m.qlarge, 3, a.q, q_dims, q_strides, l_box) ||
        !map(&m.kt, 3, a.k_tree, t_dims, t_strides, t_box) || !map(&m.vt, 3, a.v_tree, t_dims, t_strides, t_box))
        return cudaErrorInvalidValue;
    if (a.dtype == LUCETREE_F16) return a.D == 256 ? launch_f16_256(m, W, stream) : launch_f16_128(m, W, stream);
    if (W.out_dtype == LUCETREE_BF16)
        return a.D == 256 ? launch_bf16_256_out16(m, W, stream) : launch_bf16_128_out16(m, W, stream);
    return a.D == 256 ? launch_bf16_256(m, W, stream) : launch_bf16_128(m, W, stream);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

}  // namespace shr
}  // namespace lucetree

using namespace lucetree;

extern "C" lucetree_status lucetree_shared_plan_bytes(int B, int N, int Hq, int Hkv, int D, int groups, size_t* bytes) {
    if (!bytes) return LUCETREE_ERR_INVALID_ARG;
    shr::Dims d;
    const lucetree_status st = shr::dims_of(B, N, Hq, Hkv, D, groups, &d);
    if (st == LUCETREE_OK) *bytes = shr::plan_bytes(d, nullptr, nullptr);
    return st;
}

extern "C" lucetree_status lucetree_verify_attn_shared_workspace(int B, int N, int Hq, int Hkv, int D, int groups,
                                                                 size_t* bytes) {
    if (!bytes) return LUCETREE_ERR_INVALID_ARG;
    shr::Dims d;
    const lucetree_status st = shr::dims_of(B, N, Hq, Hkv, D, groups, &d);
    if (st == LUCETREE_OK) *bytes = shr::workspace_bytes(d);
    return st;
}

extern "C" lucetree_status lucetree_shared_plan(const lucetree_shared_plan_args* a, void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    shr::Dims d;
    const lucetree_status st = shr::dims_of(a->B, a->N, a->Hq, a->Hkv, a->D, a->groups, &d);
    if (st != LUCETREE_OK) return st;
    if (!a->page_table || !a->ctx_len || !a->group_start || !a->shared_pages || !a->plan || !a->status ||
        a->max_pages_per_seq <= 0 || a->num_pages <= 0)
        return LUCETREE_ERR_INVALID_ARG;
    if (!shr::tiles_fit(d, a->max_pages_per_seq)) return LUCETREE_ERR_UNSUPPORTED;
    const size_t bytes = shr::plan_bytes(d, nullptr, nullptr);
    if (!shr::aligned(a->plan, 256) || a->plan_bytes < bytes) return LUCETREE_ERR_WORKSPACE;
    const struct {
        const void* at;
        long long n;
    } in[] = {{a->page_table, 4ll * a->B * a->max_pages_per_seq}, {a->ctx_len, 4ll * a->B}, {a->group_start, 4ll * (a->groups + 1ll)}};
    for (const auto& x : in)
        if (bytes_overlap(a->plan, (long long)bytes, x.at, x.n) || bytes_overlap(a->shared_pages, 4ll * a->groups, x.at, x.n))
            return LUCETREE_ERR_INVALID_ARG;
    if (bytes_overlap(a->plan, (long long)bytes, a->shared_pages, 4ll * a->groups)) return LUCETREE_ERR_INVALID_ARG;
    return shr::launch_shared_plan(*a, d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LUCETREE_OK
                                                                                               : LUCETREE_ERR_CUDA;
}

extern "C" lucetree_status lucetree_verify_attn_shared(const lucetree_shared_args* w, void* workspace,
                                                       size_t workspace_bytes, void* stream) {
    if (!w) return LUCETREE_ERR_INVALID_ARG;
    if (!w->out || !w->plan) return LUCETREE_ERR_INVALID_ARG;
    if (w->out_dtype != LUCETREE_F32 && w->out_dtype != w->attn.dtype) return LUCETREE_ERR_UNSUPPORTED;
    lucetree_attn_args a = w->attn;
    a.out = reinterpret_cast<float*>(w->out);  // checked like the full attention's; written as out_dtype
    AttnLaunch full;
    lucetree_status st = verify_attn_check(&a, true, LUCETREE_V_SAME, &full);
    if (st != LUCETREE_OK) return st;
    shr::Launch W;
    st = shr::dims_of(a.B, a.N, a.Hq, a.Hkv, a.D, w->groups, &W.d);
    if (st != LUCETREE_OK) return st;
    if (!shr::tiles_fit(W.d, a.max_pages_per_seq)) return LUCETREE_ERR_UNSUPPORTED;
    const size_t plan_size = shr::plan_bytes(W.d, &W.plan, const_cast<void*>(w->plan));
    if (!shr::aligned(w->plan, 256) || w->plan_bytes < plan_size) return LUCETREE_ERR_WORKSPACE;
    // rows are written while others are still to be read
    const long long rows = (long long)a.B * a.N, q_elems = rows * a.Hq * a.D, t_bytes = rows * a.Hkv * a.D * 2;
    const long long out_bytes = q_elems * (w->out_dtype == LUCETREE_F32 ? 4 : 2);
    if (bytes_overlap(w->out, out_bytes, a.q, q_elems * 2) || bytes_overlap(w->out, out_bytes, a.k_tree, t_bytes) ||
        bytes_overlap(w->out, out_bytes, a.v_tree, t_bytes) || bytes_overlap(w->out, out_bytes, w->plan, (long long)plan_size))
        return LUCETREE_ERR_INVALID_ARG;
    const size_t need = shr::workspace_bytes(W.d);
    if (!workspace || workspace_bytes < need || !shr::aligned(workspace, 256)) return LUCETREE_ERR_WORKSPACE;
    W.a = a;
    W.ws = reinterpret_cast<float*>(workspace);
    W.scale_log2 = full.scale_log2;
    W.out_dtype = w->out_dtype;
    W.out = w->out;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (shr::launch_shared(W, s) != cudaSuccess) return LUCETREE_ERR_CUDA;
    if (shr::launch_shared_merge(W, s) != cudaSuccess) return LUCETREE_ERR_CUDA;
    return LUCETREE_OK;
}
