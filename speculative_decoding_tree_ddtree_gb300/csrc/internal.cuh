// internal.cuh -- shared definitions of the lucetree CUDA library (not part of the ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "lucetree.h"

namespace lucetree {

// ---------------------------------------------------------------------------
// Split plan of the committed-prefix attention.
//
// Query rows of one (sequence b, KV head g) are the N*G pairs (node i, head
// h' in the group).  They are cut into NG row groups of NPG consecutive nodes
// so a group has at most kRowsMax rows (the tensor-core tile's N extent).
// A "key segment" is one (b, g), s = b * Hkv + g, owning ceil(L_b / kTileKeys)
// key tiles.  Concatenating the segments' tiles gives a flat list of T tiles.
// The grid is NG sub-grids of Cg CTAs; CTA c of sub-grid rg takes tiles
// [floor(c*T/Cg), floor((c+1)*T/Cg)) for row group rg, so the NG CTAs that
// need the same K/V tiles stream them at the same time.  A CTA writes one
// partial (O, max, sum) per key segment its range touches, into workspace slot
// rg * (Cg + S - 1) + c + s; (c, s) is unique because both partitions are
// ordered, so Cg + S - 1 slots per row group always suffice.
// ---------------------------------------------------------------------------
constexpr int kTileKeys = 128;  // keys per tile: two 64-token pages
constexpr int kRowsMax = 144;   // rows per CTA (multiple of 16)
constexpr int kPage = LUCETREE_PAGE_SIZE;

struct RowGroups {
    int NG;   // number of row groups
    int NPG;  // nodes per group (the last group may hold fewer)
    int RG;   // rows per group = NPG * G
};

__host__ __device__ inline RowGroups make_row_groups(int N, int G) {
    RowGroups r;
    r.NG = (N * G + kRowsMax - 1) / kRowsMax;
    if (r.NG < 1) r.NG = 1;
    r.NPG = (N + r.NG - 1) / r.NG;
    while (r.NPG * G > kRowsMax && r.NPG > 1) {
        r.NG += 1;
        r.NPG = (N + r.NG - 1) / r.NG;
    }
    r.NG = (N + r.NPG - 1) / r.NPG;  // no empty trailing group
    r.RG = r.NPG * G;
    return r;
}

struct PlanDims {
    int B, N, Hq, Hkv, D, G;
    RowGroups rg;
    int S;          // key segments = B * Hkv
    int Cg;         // CTAs per row group
    int max_pages;  // page-table row length
    int window;     // sliding window in positions (0: full attention)
    int sinks;      // first positions that stay visible behind the window
};

__host__ __device__ inline PlanDims make_plan(int B, int N, int Hq, int Hkv, int D, int ctas, int max_pages) {
    PlanDims p;
    p.B = B; p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.G = Hq / Hkv;
    p.rg = make_row_groups(N, p.G);
    p.S = B * Hkv;
    p.Cg = ctas / p.rg.NG;
    if (p.Cg < 1) p.Cg = 1;
    p.max_pages = max_pages;
    p.window = p.sinks = 0;
    return p;
}

__host__ __device__ inline int grid_ctas(const PlanDims& p) { return p.Cg * p.rg.NG; }

// floats per workspace slot: O [RG][D], then max [RG], then sum [RG]; the
// stride is rounded up to 256 bytes so every slot starts 16-byte aligned
__host__ __device__ inline size_t slot_floats(const PlanDims& p) {
    return ((size_t)p.rg.RG * (p.D + 2) + 63) / 64 * 64;
}

__host__ __device__ inline size_t slot_index(const PlanDims& p, int rg, int c, int s) {
    return (size_t)rg * (p.Cg + p.S - 1) + c + s;
}

__host__ __device__ inline size_t attn_workspace_bytes(const PlanDims& p) {
    return (size_t)p.rg.NG * (p.Cg + p.S - 1) * slot_floats(p) * sizeof(float);
}

// Committed length used by the kernels: out-of-range values count as 0.
__device__ inline int seq_len(const int32_t* ctx_len, int b, int max_pages, uint32_t* status) {
    int L = ctx_len[b];
    if (L < 0 || (long long)L > (long long)max_pages * kPage) {
        if (status) atomicOr(status, LUCETREE_DEV_BAD_CTX);
        return 0;
    }
    return L;
}

__device__ inline int seq_len_quiet(const int32_t* ctx_len, int b, int max_pages) {
    int L = ctx_len[b];
    if (L < 0 || (long long)L > (long long)max_pages * kPage) return 0;
    return L;
}

__device__ inline long long tiles_of(int L) { return (L + kTileKeys - 1) / kTileKeys; }

// Total flat tiles over all key segments.
__device__ inline long long total_tiles(const PlanDims& p, const int32_t* ctx_len) {
    long long t = 0;
    for (int b = 0; b < p.B; ++b) t += tiles_of(seq_len_quiet(ctx_len, b, p.max_pages));
    return t * p.Hkv;
}

// Flat offset of key segment s's first tile.
__device__ inline long long segment_offset(const PlanDims& p, const int32_t* ctx_len, int s) {
    const int b = s / p.Hkv, g = s % p.Hkv;
    long long off = 0;
    for (int bb = 0; bb < b; ++bb) off += tiles_of(seq_len_quiet(ctx_len, bb, p.max_pages)) * p.Hkv;
    return off + (long long)g * tiles_of(seq_len_quiet(ctx_len, b, p.max_pages));
}

__device__ inline long long cta_begin(long long c, long long T, int C) { return c * T / C; }

// The CTA whose range holds flat tile t (largest c with cta_begin(c) <= t).
__device__ inline int cta_of_tile(long long t, long long T, int C) {
    return (int)(((t + 1) * (long long)C - 1) / T);
}

// ---------------------------------------------------------------------------
// Sliding window with sinks.  A node at depth d of the tree is at position
// L + d and sees the committed positions p with p < sinks or L + d - p <
// window.  A sequence's key list is then made of the pages that some node can
// see: its sink pages, and the pages from the window of a depth-0 node on
// (deeper nodes see less).  These "virtual" pages are numbered without the gap
// between them, and two consecutive ones make a key tile, so the split plan
// above works on them as it does on whole prefixes.
// ---------------------------------------------------------------------------
struct WinSpan {
    int lo;    // first position that the window of a depth-0 node reaches
    int sp;    // sink pages
    int skip;  // pages between the last sink page and the window's first
    int vp;    // virtual pages
};

__host__ __device__ inline WinSpan win_span(int L, int window, int sinks) {
    WinSpan w;
    const int n = L / kPage + (L % kPage != 0);
    const int sp = sinks / kPage + (sinks % kPage != 0);
    w.lo = L - window + 1 > 0 ? L - window + 1 : 0;  // window >= 1: no overflow
    w.sp = sp < n ? sp : n;
    const int wp = w.lo >= L ? n : w.lo / kPage;
    w.skip = wp > w.sp ? wp - w.sp : 0;
    w.vp = n - w.skip;
    return w;
}

// The page of the sequence that virtual page v stands for.
__host__ __device__ inline int win_page(const WinSpan& w, int v) { return v < w.sp ? v : v + w.skip; }

__device__ inline int win_tiles(const PlanDims& p, const int32_t* ctx_len, int b) {
    return (win_span(seq_len_quiet(ctx_len, b, p.max_pages), p.window, p.sinks).vp + 1) / 2;
}

// Flat tiles of all key segments, and of those before sequence b, by the whole
// warp (the host refuses shapes whose flat tile count reaches 2^31).
__device__ inline int win_total(const PlanDims& p, const int32_t* ctx_len, int b, int* before) {
    int all = 0, pre = 0;
    for (int i = threadIdx.x & 31; i < p.B; i += 32) {
        const int t = win_tiles(p, ctx_len, i);
        all += t;
        pre += i < b ? t : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        pre += __shfl_xor_sync(0xffffffffu, pre, o);
    }
    *before = pre * p.Hkv;
    return all * p.Hkv;
}

// Where a CTA of the prefix kernel starts: its tile range and the key segment of
// its first tile, found by the whole warp from one read of the lengths.
struct WinStart {
    int t0, t1;  // tile range, empty when t0 == t1
    int b, g;    // sequence and KV head of tile t0
    int off;     // flat offset of that segment's first tile
    int L;       // committed length of sequence b
};

__device__ inline WinStart win_start(const PlanDims& p, const int32_t* ctx_len, int cta) {
    const int lane = threadIdx.x & 31;
    WinStart s = {0, 0, 0, 0, 0, 0};
    int before, nT = p.B > 32 ? win_total(p, ctx_len, 0, &before) : 0, off = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int L = b0 + lane < p.B ? seq_len_quiet(ctx_len, b0 + lane, p.max_pages) : 0;
        const int tiles = (win_span(L, p.window, p.sinks).vp + 1) / 2, mine = tiles * p.Hkv;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const int all = __shfl_sync(0xffffffffu, incl, 31);
        if (b0 == 0) {
            if (p.B <= 32) nT = all;
            if (nT == 0) return s;
            s.t0 = (int)cta_begin(cta, nT, p.Cg);
            s.t1 = (int)cta_begin(cta + 1, nT, p.Cg);
            if (s.t0 == s.t1) return s;
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

// ---------------------------------------------------------------------------
// 16-bit element helpers
// ---------------------------------------------------------------------------
template <typename T>
__device__ inline float to_f32(T x);
template <>
__device__ inline float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ inline float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// 8 consecutive 16-bit elements (16 bytes) to fp32
template <typename T>
__device__ inline void load8_f32(const T* p, float* out);
template <>
__device__ inline void load8_f32<__half>(const __half* p, float* out) {
    uint4 u = *reinterpret_cast<const uint4*>(p);
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float2 f = __half22float2(h[k]);
        out[2 * k] = f.x;
        out[2 * k + 1] = f.y;
    }
}
template <>
__device__ inline void load8_f32<__nv_bfloat16>(const __nv_bfloat16* p, float* out) {
    uint4 u = *reinterpret_cast<const uint4*>(p);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float2 f = __bfloat1622float2(h[k]);
        out[2 * k] = f.x;
        out[2 * k + 1] = f.y;
    }
}

template <typename T>
__device__ inline void load4_f32(const T* p, float* out) {
    uint2 u = *reinterpret_cast<const uint2*>(p);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int k = 0; k < 4; ++k) out[k] = to_f32<T>(e[k]);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------
// launchers (each returns cudaGetLastError() of its launch)
// ---------------------------------------------------------------------------
struct AttnLaunch {
    lucetree_attn_args a;
    PlanDims plan;
    float* ws;
    float scale_log2;    // scale * log2(e)
    int v_format;        // LUCETREE_V_SAME (v_pool in dtype), LUCETREE_V_INT8 or LUCETREE_V_INT4 (v_pool holds codes)
    const uint8_t* v_exp;  // per-token exponents of quantised V [num_pages][Hkv][64]
    int k_format;          // LUCETREE_K_SAME, or LUCETREE_K_E4M3 (k_pool holds E4M3 codes)
    const uint8_t* k_exp;  // per-token exponents of E4M3 K [num_pages][Hkv][64]
    int out_dtype;         // windowed attention: lucetree_dtype of the output (a.out holds its address)
};

int prefix_grid_ctas(int device);  // persistent grid size of the prefix kernel
bool prefix_shape_supported(const lucetree_attn_args& a);
cudaError_t launch_attn_prefix(const AttnLaunch& L, cudaStream_t stream);
cudaError_t launch_attn_merge(const AttnLaunch& L, cudaStream_t stream);
cudaError_t launch_attn_merge_win(const AttnLaunch& L, cudaStream_t stream);
cudaError_t launch_build_anc(const int32_t* parent, int B, int N, uint64_t* anc, uint32_t* status,
                             cudaStream_t stream);
cudaError_t launch_accept(const int32_t* parent, const int32_t* draft, const int32_t* argmax, int B, int N,
                          int vocab, int32_t* acc_nodes, int32_t* acc_len, int32_t* bonus, uint32_t* status,
                          cudaStream_t stream);
cudaError_t launch_commit(const lucetree_commit_args& c, cudaStream_t stream);
size_t argmax_workspace_bytes(int rows, int vocab, int device);
cudaError_t launch_argmax(const float* logits, int rows, int vocab, long long row_stride, int32_t* out_idx,
                          void* ws, int device, cudaStream_t stream);

int device_sm_count(int device);

// ---------------------------------------------------------------------------
// Host helpers shared by the launchers.  Calls may come from several host
// threads, so every lazily filled cache is atomic or a thread-safe static.
// ---------------------------------------------------------------------------
constexpr int kMaxDevices = 128;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, resolved from the driver once per process (null
// when the driver does not provide it).
EncodeTiledFn tensor_map_encoder();

// Per-device record of the CUDA context in which a kernel's dynamic
// shared-memory limit was last raised (0 = never).
typedef std::atomic<unsigned long long> SmemLimitSeen[kMaxDevices];

// Raises `kernel`'s dynamic shared-memory limit to `bytes` in the current
// context.  The attribute belongs to the context's copy of the module, so it
// is set again whenever the calling thread's context differs from the one
// recorded for this device (another device, or a context made after a device
// reset).  `bytes` must be the largest amount any launch of the kernel uses.
cudaError_t raise_smem_limit(const void* kernel, int bytes, SmemLimitSeen& seen);

// ---------------------------------------------------------------------------
// Programmatic dependent launch.  Every library kernel is launched so that it
// may start while the previous kernel on the stream finishes; it executes
// pdl_wait() (wait until the previous grid has completed and its writes are
// visible) before its first read of global memory, and pdl_trigger() to let
// the next kernel start.  Completion stays transitive: a kernel completes only
// after its own wait returned.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace lucetree
