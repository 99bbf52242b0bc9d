// attn_window_tc.cuh -- windowed tree-verify attention on the 5th-generation
// tensor cores.
//
// The tile step is that of the prefix kernel (attn_prefix_tc.cuh): keys on the
// MMA's M = 128, query rows on its N; S^T = K Q^T, a softmax over TMEM lanes with
// shifts that move only when an exponent exceeds 8, P^T to shared memory, O^T +=
// V^T P^T in TMEM; K and V stream through one ring of 16 KB chunks.  It differs in
//   - the key list (attn_window.cuh): sinks, window and tree of a segment, so the
//     tree block needs no code of its own and a segment that lies in one CTA is
//     finished here, without partial sums or a merge;
//   - masks: in the one or two tiles with the window's edge a key counts for rows
//     of nodes deep enough, in the tree's page for the nodes' descendants; one bit
//     per (key, row) in warps that need it, none elsewhere.  Rows of V that no row
//     sees are zeroed on chip (0 * NaN would poison the sum), and so are tree nodes
//     whose V is not finite, where the epilogue makes the rows that see them NaN;
//   - PV16 (bf16 with a bf16 output): P is rounded to bf16 and V is multiplied as
//     it lands.  Half a step of bf16 is 2^-8 of a term, as much as the
//     output's own rounding, and the terms' roundings are independent, so they
//     average out in the sum.  Otherwise P is fp16 (2^-11) and bf16 V is converted
//     in shared memory (exact from 2^-17 to below 65536);
//   - the softmax's passes (try, undo, shift) are one loop around one copy of the
//     code, and it runs once over nothing while the first tile loads: a cold
//     instruction cache costs microseconds in calls of a few tiles.
// Bounded by HBM while it streams with few rows (16 sequences decoding at window
// 4096: 2.9 us a tile on every SM, 6.8 TB/s; 56 us the call with start, last tile
// and merge); by the bytes in flight that the ring beside Q and P^T allows with many
// (32 sequences at budget 22, window 8192: 3.3 us a tile, 210 us, 5.2 TB/s); by the
// chain of lengths, page ids, first tile and epilogue in calls of a tile or two per
// CTA (one sequence at window 4096: 21 us; 8 nodes over 260 keys: 10.4 us).  Keys whose
// scores grow by 12 (log2) a tile, so that every tile moves the shifts: 446 us instead of 210.
#pragma once

#include <type_traits>

#include "attn_prefix_tc.cuh"
#include "attn_window.cuh"

namespace lucetree {
namespace win {

using namespace tc;
using prefix_tc::aborted;
using prefix_tc::bf16x2_to_f16x2;
using prefix_tc::col_sum16;
using prefix_tc::ex2;
using prefix_tc::kChunkBytes;
using prefix_tc::kConvWarps;
using prefix_tc::kMaxSlots;
using prefix_tc::kSmGroups;
using prefix_tc::kSmWarps;
using prefix_tc::kSoftmaxThreads;
using prefix_tc::kTau;
using prefix_tc::kThreads;
using prefix_tc::kTmemCols;
using prefix_tc::Layout;
using prefix_tc::pack_half2;

// Register split: the block is launched with 128 per thread; where a softmax warp
// has three column chunks, warpgroup 0, whose roles walk the windowed key list, keeps
// 80 and the softmax warpgroups take 144.
constexpr uint32_t kRegsIssue = 80, kRegsSoftmax = 144;
static_assert(128 * kRegsIssue + kSoftmaxThreads * kRegsSoftmax <= 65536, "register split exceeds the launch");

struct Misc {
    uint64_t anc[LUCETREE_MAX_NODES];  // ancestor masks of the piece's sequence
    alignas(16) float neg_m[kRowsMax];  // the shifts, negated
    alignas(16) float alpha[kRowsMax];
    alignas(16) float col_red[4][kRowsMax];
    alignas(16) uint8_t depth[kRowsMax];  // of each query row's node
    alignas(16) int out_row[kRowsMax];    // its row of the output
    alignas(16) uint8_t node[kRowsMax];   // its number
    uint64_t full[kMaxSlots];
    uint64_t empty[kMaxSlots];
    uint64_t vfull[kMaxSlots];   // V chunk n at [n % kMaxSlots]: landed ...
    uint64_t vready[kMaxSlots];  // ... made the operand
    uint64_t s_full, s_free, q_full, q_empty, p_full, pv_done, drain;
    uint32_t vbad[2];  // nodes of the piece's tree whose V is not finite (0 where the piece ends before the tree)
    uint32_t tmem_base;
    int abort_flag;
    int empty_cols;  // a query row has seen no key of its range so far
    Cursor cur;      // the softmax warps' (moved on by one thread, between barriers: it would cost each some 20 registers)
};
static_assert(sizeof(Misc) <= 5632, "misc region");

__device__ __forceinline__ void set_abort(Misc* ms, uint32_t* status) {
    if (atomicExch(&ms->abort_flag, 1) == 0) atomicOr(status, LUCETREE_DEV_TIMEOUT);
}
__device__ __forceinline__ bool aborted(Misc* ms) { return *(volatile int*)&ms->abort_flag != 0; }

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
// Maximum over the warp in one instruction.
__device__ __forceinline__ float redux_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
// Bit k: byte k of eight node depths is at most dmax (0 .. 127; depths are below 64).
__device__ __forceinline__ uint32_t depths_up_to(uint2 d, int dmax) {
    // dmax - d in every byte at once, its sign bit kept out of the neighbours by the 128 added
    const uint32_t base = (uint32_t)(128 + dmax) * 0x01010101u;
    const uint32_t lo = ((base - d.x) >> 7) & 0x01010101u, hi = ((base - d.y) >> 7) & 0x01010101u;
    // bytes 0, 1, 2, 3 -> bits 0, 1, 2, 3
    return ((lo * 0x01020408u) >> 24 & 0xFu) | ((hi * 0x01020408u) >> 20 & 0xF0u);
}
// Bit k: the node whose number is byte k of `nodes` is in `set`.
__device__ __forceinline__ uint32_t nodes_in(uint2 nodes, uint64_t set) {
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        bits |= ((uint32_t)(set >> (((k < 4 ? nodes.x : nodes.y) >> (8 * (k & 3))) & 0xFFu)) & 1u) << k;
    return bits;
}

// Two fp32 in one 64-bit register pair, and one instruction for two fused multiply-adds.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t low_bits(int n) { return ~0ull >> (64 - n); }  // 1 <= n <= 64

// Whether one of eight values of V is not finite as the operand of PV (0 x is 0 or, for
// what is not finite, NaN; where bf16 becomes fp16, 65536 is not: 2^16 2^112 overflows).
template <bool BF16, bool CONVERT>
__device__ __forceinline__ bool not_finite(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (BF16) {
            __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[k]), y = *reinterpret_cast<__nv_bfloat162*>(&sum);
            if constexpr (CONVERT) x = __hmul2(x, __bfloat162bfloat162(__ushort_as_bfloat16(0x7780)));  // 2^112
            y = __hfma2(x, __bfloat162bfloat162(__ushort_as_bfloat16(0)), y);
            sum = *reinterpret_cast<uint32_t*>(&y);
        } else {
            const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&w[k]), __half2half2(__ushort_as_half(0)),
                                      *reinterpret_cast<__half2*>(&sum));
            sum = *reinterpret_cast<const uint32_t*>(&y);
        }
    }
    return (sum & 0x7FFF7FFFu) != 0;
}

// An operand's 64-row halves: pool rows, or (tree: 0 or 1) the sequence's tree nodes.
struct Operand {
    int row0, row1;
    int tree;   // -1: neither
    int node0;  // b * N
    int g;
};

template <int D, bool BF16, int RGP, bool PV16>
__global__ void __launch_bounds__(kThreads, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kt,
                     const __grid_constant__ CUtensorMap tm_vt, const WinLaunch W) {
    using Lay = Layout<D, RGP>;
    static_assert(BF16 || !PV16, "fp16 inputs run PV on fp16 anyway");
    constexpr bool kConvert = BF16 && !PV16;                 // V to fp16 on chip
    constexpr int kChunks = D / 64;                          // ring chunks per operand
    constexpr int kNch = Lay::kNch;
    constexpr int kNa = (kNch + kSmGroups - 1) / kSmGroups;  // column chunks per softmax warp (at most)
    constexpr int kNS = Lay::kNS;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem + Lay::kQOff;
    uint8_t* sP = smem + Lay::kPOff;
    uint8_t* sSlots = smem + Lay::kSlotOff;
    Misc* ms = reinterpret_cast<Misc*>(smem + Lay::kMiscOff);

    const lucetree_attn_args& a = W.L.a;
    const PlanDims& p = W.L.plan;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rg = blockIdx.x / p.Cg, cta = blockIdx.x % p.Cg;
    const int i0 = rg * p.rg.NPG;
    const int R_seg = (min(p.N, i0 + p.rg.NPG) - i0) * p.G;
    const int RG = p.rg.RG;

    // ---------------------------------------------------------------- set-up
    // (reads no global memory: it overlaps the previous kernel's tail)
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNS; ++i) {
            mbar_init(&ms->full[i], 1);
            mbar_init(&ms->empty[i], 1);
        }
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&ms->vfull[i], 1);
            mbar_init(&ms->vready[i], kConvWarps);
        }
        mbar_init(&ms->s_full, 1);
        mbar_init(&ms->s_free, kSmWarps);
        mbar_init(&ms->q_full, 1);
        mbar_init(&ms->q_empty, 1);
        mbar_init(&ms->p_full, kSmWarps);
        mbar_init(&ms->pv_done, 1);
        mbar_init(&ms->drain, 1);
        ms->abort_flag = 0;
        mbar_fence_init();
    }
    if (warp >= 4) {
        // rows RG..RGP-1 of Q are padding: zero them once (TMA never writes them)
        const int st = threadIdx.x - 128;
        for (int idx = st; idx < kChunks * RGP * 8; idx += kSoftmaxThreads) {
            const int c = idx / (RGP * 8), r = (idx / 8) % RGP, u = idx % 8;
            if (r >= RG) *reinterpret_cast<uint4*>(sQ + c * RGP * 128 + r * 128 + u * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(&ms->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_kt);
        prefetch_tensormap(&tm_vt);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms->tmem_base;

    // inputs may come from the previous kernel on the stream
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const Start start = start_of(W, cta);
    if (start.t0 >= start.t1) {  // uniform across the CTA: nothing to do but give TMEM back
        if (warp == 1) tmem_dealloc(tmem, kTmemCols);
        return;
    }
    const uint32_t n_tiles = (uint32_t)(start.t1 - start.t0);

    if (warp < 4) {
    if constexpr (kNa >= 3) regs_dec<kRegsIssue>();
    if (warp == 0) {
        // ============================================================ TMA producer
        const int oob_row = a.num_pages * p.Hkv * kPage;  // first row past the pool: zero fill
        const uint64_t pol_stream = policy_evict_first();  // K/V are read once: do not keep them in L2
        const uint32_t tree_bytes = (uint32_t)p.N * 128u;  // one 64-dim box of the tree's nodes
        uint32_t chunk = 0, vchunk = 0;
        int q_loads = 0;
        bool ok = true;
        auto issue = [&](bool is_v, const Operand& o) -> bool {
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                const int slot = chunk % kNS;
                const bool w = mbar_wait(&ms->empty[slot], ((chunk / kNS) & 1) ^ 1);
                if (!__all_sync(0xffffffffu, w)) return false;  // lanes agree on a timeout
                if (lane == 0) {
                    uint8_t* dst = sSlots + slot * kChunkBytes;
                    uint64_t* bar = &ms->full[slot];
                    if (is_v) {
                        mbar_arrive(bar);  // this fill's phase of full[slot]; the data signal is vfull
                        bar = &ms->vfull[vchunk % kMaxSlots];
                        // [64 keys of half c & 1][dims 128 * (c >> 1) .. +127]
                        const int x = 128 * (c >> 1);
                        if ((c & 1) == o.tree) {
                            mbar_arrive_expect_tx(bar, 2 * tree_bytes);
                            tma_load_3d(dst, &tm_vt, x, o.g, o.node0, bar);
                            tma_load_3d(dst + 8192, &tm_vt, x + 64, o.g, o.node0, bar);
                        } else {
                            const int row = (c & 1) ? o.row1 : o.row0;
                            mbar_arrive_expect_tx(bar, kChunkBytes);
                            tma_load_2d_hint(dst, &tm_v, x, row, bar, pol_stream);
                            tma_load_2d_hint(dst + 8192, &tm_v, x + 64, row, bar, pol_stream);
                        }
                    } else {
                        // [128 keys: half 0 then half 1][dims 64 * c .. +63]
                        mbar_arrive_expect_tx(bar, o.tree >= 0 ? 8192 + tree_bytes : kChunkBytes);
                        if (o.tree == 0) tma_load_3d(dst, &tm_kt, 64 * c, o.g, o.node0, bar);
                        else tma_load_2d_hint(dst, &tm_k, 64 * c, o.row0, bar, pol_stream);
                        if (o.tree == 1) tma_load_3d(dst + 8192, &tm_kt, 64 * c, o.g, o.node0, bar);
                        else tma_load_2d_hint(dst + 8192, &tm_k, 64 * c, o.row1, bar, pol_stream);
                    }
                }
                __syncwarp();
                ++chunk;
                vchunk += is_v ? 1u : 0u;
            }
            return true;
        };
        Cursor cur;
        cur.start(start);
        const int32_t* pt = a.page_table;
        // page ids of the current piece, 16 tiles (32 pages) per warp-wide load, one batch ahead
        auto load_batch = [&](int tb) {
            const int v = 2 * tb + lane;
            int pid = -1;
            if (v < cur.pc.w.vp && v < 2 * cur.pc.te) {
                const int x = pt[page_of(cur.pc.w, v)];
                if (x >= 0 && x < a.num_pages) pid = x;
                else atomicOr(a.status, LUCETREE_DEV_BAD_PAGE);
            }
            return pid;
        };
        int pid_cur = -1, pid_next = -1;
        Operand v_op = {0, 0, -1, 0, 0};  // of the tile whose V is still to be loaded
        bool have_v = false;
        // K(t), then V(t-1); after the last tile its V alone
        while (ok && cur.live) {
            cur.step(W);
            Operand op = v_op;
            const bool have_k = cur.live;
            if (have_k) {
                const int rel = cur.t - cur.pc.ta;
                if (rel == 0) {
                    // a new segment: its queries replace the previous ones once their last QK is done
                    if (cur.piece_no > 0) {
                        const bool w = mbar_wait(&ms->q_empty, (cur.piece_no - 1) & 1);
                        if (!(ok = __all_sync(0xffffffffu, w))) break;
                    }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&ms->q_full, kChunks * RG * 128);
#pragma unroll 1
                        for (int c = 0; c < kChunks; ++c)
                            tma_load_3d(sQ + c * RGP * 128, &tm_q, 64 * c, cur.pc.g * p.G, cur.pc.b * p.N + i0, &ms->q_full);
                    }
                    __syncwarp();
                    ++q_loads;
                    pt = a.page_table + (size_t)cur.pc.b * p.max_pages;
                    pid_cur = load_batch(cur.pc.ta);
                } else if ((rel & 15) == 0) {
                    pid_cur = pid_next;
                }
                if ((rel & 15) == 0) pid_next = load_batch(cur.t + 16);
                int row[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int pid = __shfl_sync(0xffffffffu, pid_cur, 2 * (rel & 15) + h);
                    row[h] = pid >= 0 ? (pid * p.Hkv + cur.pc.g) * kPage : oob_row;
                }
                const int tree = cur.pc.w.vp - 2 * cur.t;
                op = {row[0], row[1], tree == 0 || tree == 1 ? tree : -1, cur.pc.b * p.N, cur.pc.g};
            }
#pragma unroll 1
            for (int is_v = have_k ? 0 : 1; is_v < (have_v ? 2 : 1) && ok; ++is_v) ok = issue(is_v != 0, is_v ? v_op : op);
            v_op = op;
            have_v = have_k;
        }
        if (!ok || aborted(ms)) {
            set_abort(ms, a.status);
            // wait (bounded) for this CTA's own copies still in flight
            if (lane == 0) {
                const uint32_t first = chunk > (uint32_t)kNS ? chunk - kNS : 0u;
                for (uint32_t c = first; c < chunk; ++c) mbar_wait(&ms->full[c % kNS], (c / kNS) & 1, 200000000ll);
                const uint32_t vfirst = vchunk > (uint32_t)kNS ? vchunk - kNS : 0u;
                for (uint32_t c = vfirst; c < vchunk; ++c)
                    mbar_wait(&ms->vfull[c % kMaxSlots], (c / kMaxSlots) & 1, 200000000ll);
                if (q_loads > 0) mbar_wait(&ms->q_full, (q_loads - 1) & 1, 200000000ll);
            }
        }
    } else if (warp == 1) {
        // ============================================================ MMA issuer
        if (lane == 0) {
            const uint32_t id_qk = idesc_f16(128, RGP, BF16 ? 1u : 0u, 0, 0);
            const uint32_t id_pv = idesc_f16(128, RGP, PV16 ? 1u : 0u, 1, 1);
            constexpr uint64_t hi_k = desc_hi(16, 1024, kLayoutSwizzle128);
            constexpr uint64_t hi_v = desc_hi(8192, 1024, kLayoutSwizzle128);  // 2nd 64-dim box at +8 KB
            constexpr uint64_t hi_p = desc_hi(128, 2048, kLayoutInterleave);
            const uint32_t aQ = smem_u32(sQ), aP = smem_u32(sP), aS = smem_u32(sSlots);
            uint32_t chunk = 0, jq = 0, j = 0;
            uint32_t first_bits = 0;  // bit k: the k-th last QK issued opened a piece
            bool ok = true;
            Cursor qk;
            qk.start(start);
            // QK(0); then QK(j+1) and PV(j) for every tile j
            while (ok && j < n_tiles) {
                if (qk.live) qk.step(W);
                if (qk.live) {
                    // S^T(jq) = K(jq) . Q^T; S^T is free once the softmax has read tile jq-1
                    if (jq > 0 && !(ok = mbar_wait(&ms->s_free, (jq - 1) & 1))) break;
                    if (qk.first() && !(ok = mbar_wait(&ms->q_full, qk.piece_no & 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kChunks && ok; ++c) {
                        const int slot = chunk % kNS;
                        if (!(ok = mbar_wait(&ms->full[slot], (chunk / kNS) & 1))) break;
                        tc_fence_after();
#pragma unroll
                        for (int sub = 0; sub < 4; ++sub) {
                            const uint64_t ad = make_desc(hi_k, aS + slot * kChunkBytes + sub * 32);
                            const uint64_t bd = make_desc(hi_k, aQ + c * RGP * 128 + sub * 32);
                            mma_f16_ss(tmem, ad, bd, id_qk, (c | sub) != 0);
                        }
                        mma_commit(&ms->empty[slot]);
                        ++chunk;
                    }
                    if (!ok) break;
                    mma_commit(&ms->s_full);
                    if (qk.last()) mma_commit(&ms->q_empty);
                    first_bits = (first_bits << 1) | (qk.first() ? 1u : 0u);
                    if (jq++ == 0) continue;
                }
                if (aborted(ms)) {
                    ok = false;
                    break;
                }
                // O^T += V^T . P^T once the softmax has written P^T(j)
                if (!(ok = mbar_wait(&ms->p_full, j & 1))) break;
                tc_fence_after();
                const bool first = (first_bits >> (jq - 1 - j)) & 1u;
                // chunk c: output dims 128 (c >> 1) .., keys 64 (c & 1) ..
#pragma unroll 1
                for (int c = 0; c < kChunks && ok; ++c) {
                    const uint32_t dO = tmem + (c >> 1 ? Lay::kColO1 : Lay::kColO0);
                    const int slot = chunk % kNS;
                    const uint32_t vn = j * kChunks + c;
                    if (!(ok = mbar_wait(&ms->vready[vn % kMaxSlots], (vn / kMaxSlots) & 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ad = make_desc(hi_v, aS + slot * kChunkBytes + ks * 2048);
                        const uint64_t bd = make_desc(hi_p, aP + (4 * (c & 1) + ks) * 256);
                        mma_f16_ss(dO, ad, bd, id_pv, !(first && (c & 1) == 0 && ks == 0));
                    }
                    mma_commit(&ms->empty[slot]);
                    ++chunk;
                }
                if (!ok) break;
                mma_commit(&ms->pv_done);
                ++j;
            }
            if (!ok || aborted(ms)) {
                set_abort(ms, a.status);
                mma_commit(&ms->drain);  // every MMA issued so far has finished before TMEM is freed
                mbar_wait(&ms->drain, 0, 200000000ll);
            }
        }
        __syncwarp();
    } else {
        // ============================================================ V operand (warps 2, 3)
        // Each V chunk, once landed: bf16 -> fp16 in place where PV runs on fp16,
        // and zeros in the rows of keys that no row sees (past L, past the tree's
        // nodes, between sinks and window: arbitrary data); then vready.  Thread
        // ct owns 16-byte units ct + 64 i of a chunk; unit u holds 8 dims of key
        // (u % 512) / 8 of the chunk's half (each 8 KB box is [64 keys][128 B]; the
        // swizzle permutes units only within a key's row).
        const int ct = threadIdx.x - 64;  // 0 .. 63
        Cursor cur;
        cur.start(start);
        uint32_t j = 0;
        bool ok = true;
        while (ok) {
            cur.step(W);
            if (!cur.live) break;
            // ring position of V(j)'s first chunk: the K operands before it
            // (K(0) .. K(j+1), or .. K(j) for the last tile) and V(0) .. V(j-1)
            const uint32_t vbase = ((j + 1 < n_tiles ? j + 2 : j + 1) + j) * kChunks;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                const uint32_t vn = j * kChunks + c;
                const bool landed = mbar_wait(&ms->vfull[vn % kMaxSlots], (vn / kMaxSlots) & 1);
                if (!__all_sync(0xffffffffu, landed) || aborted(ms)) {
                    ok = false;
                    break;
                }
                uint4* base = reinterpret_cast<uint4*>(sSlots + ((vbase + c) % kNS) * kChunkBytes);
                // keys [0, nv) exist; of those the first ns (sinks) and those from nl on (window) count
                const int v = 2 * cur.t + (c & 1);
                int nv = 0, ns = kPage, nl = 0;
                if (v < cur.pc.w.vp) {
                    const int p0 = page_of(cur.pc.w, v) * kPage;
                    nv = cur.pc.L - p0;
                    ns = W.sinks - p0;
                    nl = cur.pc.w.lo - p0;
                } else if (v == cur.pc.w.vp) {
                    nv = p.N;
                }
                const bool whole = nv >= kPage && (ns >= kPage || nl <= 0);
                constexpr int kUnits = kChunkBytes / 16 / (32 * kConvWarps);  // 16 per thread
                constexpr int kBatch = 4;                                      // loads in flight
                if (kConvert || !whole) {
#pragma unroll 1
                    for (int u0 = 0; u0 < kUnits; u0 += kBatch) {
                        uint4 x[kBatch];
                        bool kv[kBatch];
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            const int u = ct + 32 * kConvWarps * (u0 + k), key = (u & 511) >> 3;
                            kv[k] = whole || (key < nv && (key < ns || key >= nl));
                            x[k] = kv[k] ? base[u] : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            const int u = ct + 32 * kConvWarps * (u0 + k);
                            if constexpr (kConvert) {
                                x[k].x = bf16x2_to_f16x2(x[k].x);
                                x[k].y = bf16x2_to_f16x2(x[k].y);
                                x[k].z = bf16x2_to_f16x2(x[k].z);
                                x[k].w = bf16x2_to_f16x2(x[k].w);
                            }
                            if (kConvert || !kv[k]) base[u] = x[k];
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms->vready[vn % kMaxSlots]);
            }
            ++j;
        }
        if (!ok) set_abort(ms, a.status);
    }
    } else {
        if constexpr (kNa >= 3) regs_inc<kRegsSoftmax>();
        // ============================================================ softmax + epilogue
        // 12 warps: warp w reads TMEM lanes 32*(w%4)..+31 (its key lanes) and
        // handles share hf = (w-4)/4 of the row tile's column chunks.
        const int quarter = warp & 3;
        const int hf = (warp - 4) >> 2;
        const int kl = quarter * 32 + lane;  // key lane of S^T, output dim of O^T
        const int key = kl & (kPage - 1);    // my key within its page
        const int half = quarter >> 1;       // which of the tile's pages holds it
        const int st = threadIdx.x - 128;    // 0..383
        const int cb = min(hf * kNa, kNch), ce = min(cb + kNa, kNch);
        const int nch = ce - cb;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        const float sl2 = W.L.scale_log2;
        uint32_t j = 0;
        bool bad = false;  // warp-uniform at every tcgen05 load / store below
        // bounded wait whose outcome all lanes of the warp agree on
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
            const bool w = mbar_wait(bar, parity);
            return __all_sync(0xffffffffu, w);
        };

        const Piece& pc = ms->cur.pc;
        if (st == 0) ms->cur.start(start);

        while (true) {
            if (st == 0) {
                ms->cur.next_piece(W);
                ms->vbad[0] = ms->vbad[1] = 0;
            }
            bar_sync(1, kSoftmaxThreads);
            if (!ms->cur.live) break;
            // V of the tree's nodes is visible to some rows and not to others (0 * NaN): nodes that
            // are not finite are found here, while the first tile loads, two units of 16 bytes a thread
            // with the loads below (one tile for each CTA 20.9 -> 21.3 us, 32 sequences 206 -> 209.5, with
            // an fp32 output 266.5 either way; in the V warps, where V is in shared memory, 272)
            constexpr int kNodeUnits = D / 8, kNodeStep = kSoftmaxThreads / kNodeUnits;
            static_assert(kSoftmaxThreads % kNodeUnits == 0, "a thread's units are kNodeStep nodes apart");
            const int tree_nodes = pc.te == tiles_of(pc.w) ? p.N : 0;
            int vi = st / kNodeUnits;
            const uint4* vt = reinterpret_cast<const uint4*>(a.v_tree) +
                              (((size_t)pc.b * p.N + vi) * p.Hkv + pc.g) * kNodeUnits + st % kNodeUnits;
            uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
            if (vi < tree_nodes) v0 = __ldg(vt);
            if (vi + kNodeStep < tree_nodes) v1 = __ldg(vt + p.Hkv * kSoftmaxThreads);
            // no shift yet (-inf); padding columns keep +inf, so their exponents are -inf and P = 0
            for (int col = st; col < RGP; col += kSoftmaxThreads) {
                ms->neg_m[col] = col < R_seg ? INFINITY : -INFINITY;
                const int i = col < R_seg ? i0 + col / p.G : i0;
                const uint64_t anc = a.anc_mask[(size_t)pc.b * p.N + i] & low_bits(p.N);
                if (!((anc >> i) & 1u)) atomicOr(a.status, LUCETREE_DEV_BAD_NODE);
                ms->depth[col] = (uint8_t)max(__popcll(anc) - 1, 0);  // its proper ancestors
                ms->node[col] = (uint8_t)i;
                ms->out_row[col] = (pc.b * p.N + i) * p.Hq + pc.g * p.G + col % p.G;
            }
            for (int i = st; i < p.N; i += kSoftmaxThreads)
                ms->anc[i] = a.anc_mask[(size_t)pc.b * p.N + i] & low_bits(p.N);
            while (vi < tree_nodes) {
                if (not_finite<BF16, kConvert>(v0)) atomicOr(&ms->vbad[vi >> 5], 1u << (vi & 31));
                if (not_finite<BF16, kConvert>(v1)) atomicOr(&ms->vbad[(vi + kNodeStep) >> 5], 1u << ((vi + kNodeStep) & 31));
                if ((vi += 2 * kNodeStep) >= tree_nodes) break;
                vt += 2 * p.Hkv * kSoftmaxThreads;
                v0 = __ldg(vt);
                v1 = make_uint4(0, 0, 0, 0);
                if (vi + kNodeStep < tree_nodes) v1 = __ldg(vt + p.Hkv * kSoftmaxThreads);
            }
            if (st == 0) {
                ms->empty_cols = 0;
                if (pc.g == 0 && rg == 0) seq_len(a.ctx_len, pc.b, p.max_pages, a.status);  // flags a bad length
            }
            bar_sync(1, kSoftmaxThreads);
            uint64_t lpart[kNa * 8];  // my key's part of the row sums, two columns each
#pragma unroll
            for (int i = 0; i < kNa * 8; ++i) lpart[i] = 0;
            uint32_t page_bits = 0;
            bool stop = false;  // some warp timed out: set by all at the same barrier

#pragma unroll 1
            for (int t = pc.ta; t < pc.te; ++t) {
                // validity of my page for 32 tiles at a time (one load per lane)
                const int tb = (t - pc.ta) & 31;
                if (tb == 0) {
                    const int v = 2 * (t + lane) + half;
                    bool okp = v == pc.w.vp;
                    if (t + lane < pc.te && v < pc.w.vp) {
                        const int pid = a.page_table[(size_t)pc.b * p.max_pages + page_of(pc.w, v)];
                        okp = pid >= 0 && pid < a.num_pages;
                    }
                    page_bits = __ballot_sync(0xffffffffu, okp);
                }
                const int v = 2 * t + half;
                const bool tree = v == pc.w.vp;  // my page holds the tree's nodes (the same for the whole warp)
                bool valid = v <= pc.w.vp && ((page_bits >> tb) & 1u);
                int dmax = 64;     // committed key: it counts for rows of at most this depth
                uint64_t desc = 0;  // tree key: the nodes that see it
                bool part = tree;   // some lane's key does not count for all rows
                if (tree) {
                    valid = valid && key < p.N;
                    if (W.window >= p.N) {
                        // every ancestor is near: the nodes whose masks have my key's bit, by a vote of the
                        // warp for each of its keys (node by node it took as long as the softmax)
                        const uint32_t up = (quarter & 1) * 32, n = p.N > (int)up ? min(p.N - (int)up, 32) : 0;
                        const uint32_t a0 = lane < p.N ? (uint32_t)(ms->anc[lane] >> up) : 0u;
                        const uint32_t a1 = lane + 32 < p.N ? (uint32_t)(ms->anc[lane + 32] >> up) : 0u;
#pragma unroll 4
                        for (uint32_t k = 0; k < n; ++k) {
                            const uint32_t lo = __ballot_sync(0xffffffffu, (a0 >> k) & 1u);
                            const uint32_t hi = __ballot_sync(0xffffffffu, (a1 >> k) & 1u);
                            if (lane == k) desc = (uint64_t)hi << 32 | lo;
                        }
                    } else {
                        const int dj = valid ? max(__popcll(ms->anc[key]) - 1, 0) : 0;
                        const bool sink = (long long)pc.L + dj < W.sinks;
#pragma unroll 1
                        for (int i = 0; i < p.N; ++i) {
                            const uint64_t anc = ms->anc[i];
                            const bool near = __popcll(anc) - 1 - dj < W.window;
                            if (((anc >> key) & 1u) && (near || sink)) desc |= 1ull << i;
                        }
                    }
                } else if (valid) {
                    const int pos = page_of(pc.w, v) * kPage + key;
                    if (pos >= W.sinks) dmax = min(pos - max(pc.L - W.window + 1, -64), 64);
                    valid = pos < pc.L && dmax >= 0;
                }
                if (!tree) part = __any_sync(0xffffffffu, valid && dmax < p.N - 1);
                const bool first = t == pc.ta;

                // The columns of my share whose rows my key counts for, 16 bits a chunk.
                const bool plain = __all_sync(0xffffffffu, valid) && !part;  // all keys of the warp for all rows
                uint64_t vis = valid ? ~0ull : 0;
                if (part) {
                    vis = 0;
#pragma unroll 1
                    for (int b8 = 2 * nch - 1; b8 >= 0 && valid; --b8) {
                        const uint2 d = *reinterpret_cast<const uint2*>((tree ? ms->node : ms->depth) + 16 * cb + 8 * b8);
                        vis = vis << 8 | (tree ? nodes_in(d, desc) : depths_up_to(d, dmax));
                    }
                }

                // The exponents of a tile: P = 2^(s * scale * log2 e - m) with the current
                // shifts, kept in registers (fp16 or bf16 pairs), sums added, the largest
                // exponent tracked.
                //   kTry    with the shifts as they are; if no exponent exceeds kTau, done;
                //   kUndo   else the same pass with the sums subtracted.  What is left is off by at
                //           most 2^-24 p, which kShift scales with the sum to 2^-24 of the
                //           tile's largest term.  From an exponent of 128 on p is infinite and
                //           what is left is not a number;
                //   kShift  the tile's column maxima move the shifts, the sums and O^T
                //           columns so far move with them, then the pass again.  Such a column's
                //           alpha is 0 (at most 2^-128, flushed), which sets its old sum to 0.
                // A range's first tile, or one with a row that has seen no key yet, has no
                // shifts to go by and starts at kShift.  kWarm: the passes that the CTA's
                // first tile needs over nothing, while it loads (both copies of the
                // exponent pass took longer than that with 144 rows: 21.4 us a call, now 20.4).
                enum { kWarm, kTry, kUndo, kShift };
                int phase = j == 0 ? kWarm : first || ms->empty_cols != 0 ? kShift : kTry;
                uint32_t ph[kNa * 8];
                bool pv_prev_done = j == 0;  // PV(j-1) known complete
                if (phase != kWarm) {
                    if (!bad && !wait_all(&ms->s_full, j & 1)) bad = true;
                    if (!bad) tc_fence_after();
                    if (phase == kShift) {
                        if (bar_sync_or(1, kSoftmaxThreads, bad || aborted(ms))) {
                            bad = true;
                            break;
                        }
                        if (st == 0) ms->empty_cols = 0;
                    }
                }
#pragma unroll 1
                while (true) {
                    if (phase == kShift || phase == kWarm) {
#pragma unroll 1
                        for (int cc = 0; cc < (phase == kWarm ? min(nch, 1) : nch); ++cc) {
                            const int c = cb + cc;
                            uint32_t r[16];
                            tmem_ld16(tl + 16 * c, r);
                            tmem_wait_ld_regs16(r);
                            const int lim = R_seg - 16 * c;
                            uint32_t on = phase == kWarm ? 0u : (uint32_t)(vis >> (16 * cc)) & 0xFFFFu;
                            if (lim < 16) on &= (1u << max(lim, 0)) - 1u;
                            // maxima of the 16 columns over the warp's 32 key lanes
                            float mine = 0.f;
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float cm =
                                    redux_max((on >> k) & 1u ? __uint_as_float(r[k]) * sl2 : -INFINITY);
                                if (lane == k) mine = cm;
                            }
                            if (lane < 16) ms->col_red[quarter][16 * c + lane] = mine;
                        }
                    }
                    if (phase == kShift) {
                        bar_sync(1, kSoftmaxThreads);
                        for (int col = st; col < RGP; col += kSoftmaxThreads) {
                            const float cm = fmaxf(fmaxf(ms->col_red[0][col], ms->col_red[1][col]),
                                                   fmaxf(ms->col_red[2][col], ms->col_red[3][col]));
                            const float mo = -ms->neg_m[col];
                            const float mn = fmaxf(mo, cm);
                            ms->alpha[col] = mn > mo ? ex2(mo - mn) : 1.f;
                            ms->neg_m[col] = -mn;
                            if (mn == -INFINITY) ms->empty_cols = 1;
                        }
                        bar_sync(1, kSoftmaxThreads);
#pragma unroll
                        for (int cc = 0; cc < kNa; ++cc) {
                            if (cc >= nch) continue;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float2 al = *reinterpret_cast<const float2*>(ms->alpha + 16 * (cb + cc) + 2 * k);
                                const float2 l = unpack2(lpart[cc * 8 + k]);
                                lpart[cc * 8 + k] = pack2(al.x > 0.f ? l.x * al.x : 0.f, al.y > 0.f ? l.y * al.y : 0.f);
                            }
                        }
                        if (!first) {
                            // O^T columns accumulated so far move with their shift, once
                            // PV(j-1) has finished adding to them (a warp that timed out
                            // here skips its TMEM accesses but keeps to the barriers)
                            if (!bad && j > 0 && !wait_all(&ms->pv_done, (j - 1) & 1)) bad = true;
                            pv_prev_done = true;
                            if (!bad) tc_fence_after();
#pragma unroll 1
                            for (int cc = 0; cc < nch && !bad; ++cc) {
                                const int c = cb + cc;
                                bool any = false;
#pragma unroll
                                for (int k = 0; k < 16; ++k) any |= ms->alpha[16 * c + k] != 1.f;
                                if (!any) continue;
#pragma unroll 1
                                for (int h = 0; h < Lay::kDh; ++h) {
                                    uint32_t r[16];
                                    const uint32_t addr = tl + (h ? Lay::kColO1 : Lay::kColO0) + 16 * c;
                                    tmem_ld16(addr, r);
                                    tmem_wait_ld_regs16(r);
#pragma unroll
                                    for (int k = 0; k < 16; ++k)
                                        r[k] = __float_as_uint(__uint_as_float(r[k]) * ms->alpha[16 * c + k]);
                                    tmem_st16(addr, r);
                                }
                            }
                            if (!bad) tmem_wait_st();
                        }
                    }
                    float ex = -INFINITY;
                    // One pass in two copies, without masks and with them: the hot one is a
                    // short straight line (instruction fetch is what the softmax warps wait
                    // for most).  16-column chunks; the TMEM load of the next one is in
                    // flight while one is computed.
                    auto pass = [&](auto masked) {
                        const float sign1 = phase == kUndo ? -1.f : 1.f;
                        const uint64_t sign = pack2(sign1, sign1), scale = pack2(sl2, sl2);
                        const uint64_t on = masked.value && phase != kWarm ? vis : 0;
                        uint32_t rn[16];
                        tmem_ld16(tl + 16 * cb, rn);
#pragma unroll
                        for (int cc = 0; cc < kNa; ++cc) {
                            if (cc >= nch) continue;
                            uint32_t r[16];
                            tmem_wait_ld_regs16(rn);
#pragma unroll
                            for (int k = 0; k < 16; ++k) r[k] = rn[k];
                            if (cc + 1 < nch) tmem_ld16(tl + 16 * (cb + cc + 1), rn);
                            const int c = cb + cc;
#pragma unroll
                            for (int hb = 0; hb < 2; ++hb) {
                                const ulonglong2* nm = reinterpret_cast<const ulonglong2*>(ms->neg_m + 16 * c + 8 * hb);
                                const ulonglong2 na = nm[0], nb = nm[1];
                                const uint64_t m2[4] = {na.x, na.y, nb.x, nb.y};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int i = 8 * hb + 2 * k;
                                    float2 x = unpack2(fma2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), scale,
                                                            m2[k]));
                                    if constexpr (masked.value) {
                                        if (!((on >> (16 * cc + i)) & 1u)) x.x = -INFINITY;
                                        if (!((on >> (16 * cc + i + 1)) & 1u)) x.y = -INFINITY;
                                    }
                                    ex = fmaxf(ex, fmaxf(x.x, x.y));
                                    const float p0 = ex2(x.x), p1 = ex2(x.y);
                                    uint64_t& acc = lpart[cc * 8 + 4 * hb + k];
                                    acc = fma2(sign, pack2(p0, p1), acc);
                                    ph[8 * cc + 4 * hb + k] = PV16 ? pack_bf162(p0, p1) : pack_half2(p0, p1);
                                }
                            }
                        }
                    };
                    if (!bad && !plain) pass(std::true_type{});
                    if (!bad && plain) pass(std::false_type{});
                    if (phase == kWarm) {
                        // (nothing has been multiplied yet: it has summed up whatever TMEM held)
#pragma unroll
                        for (int i = 0; i < kNa * 8; ++i) lpart[i] = 0;
                    }
                    if (phase == kShift) break;
                    if (phase == kUndo) {
                        phase = kShift;
                        continue;
                    }
                    if (phase == kWarm && !wait_all(&ms->s_full, 0)) bad = true;
                    if (phase == kWarm && !bad) tc_fence_after();
                    // one barrier decides the path; a second one only when it says "again", to
                    // tell a timeout (somewhere) from a shift update
                    const bool bad_now = bad || aborted(ms);
                    if (!bar_sync_or(1, kSoftmaxThreads, bad_now || phase == kWarm || ex > kTau)) break;
                    if (bar_sync_or(1, kSoftmaxThreads, bad_now)) {
                        bad = stop = true;
                        break;
                    }
                    if (st == 0) ms->empty_cols = 0;
                    phase = phase == kWarm ? kShift : kUndo;
                }
                if (stop) break;
                // S^T is no longer read: the next tile's QK may overwrite it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms->s_free);

                // P^T is free once PV(j-1) has completed; then this tile's P goes in:
                // [8-column block][128 keys][8 columns]
                if (!pv_prev_done && !wait_all(&ms->pv_done, (j - 1) & 1)) bad = true;
                if (!bad) {
                    tc_fence_after();
#pragma unroll
                    for (int bi = 0; bi < 2 * kNa; ++bi) {
                        if (bi >= 2 * nch) continue;
                        *reinterpret_cast<uint4*>(sP + (2 * cb + bi) * 2048 + kl * 16) =
                            make_uint4(ph[4 * bi], ph[4 * bi + 1], ph[4 * bi + 2], ph[4 * bi + 3]);
                    }
                }
                if (__builtin_expect(t == pc.te - 1 && (ms->vbad[0] | ms->vbad[1]) != 0, 0)) {
                    // V(j) is in the ring until its PV, which waits for this warp's P^T: the chunks of
                    // the tree's half, as the V warps left them (ring position as there)
                    const uint32_t vbase = ((j + 1 < n_tiles ? j + 2 : j + 1) + j) * kChunks;
#pragma unroll 1
                    for (int c = (pc.w.vp & 1); c < kChunks; c += 2) {
                        const uint32_t vn = j * kChunks + c;
                        if (!bad && !wait_all(&ms->vready[vn % kMaxSlots], (vn / kMaxSlots) & 1)) bad = true;
                        uint4* base = reinterpret_cast<uint4*>(sSlots + ((vbase + c) % kNS) * kChunkBytes);
                        for (int u = st; u < kChunkBytes / 16 && !bad; u += kSoftmaxThreads)
                            if ((ms->vbad[(u & 511) >> 8] >> ((u >> 3) & 31)) & 1u) base[u] = make_uint4(0, 0, 0, 0);
                    }
                }
                tc_fence_before();
                fence_proxy_async_smem();  // P^T stores -> tensor-core reads
                __syncwarp();              // every lane's stores and fence come before lane 0's arrive
                if (!bad && lane == 0) mbar_arrive(&ms->p_full);
                ++j;
            }

            // ---------------------------------------------------------- epilogue
            // Row sums and shifts first: they are final once the last tile's
            // exponent pass is done, while the last PV is still running.
#pragma unroll
            for (int cc = 0; cc < kNa; ++cc) {
                if (cc >= nch) continue;
                float v[16];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 y = unpack2(lpart[cc * 8 + k]);
                    v[2 * k] = y.x;
                    v[2 * k + 1] = y.y;
                }
                const float cs = col_sum16(v, lane);
                if ((lane & 1) == 0) ms->col_red[quarter][16 * (cb + cc) + (lane >> 1)] = cs;
            }
            bar_sync(1, kSoftmaxThreads);
            const bool whole = pc.whole();
            float* slot = W.L.ws + slot_index(p, rg, cta, pc.b * p.Hkv + pc.g) * slot_floats(p);
            for (int col = st; col < R_seg; col += kSoftmaxThreads) {
                const float l = (ms->col_red[0][col] + ms->col_red[1][col]) + (ms->col_red[2][col] + ms->col_red[3][col]);
                const float m = -ms->neg_m[col];
                if (whole) {
                    // (0: no key; a sum that is not a number makes the row one, and is flagged below)
                    ms->alpha[col] = l != 0.f ? 1.f / l : 0.f;
                    if (a.lse) a.lse[ms->out_row[col]] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
                } else {
                    slot[(size_t)RG * D + col] = m;
                    slot[(size_t)RG * D + RG + col] = l;
                }
            }
            // the consensus point for a timeout in the piece's last tile (a
            // piece that failed has written garbage sums; the call reports the
            // failure through the status word)
            const bool got = !bad && mbar_wait(&ms->pv_done, (j - 1) & 1);
            if (bar_sync_or(1, kSoftmaxThreads, bad || !got || aborted(ms))) {
                bad = true;
                break;
            }
            tc_fence_after();
            if (__builtin_expect((ms->vbad[0] | ms->vbad[1]) != 0, 0)) {
                for (int col = st; col < R_seg; col += kSoftmaxThreads) {
                    const uint64_t anc = ms->anc[ms->node[col]];
                    bool hit = false;
                    for (uint64_t rest = anc & ((uint64_t)ms->vbad[1] << 32 | ms->vbad[0]); rest != 0 && !hit; rest &= rest - 1) {
                        const int dj = max(__popcll(ms->anc[__ffsll((long long)rest) - 1]) - 1, 0);
                        hit = __popcll(anc) - 1 - dj < W.window || (long long)pc.L + dj < W.sinks;
                    }
                    if (!hit) continue;
                    const float nan = __int_as_float(0x7FC00000);
                    if (!whole) {
                        slot[(size_t)RG * D + RG + col] = nan;
                        continue;
                    }
                    ms->alpha[col] = nan;
                    if (a.lse) a.lse[ms->out_row[col]] = nan;
                }
                bar_sync(1, kSoftmaxThreads);
            }
            bool finite = true;
#pragma unroll 1
            for (int x = 0; x < nch * Lay::kDh; ++x) {
                const int c = cb + x / Lay::kDh, h = x % Lay::kDh, d = h * 128 + kl;
                uint32_t r[16];
                tmem_ld16(tl + (h ? Lay::kColO1 : Lay::kColO0) + 16 * c, r);
                tmem_wait_ld_regs16(r);
                float* part = slot + (size_t)(16 * c) * D + d;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int col = 16 * c + k;
                    if (col >= R_seg) continue;
                    float o = __uint_as_float(r[k]);
                    if (!whole) {
                        part[k * D] = o;
                        continue;
                    }
                    o *= ms->alpha[col];
                    finite = finite && isfinite(o);
                    const size_t at = (size_t)ms->out_row[col] * D + d;
                    if constexpr (PV16) {
                        store_out(reinterpret_cast<__nv_bfloat16*>(W.out) + at, o);
                    } else {
                        if (BF16 || W.out_dtype == LUCETREE_F32) reinterpret_cast<float*>(W.out)[at] = o;
                        else store_out(reinterpret_cast<__half*>(W.out) + at, o);
                    }
                }
            }
            if (!finite) atomicOr(a.status, LUCETREE_DEV_NONFINITE);
            tc_fence_before();
            bar_sync(1, kSoftmaxThreads);  // the piece's values in shared memory are no longer read
        }
        if (bad) set_abort(ms, a.status);
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

struct Maps {
    CUtensorMap k, v, q, kt, vt;
};

template <int D, bool BF16, int RGP, bool PV16>
cudaError_t launch_one(const Maps& m, const WinLaunch& W, cudaStream_t stream) {
    using Lay = Layout<D, RGP>;
    auto kern = window_tc_kernel<D, BF16, RGP, PV16>;
    static SmemLimitSeen seen;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), Lay::kBytes, seen);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid_ctas(W.L.plan)), dim3(kThreads), Lay::kBytes, stream, m.k, m.v, m.q, m.kt, m.vt, W);
}

template <int D, bool BF16, bool PV16>
cudaError_t launch_rgp(const Maps& m, const WinLaunch& W, cudaStream_t stream) {
    static_assert(kRowsMax == 144, "one instantiation per padded row count up to kRowsMax");
    switch ((W.L.plan.rg.RG + 15) / 16) {
        case 1: return launch_one<D, BF16, 16, PV16>(m, W, stream);
        case 2: return launch_one<D, BF16, 32, PV16>(m, W, stream);
        case 3: return launch_one<D, BF16, 48, PV16>(m, W, stream);
        case 4: return launch_one<D, BF16, 64, PV16>(m, W, stream);
        case 5: return launch_one<D, BF16, 80, PV16>(m, W, stream);
        case 6: return launch_one<D, BF16, 96, PV16>(m, W, stream);
        case 7: return launch_one<D, BF16, 112, PV16>(m, W, stream);
        case 8: return launch_one<D, BF16, 128, PV16>(m, W, stream);
        case 9: return launch_one<D, BF16, 144, PV16>(m, W, stream);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_bf16_256(const Maps&, const WinLaunch&, cudaStream_t);
cudaError_t launch_bf16_128(const Maps&, const WinLaunch&, cudaStream_t);
cudaError_t launch_bf16_256_out16(const Maps&, const WinLaunch&, cudaStream_t);
cudaError_t launch_bf16_128_out16(const Maps&, const WinLaunch&, cudaStream_t);
cudaError_t launch_f16_256(const Maps&, const WinLaunch&, cudaStream_t);
cudaError_t launch_f16_128(const Maps&, const WinLaunch&, cudaStream_t);

}  // namespace win
}  // namespace lucetree
