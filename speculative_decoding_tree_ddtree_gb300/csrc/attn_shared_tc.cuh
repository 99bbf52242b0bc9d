// attn_shared_tc.cuh -- tree-verify attention over shared prefixes on the
// 5th-generation tensor cores.
//
// A CTA goes through the pieces that the plan made for it: a block of up to 128
// query rows against key tiles of two 64-token pages.  S = Q K^T with the rows on
// the MMA's M = 128 and the keys on its N = 128, a softmax with one row to a tensor
// memory lane (so a row's maximum and sum need no exchange between lanes), P written
// over S, O += P V with P read from tensor memory.  Per tile that reads Q, K and V from
// shared memory once each (192 KB with D = 256); with the keys on M, as the windowed
// attention has them for its few rows, it is V^T and P^T instead of V (272 KB for 144 rows),
// and shared memory's bandwidth is what bounds many rows.
//   - Pairs of CTAs (cta_group::2, M = 256) where the mean group has more than 128 rows: each CTA has
//     half of the block's nodes and loads half of the keys (K) and of the dims (V), so a tile costs
//     half of the loads and of shared memory's reads for a row.  Without them 16 sequences at budget
//     22 under 16,384 tokens took 148 us instead of 113.
//   - Two S buffers: QK of the next tile runs while a tile's softmax does.  D = 256 uses all
//     512 columns (S 2 x 128, O 256).
//   - Eight softmax warps: a tile's first page belongs to one warpgroup, the second to
//     the other.  A page is all that a row's mask depends on, so it is one 64-bit word
//     for each thread: all keys (common pages), the first n (a sequence's own last
//     page), the row's ancestors (its tree's page), none (another sequence's page: no
//     exponents are computed where that holds for the whole warp).
//   - Shifts (a row's reference maximum) move only when an exponent exceeds 8; one
//     barrier a tile says whether any does.  Then the sums as they were before the tile and
//     the O rows so far are scaled, and the pass is made again.
//   - P is bf16 for a bf16 output (half a step of it is 2^-8 of a term, as much as the
//     output's own rounding, and the terms' roundings average out) and V is multiplied
//     as it lands; otherwise P is fp16 (2^-11) and bf16 V is converted in shared memory
//     (exact from 2^-17 to below 65536).
//
// Measured with 24 query and 4 KV heads of 256 dims, bf16 in and out, the merge included: 96
// sequences at budget 22 under 16,384 tokens 457 to 460 us (1.85 PFLOP/s; 500 to 520 in long runs, where
// the clock gives way); 16 such sequences 98; one token each of 192 60, of 96 41, of 8 21 (67 MB of keys and values, 10 us at HBM's rate;
// four tiles in most CTAs where the mean is 3.4 are 1.8 of the rest, the others the chain of plan,
// page table and first tile, the last tile and the merge).  With one CTA a tile of 128 KB takes 2.9 us
// where every page is read once (24 groups of 8 beams: 86 us), which is HBM's rate.
#pragma once

#include "attn_prefix_tc.cuh"
#include "attn_shared.cuh"

namespace lucetree {
namespace shr {

using namespace tc;
using prefix_tc::bf16x2_to_f16x2;
using prefix_tc::ex2;
using prefix_tc::kChunkBytes;
using prefix_tc::kSmemLimit;
using prefix_tc::kTau;
using prefix_tc::kTmemCols;
using prefix_tc::pack_half2;

constexpr int kConvWarps = 2;                      // warps 2, 3
constexpr int kSmWarps = 8;                        // warps 4 .. 11: two warpgroups
constexpr int kSoftmaxThreads = 32 * kSmWarps;
constexpr int kThreads = 128 + kSoftmaxThreads;
constexpr int kMaxSlots = 12;
constexpr int kNodeWords = 12;  // tree nodes of a block's sequences: at most 254 + 2 N
constexpr int kBadWords = kNodeWords + 8;  // ... and the sequences

struct Misc {
    float xchg[2][kRows];        // a row's values for the other warpgroup's half
    uint64_t empty[kMaxSlots];   // of ring slots
    uint64_t kfull[kMaxSlots];   // K chunk n at [n % kMaxSlots]: landed, in the first CTA of a pair: in both
    uint64_t vfull[kMaxSlots];   // V chunk n at [n % kMaxSlots]: landed ...
    uint64_t vready[kMaxSlots];  // ... made the operand
    uint64_t s_full[2], p_full[2];  // of tiles j, at [j & 1]
    uint64_t pv_done[2];            // (PV(j - 2) is done once S(j) is there: two of them tell PV(j) from it)
    uint64_t q_full, q_empty, drain;
    uint32_t tmem_base;
    int abort_flag;
    int pass;   // 1: the second one, with all values looked at ...
    int again;  // ... which comes if this is 1
    // piece n at [n % Lay::kBadSets]: tree nodes, and sequences with own pages, whose V is not finite
    uint32_t vbad[][kBadWords];
};

template <int D, bool PAIR>
struct Lay {
    // Ring chunks per operand.  One CTA: 16 KB each, K [128 keys][64 dims], V [64 keys][128 dims].  A
    // pair, whose CTAs hold half of each operand: all of it, K [64 keys of its page][D dims], V
    // [128 keys][D / 2 dims] (in chunks of 16 KB with D = 256, 96 sequences at budget 22 took
    // 531 us instead of 470: the waits and commits of the warp that issues the MMAs count).
    static constexpr int kChunks = PAIR ? 1 : D / 64;
    static constexpr int kSlotBytes = PAIR ? D / 128 * kChunkBytes : kChunkBytes;
    static constexpr int kQBytes = D / 64 * kChunkBytes;
    // Pieces from the one whose rows are being finished to the last one with V in the ring: its next
    // six (12 slots of K and V in turn), three or fewer.
    static constexpr int kBadSets = PAIR && D == 128 ? 8 : 4;
    static constexpr int kMiscBytes = (sizeof(Misc) + 4 * kBadSets * kBadWords + 127) / 128 * 128;
    static constexpr int kRaw = (kSmemLimit - 1024 - kQBytes - kMiscBytes) / kSlotBytes;
    static constexpr int kNS = kRaw > kMaxSlots ? kMaxSlots : kRaw;
    static constexpr int kSlotOff = kQBytes;
    static constexpr int kMiscOff = kSlotOff + kNS * kSlotBytes;
    static constexpr int kBytes = kMiscOff + kMiscBytes + 1024;
    static constexpr uint32_t kColO = 256;  // after S 0 and S 1
    static_assert(kNS >= 2 * kChunks, "the ring holds a K and a V operand");
    static_assert(kBytes <= kSmemLimit && kBytes > kSmemLimit / 2, "one CTA per SM: it owns all tensor memory columns");
    static_assert(kColO + D <= kTmemCols, "tensor memory columns");
};

__device__ __forceinline__ void set_abort(Misc* ms, uint32_t* status) {
    if (atomicExch(&ms->abort_flag, 1) == 0) atomicOr(status, LUCETREE_DEV_TIMEOUT);
}
__device__ __forceinline__ bool aborted(Misc* ms) { return *(volatile int*)&ms->abort_flag != 0; }

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
// Two fp32 in one 64-bit register pair, and one instruction for two operations.
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Four lanes with four units of U words each: unit k of lane i becomes unit i of lane k.
template <int U>
__device__ __forceinline__ void turn4(uint32_t (&v)[4 * U], int lane) {
#pragma unroll
    for (int s = 1; s < 4; s <<= 1) {
        const bool odd = (lane & s) != 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & s) continue;
#pragma unroll
            for (int y = 0; y < U; ++y) {
                uint32_t &lo = v[k * U + y], &hi = v[(k + s) * U + y];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, s);
                if (odd) lo = got;
                else hi = got;
            }
        }
    }
}

__device__ __forceinline__ uint64_t low_bits(int n) { return n > 0 ? ~0ull >> (64 - n) : 0ull; }  // n <= 64

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

// The CTA's tiles in order: piece and tile within its segment.
struct Cursor {
    int next, then, left;  // the places of the next two pieces in the plan, and how many come
    int serial;      // number of the current one, counted over both passes
    int t;
    bool live;
    Piece pc;
    __device__ void start(const Launch& W, const Cta& c, int pass) {
        next = (int)blockIdx.x / W.d.pair;
        then = c.next;
        left = c.pieces;
        serial = pass * c.pieces - 1;
        t = -1;
        pc.te = 0;
        live = true;
    }
    __device__ void next_piece(const Launch& W) {
        live = left > 0;
        if (!live) return;
        --left;
        ++serial;
        const int4* x = reinterpret_cast<const int4*>(W.plan.piece + next);
        next = then++;
        int4* w = reinterpret_cast<int4*>(&pc);
        w[0] = __ldg(x);
        w[1] = __ldg(x + 1);
        w[2] = __ldg(x + 2);
        t = pc.ta;
    }
    __device__ bool first() const { return t == pc.ta; }
    __device__ bool last() const { return t == pc.te - 1; }
    __device__ void step(const Launch& W) {
        if (++t >= pc.te) next_piece(W);
    }
};

// A page of a block's key list.
struct Page {
    int id;    // pool page, -1: none; a tree page: its first node
    int seq;   // a sequence's own page: which of the block's; a tree page: its number; -1: all see it
    int keys;  // keys of it that exist (0: a page that is missing)
    bool tree;
};
__device__ __forceinline__ Page page_at(const Launch& W, const Piece& p, int v) {
    Page r = {-1, -1, 0, false};
    if (v >= p.vp) return r;
    int col = v;
    long long row = p.b0;
    r.keys = kPage;
    if (v >= p.used) {
        const int x = __ldg(&W.plan.seq[p.b0].off) + v - p.used;
        const int past = x - __ldg(&W.plan.seq[p.b0 + p.seqs].off);
        if (past >= 0) {
            r.tree = true;
            r.seq = past;
            r.id = p.b0 * W.d.N + past * kPage;
            r.keys = min(kPage, p.seqs * W.d.N - past * kPage);
            return r;
        }
        int lo = p.b0, hi = p.b0 + p.seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (__ldg(&W.plan.seq[mid].off) <= x) lo = mid;
            else hi = mid - 1;
        }
        row = lo;
        r.seq = lo - p.b0;
        col = p.used + x - __ldg(&W.plan.seq[lo].off);
        r.keys = min(kPage, __ldg(&W.plan.seq[lo].L) - col * kPage);
    }
    const int id = __ldg(W.a.page_table + row * W.a.max_pages_per_seq + col);
    if (id >= 0 && id < W.a.num_pages) r.id = id;
    else r.keys = 0;
    return r;
}
// In one word: keys, tree, seq + 1.
__device__ __forceinline__ int page_word(const Page& p) { return p.keys | (p.tree ? 0x80 : 0) | (p.seq + 1) << 8; }

template <int D, bool BF16, bool PV16, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    shared_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qown,
                     const __grid_constant__ CUtensorMap tm_qlarge,
                     const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                     const __grid_constant__ Launch W) {
    using L = Lay<D, PAIR>;
    static_assert(BF16 || !PV16, "fp16 inputs run PV on fp16 anyway");
    constexpr bool kConvert = BF16 && !PV16;  // V to fp16 on chip
    constexpr int kChunks = L::kChunks;
    constexpr int kNS = L::kNS;
    constexpr int kBadSets = L::kBadSets;
    constexpr int kSlotBytes = L::kSlotBytes;
    constexpr int kPageBytes = kSlotBytes / 2;  // of V in a pair

    extern __shared__ uint8_t smem_raw[];
    uint8_t* const base0 = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc* ms = reinterpret_cast<Misc*>(base0 + L::kMiscOff);

    const lucetree_attn_args& a = W.a;
    const Dims& d = W.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0u;  // CTA of the pair

    // ---------------------------------------------------------------- set-up
    // (reads no global memory: it overlaps the previous kernel's tail)
    if (threadIdx.x == 0) {
        const int firsts = PAIR && rank == 0 ? 2 : 1;  // a pair's second CTA tells the first one
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&ms->empty[i], 1);
            mbar_init(&ms->kfull[i], firsts);
            mbar_init(&ms->vfull[i], 1);
            mbar_init(&ms->vready[i], PAIR ? 2 * kConvWarps : kConvWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms->s_full[i], 1);
            mbar_init(&ms->p_full[i], PAIR ? 2 * kSmWarps : kSmWarps);
            mbar_init(&ms->pv_done[i], 1);
        }
        mbar_init(&ms->q_full, firsts);
        mbar_init(&ms->q_empty, 1);
        mbar_init(&ms->drain, 1);
        ms->abort_flag = 0;
        ms->pass = ms->again = 0;
        mbar_fence_init();
    }
    if (warp == 2)
        for (int i = lane; i < kBadSets * kBadWords; i += 32) ms->vbad[i / kBadWords][i % kBadWords] = 0;
    // (rows of Q past a block's own are whatever lies there: their rows of S and O are never used)
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(&ms->tmem_base, kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&ms->tmem_base, kTmemCols);
            tmem_relinquish();
        }
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_qown);
        prefetch_tensormap(&tm_qlarge);
        prefetch_tensormap(&tm_kt);
        prefetch_tensormap(&tm_vt);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // both CTAs' barriers are there
    tc_fence_after();
    auto teardown = [&]() {
        const uint32_t tmem = ms->tmem_base;
        if (threadIdx.x >> 5 == 1) {
            if constexpr (PAIR) tmem_dealloc_pair(tmem, kTmemCols);
            else tmem_dealloc(tmem, kTmemCols);
        }
    };

    // inputs may come from the previous kernel on the stream
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    // (the record is loaded with the head, not after it, and the first piece on its way)
    if (threadIdx.x < 3)
        prefetch_l1(reinterpret_cast<const char*>(W.plan.piece + blockIdx.x / d.pair) + min(32 * threadIdx.x, 47u));
    Cta start = W.plan.cta[blockIdx.x / d.pair];
    const bool fits = plan_fits(W);
    if (!fits) start.tiles = 0;
    if (start.tiles == 0) {  // uniform across the CTA: nothing to do but give TMEM back
        if (!fits && threadIdx.x == 0) atomicOr(a.status, LUCETREE_DEV_BAD_ROW);
        __syncwarp();
        if constexpr (PAIR) cluster_sync();
        teardown();
        return;
    }

    // A value of a sequence's own pages that is not finite spoils the rows of the block's other sequences
    // too (0 x it is NaN).  Looking for those in every page takes the V warps longer than the
    // products do (32 sequences under 32,768 tokens: 50 -> 70 us); so the rows are looked at
    // instead, once a piece is done, and if one is not finite the CTA goes through its pieces
    // again and looks at all values.  Numbers of tiles, chunks and pieces go on.
#pragma unroll 1
    for (;;) {
        // (what a pass finds out anew is kept in no register for the next one)
        uint32_t zero, tid;
        asm volatile("mov.u32 %0, 0;\n\tmov.u32 %1, %%tid.x;" : "=r"(zero), "=r"(tid));
        const int warp = tid >> 5, lane = tid & 31;
        const uint32_t rank = PAIR ? cluster_rank() : 0u;
        uint8_t* const smem =
            reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + zero + 1023) & ~uintptr_t(1023));
        uint8_t* const sQ = smem;
        uint8_t* const sSlots = smem + L::kSlotOff;
        Misc* const ms = reinterpret_cast<Misc*>(smem + L::kMiscOff);
        const uint32_t tmem = *(volatile uint32_t*)&ms->tmem_base;
        const int pass = *(volatile int*)&ms->pass;
        const uint32_t n_tiles = (uint32_t)start.tiles;
        const uint32_t tiles0 = pass * n_tiles, chunks0 = tiles0 * kChunks, ring0 = 2 * chunks0;
        if (warp == 0) {
            // ============================================================ TMA producer
            const int oob_row = a.num_pages * d.Hkv * kPage;  // first row past the pool: zero fill
            const uint64_t pol_once = policy_evict_first(), pol_again = policy_evict_normal();
            uint32_t chunk = chunks0, vchunk = chunks0;  // of K, of V
            int q_loads = pass * start.pieces;
            bool ok = true;
            // A tile's pages: pool row, or for a tree page -1 - (first node)
            struct Operand {
                int at0, at1;
                int g;
                uint64_t pol;
            };
            const bool leader = elect_one();
            uint32_t slot = ring0 % kNS, turn = ring0 / kNS;  // ring position and its turn
            auto next_slot = [&]() {
                const bool w = mbar_wait(&ms->empty[slot], (turn & 1) ^ 1);
                return __all_sync(0xffffffffu, w);  // lanes agree on a timeout
            };
            auto advance = [&]() {
                if (++slot == (uint32_t)kNS) {
                    slot = 0;
                    ++turn;
                }
            };
            auto issue_k = [&](const Operand& o) -> bool {
                const bool tree0 = o.at0 < 0, tree1 = o.at1 < 0;
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    if (!next_slot()) return false;
                    if (leader) {
                        uint8_t* dst = sSlots + slot * kSlotBytes;
                        uint64_t* bar = &ms->kfull[chunk % kMaxSlots];
                        if constexpr (PAIR) {
                            // [64 keys of page `rank`][dims], 64 dims after the other 64
                            const int at = rank ? o.at1 : o.at0;
                            mbar_arrive_expect_tx(bar, kSlotBytes);
                            if (at < 0) {
#pragma unroll 1
                                for (int x = 0; x < D / 64; ++x) tma_load_3d(dst + 8192 * x, &tm_kt, 64 * x, o.g, -1 - at, bar);
                            } else {
                                tma_load_3d_hint(dst, &tm_k, 0, at, 0, bar, o.pol);
                            }
                        } else {
                            // [128 keys: page 0 then page 1][dims 64 * c .. +63]
                            mbar_arrive_expect_tx(bar, kSlotBytes);
                            if (tree0) tma_load_3d(dst, &tm_kt, 64 * c, o.g, -1 - o.at0, bar);
                            else tma_load_2d_hint(dst, &tm_k, 64 * c, o.at0, bar, o.pol);
                            if (tree1) tma_load_3d(dst + 8192, &tm_kt, 64 * c, o.g, -1 - o.at1, bar);
                            else tma_load_2d_hint(dst + 8192, &tm_k, 64 * c, o.at1, bar, o.pol);
                        }
                    }
                    __syncwarp();
                    ++chunk;
                    advance();
                }
                return true;
            };
            auto issue_v = [&](const Operand& o) -> bool {
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    if (!next_slot()) return false;
                    if (leader) {
                        uint8_t* dst = sSlots + slot * kSlotBytes;
                        uint64_t* bar = &ms->vfull[vchunk % kMaxSlots];
                        if constexpr (PAIR) {
                            // [64 keys][D / 2 dims, 64 after the other 64] of page 0, then page 1
                            mbar_arrive_expect_tx(bar, kSlotBytes);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int at = h ? o.at1 : o.at0;
                                if (at < 0) {
#pragma unroll 1
                                    for (int x = 0; x < D / 128; ++x)
                                        tma_load_3d(dst + kPageBytes * h + 8192 * x, &tm_vt, 64 * (D / 128 * rank + x), o.g,
                                                    -1 - at, bar);
                                } else {
                                    tma_load_3d_hint(dst + kPageBytes * h, &tm_v, 0, at, D / 128 * rank, bar, o.pol);
                                }
                            }
                        } else {
                            // [64 keys of a page][128 dims], 64 dims after the other 64
                            const int at = c & 1 ? o.at1 : o.at0, x = 128 * (c >> 1);
                            mbar_arrive_expect_tx(bar, kSlotBytes);
                            if (at < 0) {
                                tma_load_3d(dst, &tm_vt, x, o.g, -1 - at, bar);
                                tma_load_3d(dst + 8192, &tm_vt, x + 64, o.g, -1 - at, bar);
                            } else {
                                tma_load_3d_hint(dst, &tm_v, 0, at, x / 64, bar, o.pol);
                            }
                        }
                    }
                    __syncwarp();
                    ++vchunk;
                    advance();
                }
                return true;
            };
            Cursor cur;
            cur.start(W, start, pass);
            // the operands of 16 tiles, a page to a lane, one batch ahead
            auto load_batch = [&](int tb) {
                const int v = 2 * tb + lane;
                if (v >= 2 * cur.pc.te) return oob_row;
                const Page p = page_at(W, cur.pc, v);
                if (p.tree) return -1 - p.id;
                if (p.id < 0 && v < cur.pc.vp) atomicOr(a.status, LUCETREE_DEV_BAD_PAGE);
                return p.id >= 0 ? (p.id * d.Hkv + cur.pc.g) * kPage : oob_row;
            };
            int at_cur = 0, at_next = 0;
            Operand v_op = {0, 0, 0, pol_once};  // of the tile whose V is still to be loaded
            bool have_v = false;
            // K(t), then V(t-1); after the last tile its V alone
            while (ok && cur.live) {
                cur.step(W);
                Operand op = v_op;
                const bool have_k = cur.live;
                if (have_k) {
                    const int rel = cur.t - cur.pc.ta;
                    if ((rel & 15) == 0) at_cur = at_next;
                    if (rel == 0 || (rel & 15) == 8) {
                        at_next = load_batch(cur.t + (rel == 0 ? 0 : 8));
                        if (rel == 0) at_cur = at_next;
                    }
                    if (rel == 0) {
                        // a new segment: its queries replace the previous ones once their last QK is done
                        if (cur.serial > 0) {
                            const bool w = mbar_wait(&ms->q_empty, (cur.serial - 1) & 1);
                            if (!(ok = __all_sync(0xffffffffu, w))) break;
                        }
                        if (leader) {
                            const int kind = cur.pc.kind(), nodes = d.half(kind);
                            const CUtensorMap* tm = kind == kOwnCut ? &tm_qown : kind == kLargeCut ? &tm_qlarge : &tm_q;
                            mbar_arrive_expect_tx(&ms->q_full, D / 64 * nodes * d.G * 128);
#pragma unroll 1
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_3d(sQ + c * kChunkBytes, tm, 64 * c, cur.pc.g * d.G, cur.pc.node0 + (int)rank * nodes,
                                            &ms->q_full);
                        }
                        __syncwarp();
                        ++q_loads;
                    }
                    op.at0 = __shfl_sync(0xffffffffu, at_cur, 2 * (rel & 15));
                    op.at1 = __shfl_sync(0xffffffffu, at_cur, 2 * (rel & 15) + 1);
                    op.g = cur.pc.g;
                    op.pol = cur.pc.how & 1 ? pol_again : pol_once;
                }
                if (have_k) ok = issue_k(op);
                if (ok && have_v) ok = issue_v(v_op);
                v_op = op;
                have_v = have_k;
            }
            // Arrivals that follow MMAs come on their own, in no order that is promised, in a pair at
            // both CTAs; none may find its CTA gone.  Those of S are all waited for by the softmax; here
            // the last ones of every slot, of the queries and of the two O accumulations.
            auto arrived = [&](uint64_t* bar, uint32_t parity) {
                const bool w = mbar_wait(bar, parity);
                return __all_sync(0xffffffffu, w);
            };
            if (ok) {
                const uint32_t end = tiles0 + n_tiles;
#pragma unroll 1
                for (int c = 0; c < kNS && ok; ++c) {
                    ok = next_slot();
                    advance();
                }
                ok = ok && arrived(&ms->q_empty, cur.serial & 1);
#pragma unroll 1
                for (uint32_t j = end > 1 ? end - 2 : 0u; j < end && ok; ++j) ok = arrived(&ms->pv_done[j & 1], (j >> 1) & 1);
            }
            if (!ok || aborted(ms)) {
                set_abort(ms, a.status);
                // wait (bounded) for this CTA's own copies still in flight
                if (lane == 0) {
                    const uint32_t first = chunk > (uint32_t)kNS ? chunk - kNS : 0u;
                    for (uint32_t c = first; c < chunk; ++c)
                        mbar_wait(&ms->kfull[c % kMaxSlots], (c / kMaxSlots) & 1, 200000000ll);
                    const uint32_t vfirst = vchunk > (uint32_t)kNS ? vchunk - kNS : 0u;
                    for (uint32_t c = vfirst; c < vchunk; ++c)
                        mbar_wait(&ms->vfull[c % kMaxSlots], (c / kMaxSlots) & 1, 200000000ll);
                    if (q_loads > 0) mbar_wait(&ms->q_full, (q_loads - 1) & 1, 200000000ll);
                }
            }
        } else if (warp == 1) {
            // ============================================================ MMA issuer
            // The whole warp goes through the loop, one elected lane issues: addresses and descriptors
            // are then the warp's, in uniform registers (from one lane's registers an MMA took as long to
            // issue as to run twice).
            const bool leader = elect_one();
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool w = mbar_wait(bar, parity);
                ok = __all_sync(0xffffffffu, w);
                return ok;
            };
            if (rank != 0) {
                // the pair's second CTA: tells the first one what has landed here
                Cursor qk;
                qk.start(W, start, pass);
                uint32_t n = chunks0;
                while (ok) {
                    qk.step(W);
                    if (!qk.live) break;
                    if (qk.first()) {
                        if (!wait(&ms->q_full, qk.serial & 1)) break;
                        if (leader) mbar_arrive_at(cluster_addr(&ms->q_full, 0));
                    }
#pragma unroll 1
                    for (int c = 0; c < kChunks; ++c, ++n) {
                        if (!wait(&ms->kfull[n % kMaxSlots], (n / kMaxSlots) & 1) || __any_sync(0xffffffffu, aborted(ms))) {
                            ok = false;
                            break;
                        }
                        if (leader) mbar_arrive_at(cluster_addr(&ms->kfull[n % kMaxSlots], 0));
                        __syncwarp();
                    }
                }
                if (!ok) set_abort(ms, a.status);
            } else {
                constexpr uint32_t M = PAIR ? 256 : 128, kNv = PAIR ? D : 128;  // PV's N
                constexpr uint32_t id_qk = idesc_f16(M, 128, BF16 ? 1u : 0u, 0, 0);
                constexpr uint32_t id_pv = idesc_f16(M, kNv, PV16 ? 1u : 0u, 0, 1);
                constexpr uint64_t hi_k = desc_hi(16, 1024, kLayoutSwizzle128);
                constexpr uint64_t hi_v = desc_hi(8192, 1024, kLayoutSwizzle128);  // 2nd 64-dim box at +8 KB
                const uint32_t aQ = smem_u32(sQ), aS = smem_u32(sSlots);
                uint32_t slot = ring0 % kNS, jq = tiles0;   // ring position; tiles whose QK is issued
                uint32_t kn = chunks0, vn = chunks0;        // chunks of K and of V so far
                uint32_t first_bits = 0;        // bit k: the k-th last QK issued opened a piece
                auto commit = [&](uint64_t* bar) {
                    if constexpr (PAIR) mma_commit_pair(bar);
                    else mma_commit(bar);
                };
                auto advance = [&]() {
                    if (++slot == (uint32_t)kNS) slot = 0;
                };
                Cursor qk;
                qk.start(W, start, pass);
                // S(jq) = Q . K(jq)^T.  Its buffer held P(jq - 2), whose PV has been issued before
                // (MMAs of one thread run in order).
                auto next_qk = [&]() {
                    qk.step(W);
                    if (!qk.live) return;
                    if (qk.first()) {
                        if (!wait(&ms->q_full, qk.serial & 1)) return;
                    }
                    const uint32_t dS = tmem + (jq & 1) * 128;
#pragma unroll 1
                    for (int c = 0; c < kChunks; ++c) {
                        if (!wait(&ms->kfull[kn % kMaxSlots], (kn / kMaxSlots) & 1)) return;
                        tc_fence_after();
                        if (leader) {
                            const uint32_t at = aS + slot * kSlotBytes;
                            if constexpr (PAIR) {
#pragma unroll
                                for (int k = 0; k < D / 16; ++k)
                                    mma_f16_ss_pair(dS, make_desc(hi_k, aQ + k / 4 * kChunkBytes + k % 4 * 32),
                                                    make_desc(hi_k, at + k / 4 * 8192 + k % 4 * 32), id_qk, k != 0);
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_f16_ss(dS, make_desc(hi_k, aQ + c * kChunkBytes + k * 32), make_desc(hi_k, at + k * 32),
                                               id_qk, (c | k) != 0);
                            }
                            commit(&ms->empty[slot]);
                        }
                        __syncwarp();
                        ++kn;
                        advance();
                    }
                    if (leader) {
                        commit(&ms->s_full[jq & 1]);
                        if (qk.last()) commit(&ms->q_empty);
                    }
                    __syncwarp();
                    first_bits = (first_bits << 1) | (qk.first() ? 1u : 0u);
                    ++jq;
                };
                next_qk();
                if (ok && n_tiles > 1) next_qk();
                for (uint32_t j = tiles0; ok && j < tiles0 + n_tiles; ++j) {
                    if (__any_sync(0xffffffffu, aborted(ms))) break;
                    // O += P(j) . V(j) once the softmax has written P(j); P's columns of a page begin
                    // where S's did
                    if (!wait(&ms->p_full[j & 1], (j >> 1) & 1)) break;
                    const uint32_t more = ((first_bits >> (jq - 1 - j)) & 1u) ^ 1u, aP = tmem + (j & 1) * 128;
#pragma unroll 1
                    for (int c = 0; c < kChunks; ++c) {
                        if (!wait(&ms->vready[vn % kMaxSlots], (vn / kMaxSlots) & 1)) break;
                        tc_fence_after();
                        if (leader) {
                            const uint32_t at = aS + slot * kSlotBytes, dO = tmem + L::kColO;
                            if constexpr (PAIR) {
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    mma_f16_ts_pair(dO, aP + 64 * (k / 4) + 8 * (k % 4),
                                                    make_desc(hi_v, at + k / 4 * kPageBytes + k % 4 * 2048), id_pv,
                                                    k == 0 ? more : 1u);
                            } else {
                                // chunk c: output dims 128 (c >> 1) .., keys 64 (c & 1) ..
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_f16_ts(dO + 128 * (c >> 1), aP + 64 * (c & 1) + 8 * k, make_desc(hi_v, at + k * 2048),
                                               id_pv, (c & 1) == 0 && k == 0 ? more : 1u);
                            }
                            commit(&ms->empty[slot]);
                        }
                        __syncwarp();
                        ++vn;
                        advance();
                    }
                    if (!ok) break;
                    if (leader) commit(&ms->pv_done[j & 1]);
                    __syncwarp();
                    if (j + 2 < tiles0 + n_tiles) next_qk();
                }
                if (!ok || __any_sync(0xffffffffu, aborted(ms))) {
                    set_abort(ms, a.status);
                    if (leader) commit(&ms->drain);  // every MMA issued so far has finished before TMEM is freed
                    mbar_wait(&ms->drain, 0, 200000000ll);
                }
            }
            __syncwarp();
        } else if (warp < 4) {
            // ============================================================ V operand (warps 2, 3)
            // Each V chunk, once landed: bf16 -> fp16 in place where PV runs on fp16, zeros in the
            // rows of keys that no row sees (past a sequence's end, past the tree's nodes: arbitrary
            // data, and 0 * NaN would poison every row), and zeros in place of values that are not finite
            // in pages that some rows see and others do not: trees, and own pages of a block of several
            // sequences.  Their nodes and sequences are noted, and the epilogue makes the rows that see
            // them NaN.  Then vready.  Thread ct owns 16-byte units ct + 64 i of a chunk; unit u
            // holds 8 dims of key (u % 512) / 8 (each 8 KB box is [64 keys][128 B]; the swizzle
            // permutes units only within a key's row).
            const int ct = tid - 64;  // 0 .. 63
            Cursor cur;
            cur.start(W, start, pass);
            int word_cur = 0, word_next = 0;  // pages of 16 tiles, one to a lane
            uint32_t j = 0;  // of this pass
            bool ok = true;
            while (ok) {
                cur.step(W);
                if (!cur.live) break;
                const int rel = cur.t - cur.pc.ta;
                if ((rel & 15) == 0) word_cur = word_next;
                if (rel == 0 || (rel & 15) == 8) {
                    word_next = page_word(page_at(W, cur.pc, 2 * (cur.t + (rel == 0 ? 0 : 8)) + lane));
                    if (rel == 0) word_cur = word_next;
                }
                // ring position of V(j)'s first chunk: the K operands before it
                // (K(0) .. K(j+1), or .. K(j) for the last tile) and V(0) .. V(j-1)
                const uint32_t vbase = ring0 + ((j + 1 < n_tiles ? j + 2 : j + 1) + j) * kChunks;
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    const uint32_t vn = chunks0 + j * kChunks + c;
                    // the pages in the chunk's two 8 KB boxes: one page twice, or both
                    constexpr bool kBoth = PAIR;
                    const int page = kBoth ? 0 : c & 1;
                    const int word0 = __shfl_sync(0xffffffffu, word_cur, 2 * (rel & 15) + page);
                    const int word1 = kBoth ? __shfl_sync(0xffffffffu, word_cur, 2 * (rel & 15) + 1) : word0;
                    const bool landed = mbar_wait(&ms->vfull[vn % kMaxSlots], (vn / kMaxSlots) & 1);
                    if (!__all_sync(0xffffffffu, landed) || aborted(ms)) {
                        ok = false;
                        break;
                    }
                    uint4* base = reinterpret_cast<uint4*>(sSlots + ((vbase + c) % kNS) * kSlotBytes);
                    // pages that not all rows see
                    auto look = [&](int word) { return (word & 0x80) || (pass > 0 && (word >> 8) > 0 && cur.pc.seqs > 1); };
                    // (nothing to change)
                    const bool whole = (word0 & 0xff) == kPage && (word1 & 0xff) == kPage && !look(word0) && !look(word1);
                    constexpr int kUnits = kSlotBytes / 16 / (32 * kConvWarps);  // of a thread
                    constexpr int kBatch = 4;                                      // loads in flight
                    if (kConvert || !whole) {
#pragma unroll 1
                        for (int u0 = 0; u0 < kUnits; u0 += kBatch) {
                            // (a batch lies in one box)
                            const int word = u0 < kUnits / 2 ? word0 : word1, keys = word & 0x7f;
                            const bool looked = look(word);
                            uint4 x[kBatch];
                            bool on[kBatch];
#pragma unroll
                            for (int k = 0; k < kBatch; ++k) {
                                const int u = ct + 32 * kConvWarps * (u0 + k), key = (u & 511) >> 3;
                                on[k] = key < keys;
                                x[k] = on[k] ? base[u] : make_uint4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int k = 0; k < kBatch; ++k) {
                                const int u = ct + 32 * kConvWarps * (u0 + k);
                                if (looked && not_finite<BF16, kConvert>(x[k])) {
                                    const int owner = (word >> 8) - 1;
                                    const int at = word & 0x80 ? owner * kPage + ((u & 511) >> 3) : kNodeWords * 32 + owner;
                                    uint32_t* to = &ms->vbad[cur.serial % kBadSets][at >> 5];
                                    const uint32_t bit = 1u << (at & 31);
                                    if (*reinterpret_cast<volatile uint32_t*>(to) & bit) {
                                        // (noted, in a pair by someone who tells the other CTA too)
                                    } else if constexpr (PAIR) {  // its other dims, and other rows, are the other CTA's
                                        or_at(cluster_addr(to, 0), bit);
                                        or_at(cluster_addr(to, 1), bit);
                                        fence_cluster();
                                    } else {
                                        atomicOr(to, bit);
                                    }
                                    x[k] = make_uint4(0, 0, 0, 0);
                                    on[k] = false;
                                }
                                if constexpr (kConvert) {
                                    x[k].x = bf16x2_to_f16x2(x[k].x);
                                    x[k].y = bf16x2_to_f16x2(x[k].y);
                                    x[k].z = bf16x2_to_f16x2(x[k].z);
                                    x[k].w = bf16x2_to_f16x2(x[k].w);
                                }
                                if (kConvert || !on[k]) base[u] = x[k];
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (PAIR) mbar_arrive_at(cluster_addr(&ms->vready[vn % kMaxSlots], 0));
                        else mbar_arrive(&ms->vready[vn % kMaxSlots]);
                    }
                }
                ++j;
            }
            if (!ok) set_abort(ms, a.status);
        } else {
            // ============================================================ softmax + epilogue
            // Thread: row `row` (its TMEM lane), page `half` of every tile.
            const int half = (warp - 4) >> 2;
            const int row = (warp & 3) * 32 + lane;
            const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);  // the warp's lanes
            const float sl2 = W.scale_log2;
            uint32_t j = tiles0;
            bool bad = false;  // warp-uniform at every tcgen05 load / store below
            // bounded wait whose outcome all lanes of the warp agree on
            auto wait_all = [&](uint64_t* bar, uint32_t parity) {
                const bool w = mbar_wait(bar, parity);
                return __all_sync(0xffffffffu, w);
            };
            Cursor cur;
            cur.start(W, start, pass);
            while (!bad) {
                cur.next_piece(W);
                if (!cur.live) break;
                const Piece& blk = cur.pc;
                const int first_nodes = d.half(cur.pc.kind()), before = (int)rank * first_nodes;  // the block's nodes in the pair's first CTA
                const bool mine = row < min(first_nodes, blk.nodes - before) * d.G;
                const int node = blk.node0 + (mine ? before + row / d.G : 0);
                const int b = node / d.N, i = node - b * d.N;
                // (rows past the block's own go along with what all rows see, so that their warp needs no masks)
                const int seq = mine || blk.seqs == 1 ? b - blk.b0 : -2;
                const uint64_t anc = __ldg(a.anc_mask + node) & low_bits(d.N);
                if (mine && half == 0 && !((anc >> i) & 1u)) atomicOr(a.status, LUCETREE_DEV_BAD_NODE);
                float neg_m = INFINITY;  // the shift, negated: none yet
                float l = 0.f;           // my page's part of the row's sum
                int word_cur = 0, word_next = 0;  // my page of 32 tiles, one to a lane
#pragma unroll 1
                for (int t = cur.pc.ta; t < cur.pc.te; ++t) {
                    const int rel = t - cur.pc.ta;
                    const bool first = rel == 0;
                    if ((rel & 31) == 0) word_cur = word_next;
                    if (first || (rel & 31) == 16) {
                        word_next = page_word(page_at(W, cur.pc, 2 * (t + (first ? 0 : 16) + lane) + half));
                        if (first) word_cur = word_next;
                    }
                    const int word = __shfl_sync(0xffffffffu, word_cur, rel & 31);
                    const int owner = (word >> 8) - 1;
                    uint64_t vis = low_bits(word & 0x7f);
                    if (word & 0x80) {
                        const int at = seq * d.N - owner * kPage;  // my tree's first node in the page
                        vis = at >= kPage || at <= -kPage ? 0 : at >= 0 ? anc << at : anc >> -at;
                    } else if (owner >= 0 && owner != seq) {
                        vis = 0;
                    }
                    const bool plain = __all_sync(0xffffffffu, vis == ~0ull);
                    const bool none = __all_sync(0xffffffffu, vis == 0);

                    if (!wait_all(&ms->s_full[j & 1], (j >> 1) & 1)) bad = true;
                    if (!bad) tc_fence_after();
                    const uint32_t ts = tl + (j & 1) * 128 + half * 64;
                    uint32_t x[64];  // scores in units of log2; masked ones -infinity
                    float top = -INFINITY;
                    if (!bad && !none) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld16(ts + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&x[16 * c]));
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_wait_ld_regs16(*reinterpret_cast<uint32_t(*)[16]>(&x[16 * c]));
                        const uint64_t scale = pack2(sl2, sl2);
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float2 y = unpack2(mul2(pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), scale));
                            x[2 * k] = __float_as_uint(y.x);
                            x[2 * k + 1] = __float_as_uint(y.y);
                        }
                        if (!plain) {
#pragma unroll
                            for (int k = 0; k < 64; ++k)
                                if (!((vis >> k) & 1u)) x[k] = 0xFF800000u;
                        }
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int k = 0; k < 64; ++k) m4[k & 3] = fmaxf(m4[k & 3], __uint_as_float(x[k]));
                        top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    }
                    // one barrier decides whether shifts have to move (a row without one has neg_m = infinity);
                    // rows past the block's own have no say, or what lies there would decide the others' roundings
                    const bool bad_now = bad || aborted(ms);
                    if (bar_sync_or(1, kSoftmaxThreads, bad_now || first || (mine && top + neg_m > kTau))) {
                        ms->xchg[half][row] = top;  // for the row's other page
                        if (bar_sync_or(1, kSoftmaxThreads, bad_now)) {
                            bad = true;
                            break;
                        }
                        const float mo = -neg_m, mn = fmaxf(mo, fmaxf(top, ms->xchg[half ^ 1][row]));
                        // (the shift of a row that has seen no key stays -infinity: its sum is 0)
                        const float alpha = mn > mo ? ex2(mo - mn) : 1.f;
                        neg_m = -mn;
                        l = alpha > 0.f || l != l ? l * alpha : 0.f;  // (NaN stays: a score was NaN, though no shift tells)
                        if (!first) {
                            // the O row so far moves with its shift, once PV(j-1) has finished adding to it:
                            // each warpgroup half of the dims (a warp that timed out skips its TMEM
                            // accesses but keeps to the barriers)
                            if (!wait_all(&ms->pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1)) bad = true;
                            if (!bad) tc_fence_after();
                            if (!bad && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                                for (int c = 0; c < D / 32; ++c) {
                                    uint32_t r[16];
                                    const uint32_t at = tl + L::kColO + half * (D / 2) + 16 * c;
                                    tmem_ld16(at, r);
                                    tmem_wait_ld_regs16(r);
#pragma unroll
                                    for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha);
                                    tmem_st16(at, r);
                                }
                                tmem_wait_st();
                            }
                        }
                        // (nobody overwrites the exchanged maxima before everybody has read them)
                        if (bar_sync_or(1, kSoftmaxThreads, bad)) {
                            bad = true;
                            break;
                        }
                    }
                    // P = 2^(x - m) as 16-bit pairs, over S: [row][32 columns of two keys each] where my
                    // page's S began
                    uint32_t ph[32];
                    if (none) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) ph[k] = 0;
                    } else {
                        const float shift = neg_m == INFINITY ? 0.f : neg_m;  // (no key yet: every x is -infinity)
                        const uint64_t m2 = pack2(shift, shift);
                        uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float2 y = unpack2(add2(pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), m2));
                            const float p0 = ex2(y.x), p1 = ex2(y.y);
                            acc[k & 3] = add2(acc[k & 3], pack2(p0, p1));
                            ph[k] = PV16 ? pack_bf162(p0, p1) : pack_half2(p0, p1);
                        }
                        const float2 s = unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
                        l += s.x + s.y;
                    }
                    tmem_st16(ts, *reinterpret_cast<uint32_t(*)[16]>(&ph[0]));
                    tmem_st16(ts + 16, *reinterpret_cast<uint32_t(*)[16]>(&ph[16]));
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (PAIR) mbar_arrive_at(cluster_addr(&ms->p_full[j & 1], 0));
                        else mbar_arrive(&ms->p_full[j & 1]);
                    }
                    ++j;
                }
                if (bad) break;

                // ---------------------------------------------------------- epilogue
                ms->xchg[half][row] = l;
                const Piece& done = cur.pc;
                const bool got = mbar_wait(&ms->pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1);
                if (bar_sync_or(1, kSoftmaxThreads, !got || aborted(ms))) {
                    bad = true;
                    break;
                }
                tc_fence_after();
                l += ms->xchg[half ^ 1][row];
                const uint32_t* vb = ms->vbad[cur.serial % kBadSets];
                uint32_t any = 0;
#pragma unroll
                for (int k = 0; k < kBadWords; ++k) any |= vb[k];
                if (__builtin_expect(any != 0, 0) && mine) {
                    // bits seq * N .. + N - 1
                    const int at = seq * d.N, w = at >> 5, s = at & 31;
                    const uint64_t lo = (uint64_t)vb[w] | (uint64_t)(w + 1 < kNodeWords ? vb[w + 1] : 0) << 32;
                    const uint64_t hi = w + 2 < kNodeWords ? vb[w + 2] : 0;
                    const bool own = (vb[kNodeWords + (seq >> 5)] >> (seq & 31)) & 1u;
                    const uint64_t bits = s ? lo >> s | hi << (64 - s) : lo;
                    if ((bits & anc) != 0 || own) l = __int_as_float(0x7FC00000);
                }
                const bool whole = done.slot < 0;
                // rows of the output, or of the partial sums: mine, and the four of my lane's group of four
                const int my_row = whole ? node * d.Hq + done.g * d.G + row % d.G : done.slot + before * d.G + row;
                const int row4 = row & ~3, rows = min(first_nodes, done.nodes - before) * d.G;
                int to_row[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) to_row[k] = __shfl_sync(0xffffffffu, my_row, (lane & 28) + k);
                const float inv = !whole ? 1.f : l != 0.f ? 1.f / l : 0.f;  // (0: no key; NaN makes the row NaN)
                if (mine && half == 0) {
                    if (!whole) {
                        float* s = W.ws + partial_rows(d) * D + my_row;
                        s[0] = -neg_m;
                        s[partial_rows(d)] = l;
                    } else if (a.lse) {
                        a.lse[my_row] = l != 0.f ? (log2f(l) - neg_m) * kLn2 : -INFINITY;
                    }
                }
                const bool out16 = whole && (PV16 || W.out_dtype != LUCETREE_F32);
                float zero = 0.f;  // NaN: my row holds a value that is not finite
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[16];
                    const int x = half * (D / 2) + 16 * c;
                    tmem_ld16(tl + L::kColO + x, r);
                    tmem_wait_ld_regs16(r);
                    if ((warp & 3) * 32 >= rows) continue;  // (the whole warp)
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        zero = fmaf(__uint_as_float(r[k]), 0.f, zero);
                        r[k] = __float_as_uint(__uint_as_float(r[k]) * inv);
                    }
                    // Lanes of a group of four exchange their columns, so that each of them has a quarter of
                    // all four rows and a store covers 64 bytes of a row (a lane to a row, its 16 bytes apart
                    // from all others, a piece's rows took 6,000 to 14,000 cycles; 16 sequences at budget
                    // 22 under 4,096 tokens 46 us instead of 41.5, four sequences 12.2 instead of 12.8).
                    if (out16) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float o0 = __uint_as_float(r[2 * k]), o1 = __uint_as_float(r[2 * k + 1]);
                            w[k] = PV16 ? pack_bf162(o0, o1) : pack_half2(o0, o1);
                        }
                        turn4<2>(w, lane);
                        uint16_t* const to = reinterpret_cast<uint16_t*>(W.out) + x + 4 * (lane & 3);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (row4 + k < rows)
                                *reinterpret_cast<uint2*>(to + (size_t)to_row[k] * D) = make_uint2(w[2 * k], w[2 * k + 1]);
                    } else {
                        turn4<4>(r, lane);
                        float* const to = (whole ? reinterpret_cast<float*>(W.out) : W.ws) + x + 4 * (lane & 3);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (row4 + k < rows)
                                *reinterpret_cast<uint4*>(to + (size_t)to_row[k] * D) =
                                    make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
                    }
                }
                if (mine && !(zero + l == l)) {
                    if (whole) atomicOr(a.status, LUCETREE_DEV_NONFINITE);
                    if (done.seqs > 1 && zero != zero) {
                        if constexpr (PAIR) {
                            or_at(cluster_addr(&ms->again, 0), 1u);
                            or_at(cluster_addr(&ms->again, 1), 1u);
                        } else {
                            ms->again = 1;
                        }
                    }
                }
                tc_fence_before();
                // (the barrier also says that the piece's O and values in shared memory are no longer read)
                if (bar_sync_or(1, kSoftmaxThreads, mine && zero != zero)) {
                    // All of such a row and its lse are NaN, as where the second pass notes its sequence:
                    // which of the two happens depends on what else is in the block.
                    ms->xchg[half][row] = zero;
                    bar_sync(1, kSoftmaxThreads);
                    const float both = zero + ms->xchg[half ^ 1][row];
                    if (mine && both != both) {
                        if (half == 0 && !whole) W.ws[partial_rows(d) * (D + 1) + my_row] = both;
                        if (half == 0 && whole && a.lse) a.lse[my_row] = both;
                        if (whole) {
                            const int bytes = out16 ? 2 : 4;
                            uint4* const to = reinterpret_cast<uint4*>(reinterpret_cast<char*>(W.out) +
                                                                       ((size_t)my_row * D + half * (D / 2)) * bytes);
                            const uint32_t nan = 0x7FFFFFFFu;  // (as two 16-bit numbers too)
#pragma unroll 1
                            for (int c = 0; c < D / 2 * bytes / 16; ++c) to[c] = make_uint4(nan, nan, nan, nan);
                        }
                    }
                }
                if (any && half == 0 && row < kBadWords) ms->vbad[cur.serial % kBadSets][row] = 0;
            }
            if (bad) set_abort(ms, a.status);
        }

        tc_fence_before();
        __syncthreads();
        if constexpr (PAIR) {
            // (both CTAs go on, or neither)
            if (tid < 2 && aborted(ms)) or_at(cluster_addr(&ms->again, tid), 2u);
            __syncwarp();
            cluster_sync();  // the other CTA's waits are over
            // (after an abort the first CTA's MMAs are drained, see above: the second one's notice of it)
            if (tid < 32 && rank != 0 && (*(volatile int*)&ms->again & 2)) mbar_wait(&ms->drain, 0, 200000000ll);
        }
        tc_fence_after();
        if (*(volatile int*)&ms->pass > 0 || *(volatile int*)&ms->again != 1 || (!PAIR && aborted(ms))) break;
        __syncthreads();
        if (tid == 0) ms->pass = 1;
        __syncthreads();
        start = W.plan.cta[blockIdx.x / d.pair];  // (again, so that no thread has to keep it)
    }

    // ---------------------------------------------------------------- teardown
    teardown();
}

struct Maps {
    CUtensorMap k, v, q, qown, qlarge, kt, vt;
};

template <int D, bool BF16, bool PV16, bool PAIR>
cudaError_t launch_pairs(const Maps& m, const Launch& W, cudaStream_t stream) {
    auto kern = shared_tc_kernel<D, BF16, PV16, PAIR>;
    constexpr int bytes = Lay<D, PAIR>::kBytes;
    static SmemLimitSeen seen;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), bytes, seen);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(W.d.C * W.d.pair);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, m.k, m.v, m.q, m.qown, m.qlarge, m.kt, m.vt, W);
}

template <int D, bool BF16, bool PV16>
cudaError_t launch_one(const Maps& m, const Launch& W, cudaStream_t stream) {
    return W.d.pair == 2 ? launch_pairs<D, BF16, PV16, true>(m, W, stream) : launch_pairs<D, BF16, PV16, false>(m, W, stream);
}

cudaError_t launch_bf16_256(const Maps&, const Launch&, cudaStream_t);
cudaError_t launch_bf16_128(const Maps&, const Launch&, cudaStream_t);
cudaError_t launch_bf16_256_out16(const Maps&, const Launch&, cudaStream_t);
cudaError_t launch_bf16_128_out16(const Maps&, const Launch&, cudaStream_t);
cudaError_t launch_f16_256(const Maps&, const Launch&, cudaStream_t);
cudaError_t launch_f16_128(const Maps&, const Launch&, cudaStream_t);

}  // namespace shr
}  // namespace lucetree
