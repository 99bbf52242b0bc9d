// rope.cu -- rotary positions: lucetree_rope (the tree's queries and keys) and
// lucetree_append_kv (new tokens' keys and values into the paged cache, rotated
// and, where the pools hold codes, quantised on the way).
//
// A pair (x, y) of rotated dims at position p becomes m (x cos a - y sin a,
// x sin a + y cos a), a = p f_i.  A step is f_i / 2 pi in units of 2^-64 turns, so
// p * step mod 2^64 is the angle's fraction of a turn for any position (in fp32, p f_i
// is off by 2^-24 p f_i: 0.008 at p = 131,072), and what is left of it after the nearest
// quarter turn is an integer too.  The cosine and sine are off by less than a step of
// their own in fp32 (turn), which decides how many of the keys that are stored as
// codes land on the other side of a border: of 16.8 million E4M3 codes 13 differ from those
// of 64 bits (18 with cosines that are rounded from 64 bits and no fused products; 31 with
// sincospi of the fraction in fp32, which took 1 % less time).
//
// Bound by HBM: every element is read once and written once.  A block takes a few
// tokens: their positions and cosines go to shared memory once (one a thread and
// token instead of eight in each thread that rotates), and the threads go through
// the tokens' heads, 16 dims to a thread (two 16-byte vectors, which hold both parts of
// its 8 pairs), the next two heads' vectors in flight.  The first ones are asked for
// before the positions are known, so that a single token waits for three loads in a row
// (start, page, row) and not for four.  Measured with 24 query and 4 KV heads of 256
// dims in bf16: 24,576 prompt tokens into the cache 130 to 136 us (5.9 to 6.2 TB/s, 88 to
// 93 % of a copy's rate), 6,144 into E4M3 / int8 pools 38 us (4.9 TB/s), 704 tree nodes
// 6.7 us a call back to back, 7.5 in a replayed graph over 280 MB of inputs (3.4, 3.1 TB/s; the
// launch and the chain of loads are 2 us of it: 8 nodes take 2.1).
#include <math.h>

#include "e4m3.cuh"
#include "internal.cuh"
#include "rope.h"

namespace lucetree {

namespace {

constexpr int kBlock = 256;

enum Mode {
    kHalf,      // dims i and i + r/2, r/2 a multiple of 8: a thread's two vectors
    kPairs,     // dims 2i and 2i + 1
    kHalfOdd,   // dims i and i + r/2 otherwise: the partner's elements one by one
};
enum KeyTo { kKeyRows, kKeyPages, kKeyE4M3 };
enum ValueTo { kValueSame, kValueInt8, kValueInt4 };

struct RopeLaunch {
    const char* src[3];   // k, v, q
    long long stride[3];  // bytes from one token to the next
    char* out[3];         // k, v: contiguous rows or pools; q: contiguous rows
    int H[3];             // heads
    int D, T;             // dims, tokens
    int slots, groups, tokens;  // of a block: 16-dim slots of a head, heads taken at once, tokens
    const uint64_t* steps;
    int pairs;            // rotated pairs, 0: none
    float magnitude;
    uint32_t* status;
    // positions of a tree's nodes
    int N;
    const int32_t* ctx_len;
    const uint64_t* anc;
    const int32_t* positions;
    // pages
    int B, max_pages, num_pages;
    const int32_t* start;
    const int32_t* table;
    int32_t* ctx_out;
    uint8_t* exps[2];     // of k, v codes
    int length_blocks;    // the first ones, which write the lengths
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = to_f32<T>(e[k]);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()), pack2(f[4], f[5], T()), pack2(f[6], f[7], T()));
}

// Cosine and sine of `part` 2^-64 turns, times m.  After the nearest quarter turn |x| <= pi / 4, 31 bits of it from
// its first one on (a slow pair's may lie in the lowest) in two floats, and the Taylor series to x^9 and x^10 are off by less than 2^-28;
// the leading terms (2 pi r, and 1 - (2 pi r)^2 / 2) are kept as sums of two floats: cosines and sines are off by 0.81 of
// their own steps at most, down to angles of 2^-64 of a turn (eight million angles, on the CPU).
__device__ __forceinline__ void turn(uint64_t part, float m, float& c, float& s) {
    const uint32_t q = (uint32_t)((part + (1ull << 61)) >> 62);
    const long long rest = (long long)(part - ((uint64_t)q << 62));  // 2^-64 turns, [-2^61, 2^61]
    const int up = __clzll(rest ^ (rest >> 63)) - 1;  // its top 31 bits and sign (64-bit conversions take longer)
    const int bits = (int)((rest << up) >> 32);
    const float unit = __int_as_float((127 - 32 - up) << 23), top = (float)bits;
    const float r = top * unit, rl = (float)(bits - (int)top) * unit;  // turns, in two parts
    // (products whose rounding is made good are kept from being fused into a sum)
    const float t = __fmul_rn(r, r), tl = fmaf(2.f * r, rl, fmaf(r, r, -t));
    // sin: (2 pi)^k / k!
    const float sh = __fmul_rn(r, 6.2831855f);
    float sl = fmaf(r, 6.2831855f, -sh);
    sl = fmaf(r, -1.7484556e-7f, sl);
    sl = fmaf(rl, 6.2831855f, sl);
    sl = fmaf(r * t, fmaf(t, fmaf(t, fmaf(t, 42.058693f, -76.70586f), 81.60525f), -41.341702f), sl);
    // cos
    const float u = __fmul_rn(t, -19.739208f);
    float cl = fmaf(t, -19.739208f, -u);
    cl = fmaf(t, -5.8074317e-7f, cl);
    cl = fmaf(tl, -19.739208f, cl);
    cl = fmaf(t * t, fmaf(t, fmaf(t, fmaf(t, -26.426256f, 60.24464f), -85.45682f), 64.93939f), cl);
    const float ch = __fadd_rn(1.f, u);
    cl += __fadd_rn(__fsub_rn(1.f, ch), u);
    // a sum of two floats times m, rounded once
    auto times_m = [&](float hi, float lo) {
        const float x = __fmul_rn(hi, m);
        return x + fmaf(lo, m, fmaf(hi, m, -x));
    };
    const float cx = times_m(ch, cl), sx = times_m(sh, sl);
    c = q & 1 ? sx : cx;
    s = q & 1 ? cx : sx;
    if (q == 1 || q == 2) c = -c;
    if (q & 2) s = -s;
}

// x such that max 2^x is at most `top` 2^e and above half of it (top in [0.5, 1); 0 for max = 0).
__device__ __forceinline__ int int_exponent(float m, float top, int e) {
    if (!(m > 0.f)) return 0;
    int ex;
    const float mant = frexpf(m, &ex);
    return mant <= top ? e - ex : e - 1 - ex;
}
// Times 2^p, p in [-127, 126], in two steps (2^-127 is no normal number).
__device__ __forceinline__ float times_pow2(float v, int p) {
    const int a = p / 2, b = p - a;
    return v * __int_as_float((127 + a) << 23) * __int_as_float((127 + b) << 23);
}
// Maximum of |f| over the 16 lanes that hold a row of 256.
__device__ __forceinline__ float row_max(const float* f) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(f[k]));
    const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(half, m, o));
    return m;
}

template <typename T, int MODE, int KT, int VT>
__global__ void __launch_bounds__(kBlock, 4) rope_kernel(const RopeLaunch R) {
    constexpr bool kPaged = KT != kKeyRows;
    extern __shared__ float4 s_turn[];     // cosines, then sines, of the block's tokens: [token][pair]
    __shared__ long long s_pos[kBlock];
    __shared__ long long s_row[kBlock];    // contiguous: the token; pages: its row in head 0 of its page; -2: no page, -1: no sequence
    __shared__ int s_seq[kBlock];
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();

    if (kPaged && (int)blockIdx.x < R.length_blocks) {
        // ------------------------------------------------ lengths, a warp to each sequence
        bool bad = false;
#pragma unroll 1
        for (int i = threadIdx.x; i <= R.B; i += blockDim.x) {
            const int a = R.start[i];
            bad |= a < 0 || a > R.T || (i < R.B && R.start[i + 1] < a);
        }
        bad = __syncthreads_or(bad);
        const int lane = threadIdx.x & 31, b = (int)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5);
        if (b == 0 && lane == 0 && bad) atomicOr(R.status, LUCETREE_DEV_BAD_ROW);
        if (b >= R.B) return;
        const int L = R.ctx_len[b];
        long long n = bad ? 0 : (long long)R.start[b + 1] - R.start[b];
        if (L < 0 || (long long)L > (long long)R.max_pages * kPage) {
            if (lane == 0) atomicOr(R.status, LUCETREE_DEV_BAD_CTX);
            n = 0;
        }
        if (n > 0) {
            const int c0 = L / kPage, c1 = (int)((L + n - 1) / kPage);
            int first = c1 + 1;  // the first column without a page
            for (int c = c0 + lane; c <= c1 && first > c1; c += 32) {
                const int page = c < R.max_pages ? R.table[(size_t)b * R.max_pages + c] : -1;
                if (page < 0 || page >= R.num_pages) first = c;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
            if (first <= c1) {
                n = max((long long)first * kPage - L, 0ll);
                if (lane == 0) atomicOr(R.status, LUCETREE_DEV_BAD_PAGE);
            }
        }
        if (lane == 0) R.ctx_out[b] = (int)(L + n);
        return;
    }

    const int slot = threadIdx.x % R.slots, group = threadIdx.x / R.slots;
    const int t0 = ((int)blockIdx.x - (kPaged ? R.length_blocks : 0)) * R.tokens;
    const int n = min(R.tokens, R.T - t0);
    const int heads = R.H[0] + R.H[1] + R.H[2];
    const int h2 = R.pairs;  // half of the rotated dims

    // first dims of the two vectors, and the pair of the first one's first element
    int da = 16 * slot, db = da + 8, pair = 8 * slot;
    if (MODE == kHalf && 8 * slot < h2) {
        da = 8 * slot;
        db = h2 + da;
    }
    // tensor (0 k, 1 v, 2 q) and head of number i of the token's heads
    auto which = [&](int& i) {
        int x = 0;
        if (i >= R.H[0]) {
            i -= R.H[0];
            x = 1;
            if (i >= R.H[1]) {
                i -= R.H[1];
                x = 2;
            }
        }
        return x;
    };
    // The heads of the block's tokens one after the other, every `groups`-th of them this thread's.
    struct Item {
        int t, i;
    };
    auto step_on = [&](Item& m, int by) {
        m.i += by;
        while (m.i >= heads) {
            m.i -= heads;
            ++m.t;
        }
    };
    auto load = [&](const Item& m, uint4 (&u)[2]) {
        if (m.t >= n) return;
        int i = m.i;
        const int x = which(i);
        const char* row = R.src[x] + (t0 + m.t) * R.stride[x] + (size_t)i * R.D * 2;
        const bool flat = MODE == kHalf && x == 1;  // v: its 16 dims lie together
        u[0] = *reinterpret_cast<const uint4*>(row + (flat ? 16 * slot : da) * 2);
        u[1] = *reinterpret_cast<const uint4*>(row + (flat ? 16 * slot + 8 : db) * 2);
    };
    // two heads in flight, while the positions are found already
    uint4 u0[2] = {}, u1[2] = {};
    Item now = {group < R.groups ? 0 : n, 0};
    step_on(now, group);
    Item ahead = now;
    load(ahead, u0);
    step_on(ahead, R.groups);
    load(ahead, u1);

    // ---------------------------------------------------- positions
    const int per = 8 * R.slots;  // pairs of a token
    const int tp = threadIdx.x % per;
    const uint64_t step = tp < h2 ? __ldg(R.steps + tp) : 0;
    if constexpr (kPaged) {
#pragma unroll 1
        for (int i = threadIdx.x; i < R.tokens; i += blockDim.x) s_seq[i] = -1;
        __syncthreads();
        bool bad = false;
#pragma unroll 1
        for (int b = threadIdx.x; b < R.B; b += blockDim.x) {
            const int a = R.start[b], z = R.start[b + 1], L = R.ctx_len[b];
            bad |= a < 0 || z < a || z > R.T;
            if (bad || L < 0 || (long long)L > (long long)R.max_pages * kPage) continue;
#pragma unroll 1
            for (int j = max(a, t0); j < min(z, t0 + R.tokens); ++j) {
                s_seq[j - t0] = b;
                s_pos[j - t0] = (long long)L + (j - a);
            }
        }
        bad = __syncthreads_or(bad);
#pragma unroll 1
        for (int i = threadIdx.x; i < R.tokens; i += blockDim.x) {
            const int b = bad ? -1 : s_seq[i];
            long long row = -1;
            if (b >= 0) {
                const long long pos = s_pos[i], c = pos / kPage;
                const int page = c < R.max_pages ? R.table[(size_t)b * R.max_pages + c] : -1;
                row = page >= 0 && page < R.num_pages ? (long long)page * R.H[0] * kPage + pos % kPage : -2;
            }
            s_row[i] = row;
        }
    } else {
#pragma unroll 1
        for (int i = threadIdx.x; i < R.tokens && t0 + i < R.T; i += blockDim.x) {
            const int at = t0 + i;
            long long pos;
            if (R.positions) {
                pos = R.positions[at];
            } else {
                const int b = at / R.N, node = at - b * R.N;
                int L = R.ctx_len[b];
                const uint64_t anc = R.anc[at] & (~0ull >> (64 - R.N));
                if (L < 0) {
                    atomicOr(R.status, LUCETREE_DEV_BAD_CTX);
                    L = 0;
                }
                if (!((anc >> node) & 1u)) atomicOr(R.status, LUCETREE_DEV_BAD_NODE);
                // (a mask without its own bit: no proper ancestors)
                pos = (long long)L + ((anc >> node) & 1u ? __popcll(anc) - 1 : 0);
            }
            s_pos[i] = pos;
        }
        __syncthreads();
    }

    // ---------------------------------------------------- cosines
    float* const s_cos = reinterpret_cast<float*>(s_turn);
    float* const s_sin = s_cos + R.tokens * per;
    if (tp < h2 || kBlock % per != 0)
#pragma unroll 1
        for (int i = threadIdx.x; i < R.tokens * per; i += kBlock) {
            const int p = i % per;
            if (p >= h2) continue;
            const uint64_t part = (uint64_t)s_pos[i / per] * (p == tp ? step : __ldg(R.steps + p));
            turn(part, R.magnitude, s_cos[i], s_sin[i]);
        }
    __syncthreads();

#pragma unroll 1
    for (; now.t < n; step_on(now, R.groups)) {
        uint4 u[2] = {u0[0], u0[1]};
        u0[0] = u1[0];
        u0[1] = u1[1];
        step_on(ahead, R.groups);
        load(ahead, u1);
        int i = now.i;
        const int x = which(i), t = t0 + now.t;
        const long long row0 = kPaged ? s_row[now.t] : t;
        if (kPaged && (row0 == -1 || (x < 2 && row0 < 0))) continue;
        // row of the output: contiguous [token][head], or [page][head][slot]
        const bool paged = kPaged && x < 2;
        const long long row = paged ? row0 + (long long)i * kPage : (long long)t * R.H[x] + i;
        if (x == 1) {
            if constexpr (VT == kValueSame) {
                char* o = R.out[1] + row * R.D * 2 + slot * 32;
                *reinterpret_cast<uint4*>(o) = u[0];
                *reinterpret_cast<uint4*>(o + 16) = u[1];
            } else {
                float f[16];
                unpack8<T>(u[0], f);
                unpack8<T>(u[1], f + 8);
                const float m = row_max(f);
                const int p = VT == kValueInt8 ? int_exponent(m, 0.9921875f, 7) : int_exponent(m, 0.875f, 3);
                const int e = 127 - p;
                const bool in_range = m > 0.f && e >= 1 && e <= 254;
                uint32_t q[4] = {0, 0, 0, 0};
                if (in_range) {
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        const uint32_t code = (uint32_t)__float2int_rn(times_pow2(f[y], p));
                        if constexpr (VT == kValueInt8) q[y / 4] |= (code & 0xFFu) << (8 * (y % 4));
                        else q[y / 8] |= (code & 0xFu) << (4 * (y % 8));
                    }
                }
                if constexpr (VT == kValueInt8)
                    *reinterpret_cast<uint4*>(R.out[1] + row * 256 + slot * 16) = make_uint4(q[0], q[1], q[2], q[3]);
                else
                    *reinterpret_cast<uint2*>(R.out[1] + row * 128 + slot * 8) = make_uint2(q[0], q[1]);
                if (slot == 0) R.exps[1][row] = (uint8_t)(in_range ? e : 0);
            }
            continue;
        }
        float f[16];
        if constexpr (KT != kKeyE4M3) {
            // what is not rotated is copied as it is
            const bool still = MODE == kPairs ? pair >= h2 : MODE == kHalf ? 8 * slot >= h2 : 16 * slot >= 2 * h2;
            char* o = R.out[x] + row * R.D * 2;
            if (still) {
                *reinterpret_cast<uint4*>(o + da * 2) = u[0];
                *reinterpret_cast<uint4*>(o + db * 2) = u[1];
                continue;
            }
        }
        unpack8<T>(u[0], f);
        unpack8<T>(u[1], f + 8);
        const float* cs = s_cos + now.t * per + pair;  // (pairs past the rotated ones hold nothing)
        const float* sn = s_sin + now.t * per + pair;
        if constexpr (MODE == kHalf) {
            if (8 * slot < h2) {
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const float a = f[y], b = f[y + 8], c = cs[y], s = sn[y];
                    f[y] = a * c - b * s;
                    f[y + 8] = a * s + b * c;
                }
            }
        } else if constexpr (MODE == kPairs) {
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                if (pair + y >= h2) continue;
                const float a = f[2 * y], b = f[2 * y + 1], c = cs[y], s = sn[y];
                f[2 * y] = a * c - b * s;
                f[2 * y + 1] = a * s + b * c;
            }
        } else {
            const T* in = reinterpret_cast<const T*>(R.src[x] + t * R.stride[x]) + (size_t)i * R.D;
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                const int d = 16 * slot + y;
                if (d >= 2 * h2) continue;
                const float other = to_f32<T>(in[d < h2 ? d + h2 : d - h2]);
                const int p = d < h2 ? d : d - h2;
                const float c = s_cos[now.t * per + p], s = s_sin[now.t * per + p];
                f[y] = d < h2 ? f[y] * c - other * s : f[y] * c + other * s;
            }
        }
        if (KT == kKeyE4M3 && x == 0) {
            const float m = row_max(f);
            const int p = e4m3::scale_exponent(m), e = 127 - p;
            const bool in_range = m > 0.f && e >= 1 && e <= 254;
            uint32_t q[4] = {0, 0, 0, 0};
            if (in_range) {
#pragma unroll
                for (int y = 0; y < 16; y += 2)
                    q[y / 4] |= (uint32_t)e4m3::e4m3x2(times_pow2(f[y], p), times_pow2(f[y + 1], p)) << (8 * (y & 2));
            }
            char* o = R.out[0] + row * 256;
            *reinterpret_cast<uint2*>(o + da) = make_uint2(q[0], q[1]);
            *reinterpret_cast<uint2*>(o + db) = make_uint2(q[2], q[3]);
            if (slot == 0) R.exps[0][row] = (uint8_t)(in_range ? e : 0);
        } else {
            char* o = R.out[x] + row * R.D * 2;
            *reinterpret_cast<uint4*>(o + da * 2) = pack8<T>(f);
            *reinterpret_cast<uint4*>(o + db * 2) = pack8<T>(f + 8);
        }
    }
}

// Tokens of a block: as many as fill the card evenly, kWave blocks to an SM at once (as
// many as 64 registers a thread allow), kMost / slots of them at most.  24,576 tokens of
// 256 dims at up to 4 tokens a block: 132 us; 8: 136, 16: 137.  Three blocks an SM with
// 80 registers: 149.  Blocks of 128 threads: 134, and one decoded token of 16 sequences
// 3.4 us instead of 2.9.
constexpr int kWave = 4, kMost = 64;
int block_tokens(long long tokens, int slots, int sms) {
    const long long wave = (long long)sms * kWave, most = slots < kMost ? kMost / slots : 1;
    const long long waves = (tokens + wave * most - 1) / (wave * most);
    return (int)((tokens + waves * wave - 1) / (waves * wave));
}

template <typename T, int KT, int VT>
cudaError_t launch_mode(int layout, RopeLaunch& R, cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    R.slots = R.D / 16;
    R.groups = kBlock / R.slots;
    R.tokens = R.T > 0 ? block_tokens(R.T, R.slots, device_sm_count(dev)) : 1;
    R.length_blocks = KT == kKeyRows ? 0 : (R.B + kBlock / 32 - 1) / (kBlock / 32);
    const dim3 grid((int)(((long long)R.T + R.tokens - 1) / R.tokens) + R.length_blocks), block(kBlock);
    const size_t smem = sizeof(float) * 2 * R.tokens * 8 * R.slots;
    if (layout == LUCETREE_ROPE_PAIRS) return launch_pdl(rope_kernel<T, kPairs, KT, VT>, grid, block, smem, stream, R);
    if (R.pairs % 8 != 0) return launch_pdl(rope_kernel<T, kHalfOdd, KT, VT>, grid, block, smem, stream, R);
    return launch_pdl(rope_kernel<T, kHalf, KT, VT>, grid, block, smem, stream, R);
}

}  // namespace

cudaError_t launch_rope(const lucetree_rope_args& a, cudaStream_t stream) {
    RopeLaunch R = {};
    const void* in[3] = {a.k, a.v, a.q};
    void* out[3] = {a.k_out, a.v_out, a.q_out};
    const long long stride[3] = {a.k_stride, a.v_stride, a.q_stride};
    const int H[3] = {a.Hkv, a.v ? a.Hkv : 0, a.Hq};
    for (int x = 0; x < 3; ++x) {
        R.src[x] = reinterpret_cast<const char*>(in[x]);
        R.out[x] = reinterpret_cast<char*>(out[x]);
        R.stride[x] = 2 * stride[x];
        R.H[x] = H[x];
    }
    R.D = a.D;
    R.T = a.B * a.N;
    R.steps = a.steps;
    R.pairs = a.rot_dims / 2;
    R.magnitude = a.magnitude;
    R.status = a.status;
    R.N = a.N;
    R.ctx_len = a.ctx_len;
    R.anc = a.anc_mask;
    R.positions = a.positions;
    if (a.dtype == LUCETREE_BF16) return launch_mode<__nv_bfloat16, kKeyRows, kValueSame>(a.layout, R, stream);
    return launch_mode<__half, kKeyRows, kValueSame>(a.layout, R, stream);
}

cudaError_t launch_append_kv(const lucetree_append_args& a, cudaStream_t stream) {
    RopeLaunch R = {};
    const void* in[3] = {a.k, a.v, a.q};
    void* out[3] = {a.k_pool, a.v_pool, a.q_out};
    const long long stride[3] = {a.k_stride, a.v_stride, a.q_stride};
    const int H[3] = {a.Hkv, a.Hkv, a.q ? a.Hq : 0};
    for (int x = 0; x < 3; ++x) {
        R.src[x] = reinterpret_cast<const char*>(in[x]);
        R.out[x] = reinterpret_cast<char*>(out[x]);
        R.stride[x] = 2 * stride[x];
        R.H[x] = H[x];
    }
    R.D = a.D;
    R.T = a.rows;
    R.steps = a.steps;
    R.pairs = a.steps ? a.rot_dims / 2 : 0;
    R.magnitude = a.magnitude;
    R.status = a.status;
    R.B = a.B;
    R.max_pages = a.max_pages_per_seq;
    R.num_pages = a.num_pages;
    R.start = a.start;
    R.table = a.page_table;
    R.ctx_len = a.ctx_len_in;
    R.ctx_out = a.ctx_len_out;
    R.exps[0] = a.k_exp;
    R.exps[1] = a.v_exp;
    const int layout = a.steps ? a.layout : LUCETREE_ROPE_HALF;
    const bool bf16 = a.dtype == LUCETREE_BF16;
    using B16 = __nv_bfloat16;
    if (a.k_format == LUCETREE_K_E4M3) {
        if (a.v_format == LUCETREE_V_INT8) return launch_mode<B16, kKeyE4M3, kValueInt8>(layout, R, stream);
        if (a.v_format == LUCETREE_V_INT4) return launch_mode<B16, kKeyE4M3, kValueInt4>(layout, R, stream);
        return launch_mode<B16, kKeyE4M3, kValueSame>(layout, R, stream);
    }
    if (a.v_format == LUCETREE_V_INT8)
        return bf16 ? launch_mode<B16, kKeyPages, kValueInt8>(layout, R, stream)
                    : launch_mode<__half, kKeyPages, kValueInt8>(layout, R, stream);
    if (a.v_format == LUCETREE_V_INT4)
        return bf16 ? launch_mode<B16, kKeyPages, kValueInt4>(layout, R, stream)
                    : launch_mode<__half, kKeyPages, kValueInt4>(layout, R, stream);
    return bf16 ? launch_mode<B16, kKeyPages, kValueSame>(layout, R, stream)
                : launch_mode<__half, kKeyPages, kValueSame>(layout, R, stream);
}

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Bytes from the first row of a strided tensor to the end of its last one.
long long span_bytes(long long rows, long long stride, long long elems) {
    return rows > 0 ? 2 * ((rows - 1) * stride + elems) : 0;
}

struct Span {
    const void* at;
    long long bytes;
};

// Whether an output shares bytes with an input or another output.
template <int NO, int NI>
bool any_overlap(const Span (&out)[NO], const Span (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        if (!out[i].at) continue;
        for (int j = 0; j < NI; ++j)
            if (in[j].at && bytes_overlap(out[i].at, out[i].bytes, in[j].at, in[j].bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (out[j].at && bytes_overlap(out[i].at, out[i].bytes, out[j].at, out[j].bytes)) return true;
    }
    return false;
}

bool stride_ok(long long stride, long long elems) {
    return stride >= elems && stride % 8 == 0 && stride <= (1ll << 40);
}

}  // namespace

}  // namespace lucetree

using namespace lucetree;

extern "C" lucetree_status lucetree_rope(const lucetree_rope_args* a, void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    if (a->dtype != LUCETREE_F16 && a->dtype != LUCETREE_BF16) return LUCETREE_ERR_UNSUPPORTED;
    if (a->B <= 0 || a->N <= 0 || a->Hq <= 0 || a->Hkv <= 0 || a->D <= 0) return LUCETREE_ERR_INVALID_ARG;
    if (a->D % 16 != 0 || a->D > 1024) return LUCETREE_ERR_UNSUPPORTED;
    if (a->layout != LUCETREE_ROPE_HALF && a->layout != LUCETREE_ROPE_PAIRS) return LUCETREE_ERR_UNSUPPORTED;
    if (!a->q || !a->k || !a->steps || !a->q_out || !a->k_out || !a->status || (a->v != nullptr) != (a->v_out != nullptr))
        return LUCETREE_ERR_INVALID_ARG;
    if (a->rot_dims < 2 || a->rot_dims > a->D || a->rot_dims % 2 != 0 || !isfinite(a->magnitude))
        return LUCETREE_ERR_INVALID_ARG;
    if (!a->positions) {
        if (!a->ctx_len || !a->anc_mask) return LUCETREE_ERR_INVALID_ARG;
        if (a->N > LUCETREE_MAX_NODES) return LUCETREE_ERR_UNSUPPORTED;
    }
    const long long T = (long long)a->B * a->N, qe = (long long)a->Hq * a->D, ke = (long long)a->Hkv * a->D;
    if (T > 0x7fffff00ll || qe > 0x7fffffffll || ke > 0x7fffffffll || (long long)a->Hq + 2ll * a->Hkv > 0x3fffffffll)
        return LUCETREE_ERR_UNSUPPORTED;
    if (!stride_ok(a->q_stride, qe) || !stride_ok(a->k_stride, ke) || (a->v && !stride_ok(a->v_stride, ke)))
        return LUCETREE_ERR_INVALID_ARG;
    for (const void* p : {a->q, a->k, a->v, (const void*)a->q_out, (const void*)a->k_out, (const void*)a->v_out})
        if (!aligned(p, 16)) return LUCETREE_ERR_INVALID_ARG;
    const Span out[] = {{a->q_out, 2 * T * qe}, {a->k_out, 2 * T * ke}, {a->v_out, 2 * T * ke}};
    const bool given = a->positions != nullptr;
    const Span in[] = {{a->q, span_bytes(T, a->q_stride, qe)}, {a->k, span_bytes(T, a->k_stride, ke)},
                       {a->v, span_bytes(T, a->v_stride, ke)}, {a->steps, 4ll * a->rot_dims}, {a->positions, 4 * T},
                       {given ? nullptr : a->ctx_len, 4ll * a->B}, {given ? nullptr : a->anc_mask, 8 * T}};
    if (any_overlap(out, in)) return LUCETREE_ERR_INVALID_ARG;
    return launch_rope(*a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LUCETREE_OK : LUCETREE_ERR_CUDA;
}

extern "C" lucetree_status lucetree_append_kv(const lucetree_append_args* a, void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    if (a->dtype != LUCETREE_F16 && a->dtype != LUCETREE_BF16) return LUCETREE_ERR_UNSUPPORTED;
    if (a->page_size != LUCETREE_PAGE_SIZE) return LUCETREE_ERR_UNSUPPORTED;
    if (a->B <= 0 || a->rows < 0 || a->Hkv <= 0 || a->D <= 0 || a->num_pages <= 0 || a->max_pages_per_seq <= 0)
        return LUCETREE_ERR_INVALID_ARG;
    if (a->D % 16 != 0 || a->D > 1024) return LUCETREE_ERR_UNSUPPORTED;
    const bool kq = a->k_format == LUCETREE_K_E4M3, vq = a->v_format == LUCETREE_V_INT8 || a->v_format == LUCETREE_V_INT4;
    if ((!kq && a->k_format != LUCETREE_K_SAME) || (!vq && a->v_format != LUCETREE_V_SAME)) return LUCETREE_ERR_UNSUPPORTED;
    if ((kq && (a->dtype != LUCETREE_BF16 || a->D != 256)) || (vq && a->D != 256)) return LUCETREE_ERR_UNSUPPORTED;
    if (!a->start || !a->page_table || !a->ctx_len_in || !a->ctx_len_out || !a->k_pool || !a->v_pool || !a->status ||
        (kq && !a->k_exp) || (vq && !a->v_exp))
        return LUCETREE_ERR_INVALID_ARG;
    if (a->rows > 0 && (!a->k || !a->v)) return LUCETREE_ERR_INVALID_ARG;
    if ((a->q != nullptr) != (a->q_out != nullptr) || (a->q && a->Hq <= 0)) return LUCETREE_ERR_INVALID_ARG;
    if (a->steps) {
        if (a->layout != LUCETREE_ROPE_HALF && a->layout != LUCETREE_ROPE_PAIRS) return LUCETREE_ERR_UNSUPPORTED;
        if (a->rot_dims < 2 || a->rot_dims > a->D || a->rot_dims % 2 != 0 || !isfinite(a->magnitude))
            return LUCETREE_ERR_INVALID_ARG;
    }
    const long long T = a->rows, qe = a->q ? (long long)a->Hq * a->D : 0, ke = (long long)a->Hkv * a->D;
    if (qe > 0x7fffffffll || ke > 0x7fffffffll || a->B + T > 0x7fffff00ll || a->max_pages_per_seq >= (1 << 25) ||
        (long long)(a->q ? a->Hq : 0) + 2ll * a->Hkv > 0x3fffffffll)
        return LUCETREE_ERR_UNSUPPORTED;
    if (T > 0 && (!stride_ok(a->k_stride, ke) || !stride_ok(a->v_stride, ke) || (a->q && !stride_ok(a->q_stride, qe))))
        return LUCETREE_ERR_INVALID_ARG;
    for (const void* p : {a->q, a->k, a->v, (const void*)a->q_out, (const void*)a->k_pool, (const void*)a->v_pool})
        if (!aligned(p, 16)) return LUCETREE_ERR_INVALID_ARG;
    const long long pool_rows = (long long)a->num_pages * a->Hkv * kPage;
    const long long k_row = kq ? a->D : 2ll * a->D;
    const long long v_row = a->v_format == LUCETREE_V_INT4 ? a->D / 2 : vq ? a->D : 2ll * a->D;
    const Span out[] = {{a->k_pool, pool_rows * k_row}, {a->v_pool, pool_rows * v_row}, {a->q_out, 2 * T * qe},
                        {a->ctx_len_out, 4ll * a->B}, {kq ? a->k_exp : nullptr, pool_rows}, {vq ? a->v_exp : nullptr, pool_rows}};
    const Span in[] = {{a->q, span_bytes(T, a->q_stride, qe)}, {a->k, span_bytes(T, a->k_stride, ke)},
                       {a->v, span_bytes(T, a->v_stride, ke)}, {a->start, 4ll * (a->B + 1ll)},
                       {a->page_table, 4ll * a->B * a->max_pages_per_seq}, {a->ctx_len_in, 4ll * a->B},
                       {a->steps, 4ll * a->rot_dims}};
    if (any_overlap(out, in)) return LUCETREE_ERR_INVALID_ARG;
    return launch_append_kv(*a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LUCETREE_OK : LUCETREE_ERR_CUDA;
}
