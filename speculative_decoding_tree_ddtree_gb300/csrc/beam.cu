// beam.cu -- lucetree_beam_select: the best continuations of a request's beams
// over the whole vocabulary.
//
// score(k, t) = cum_k + x_kt - log sum_t' exp x_kt'.  Within a row the order is
// that of the logits, so one pass over a row finds both its softmax sum and its
// best Kout tokens; only those can be among the request's best Kout.
//
// Launch 1 cuts the rows into chunks (no more CTAs than run at once).  While
// streaming, a thread only keeps a running maximum, the vector it lies in, and
// the sum: the Kout best elements of a chunk can only be in the Kout threads
// with the best maxima.  Those threads are found by sorting 256 (maximum,
// vector) keys, and their vectors are gone through once more for the elements.
// Keys are 64-bit integers whose order is (logit descending, index ascending),
// lists of 32 lie across a warp's lanes, and sorts and merges are bitonic
// networks of shuffles.
// Launch 2, one CTA per request, adds the chunks' sums up row by row, turns the
// chunks' lists into scores of some 48 bits (neighbouring candidates of different
// rows are closer than fp32 keeps beside a long sum) and takes the best: 3.6 us from
// the last chunk's end, of which 0.6 are the wait itself and 1.0 the loads (merging sorted
// lists by bitonic networks with fp64 scores: 6.1).
// 8 requests of 8 beams over 151,936 fp32 logits (39 MB): 15.8 us, 2.5 TB/s; 32 of
// bf16 logits, a quarter of the beams finished: 23.6 us.  Bound by the fixed part
// of a chunk (its sorts start when the stream ends: all CTAs run in one wave) and the
// second launch; smaller chunks cost more (twice as many: 19.0 us).
#include <type_traits>

#include "beam.h"
#include "internal.cuh"

namespace lucetree {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kMergeThreads = 256;  // as many registers as a CTA of the scan: it fits where one is free
constexpr int kU = 8;  // 16-byte loads in flight per thread

struct BeamLaunch {
    lucetree_beam_args a;
    int chunks;
    u64* keys;     // [rows][chunks][32]
    float2* sums;  // [rows][chunks] (maximum, sum of exp(x - maximum))
};

// Order of (x, index) as an integer: larger x first, then the lower index;
// -0.0 ties +0.0.  0 is below every element.
__device__ inline u64 pack_key(float x, unsigned idx) {
    if (x == 0.f) x = 0.f;
    unsigned u = __float_as_uint(x);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((u64)u << 32) | (u64)(~idx);
}
__device__ inline float key_value(u64 k) {
    const unsigned u = (unsigned)(k >> 32);
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}
__device__ inline unsigned key_index(u64 k) { return ~(unsigned)k; }

// Keys across the warp's lanes, descending by lane.
__device__ inline u64 exchange(u64 k, int stride, bool keep_max) {
    const u64 o = __shfl_xor_sync(0xffffffffu, k, stride);
    return (k > o) == keep_max ? k : o;
}
__device__ inline u64 sort32(u64 k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1)
            k = exchange(k, stride, ((lane & stride) == 0) == ((lane & size) == 0));
    return k;
}
// The 32 best of two descending lists.
__device__ inline u64 merge32(u64 a, u64 b) {
    const int lane = threadIdx.x & 31;
    const u64 r = __shfl_sync(0xffffffffu, b, 31 - lane);
    u64 k = a > r ? a : r;
#pragma unroll
    for (int stride = 16; stride > 0; stride >>= 1) k = exchange(k, stride, (lane & stride) == 0);
    return k;
}

template <typename T>
struct Vec {
    static constexpr int kE = 16 / sizeof(T);
};

template <typename T>
__device__ inline void unpack(const uint4& u, float (&x)[Vec<T>::kE]) {
    if constexpr (sizeof(T) == 4) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    } else {
        load8_f32<T>(reinterpret_cast<const T*>(&u), x);
    }
}

// Largest element (of 16-bit ones in their own type: no conversions to keep in registers).
template <typename T>
__device__ inline float vector_max(const uint4& u) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    } else if constexpr (std::is_same<T, __half>::value) {
        const __half2* h = reinterpret_cast<const __half2*>(&u);
        const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
}

// Vec<T>::kE elements from p on: one load where p is aligned to 16 bytes.
template <typename T, bool ALIGNED>
__device__ inline uint4 load_vector(const T* p) {
    if constexpr (ALIGNED) {
        return __ldg(reinterpret_cast<const uint4*>(p));
    } else if constexpr (sizeof(T) == 4) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
        return make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
    } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
        auto two = [&](int e) { return (uint32_t)__ldg(h + e) | (uint32_t)__ldg(h + e + 1) << 16; };
        return make_uint4(two(0), two(2), two(4), two(6));
    }
}

__device__ inline float scalar(const float* p) { return *p; }
__device__ inline float scalar(const __half* p) { return __half2float(*p); }
__device__ inline float scalar(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// exp(x - m) by the hardware's base-2 exponential (2 ulp)
__device__ inline float exp_diff(float x, float m) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x - m) * kLog2e));
    return y;
}

// Two fp32 in one register pair: one instruction for two additions or products.
__device__ inline uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ inline float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ inline float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ inline uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ inline uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ inline uint64_t exp_diff2(float x, float y, uint64_t minus_m) {
    const uint64_t r = mul2(add2(pack2(x, y), minus_m), pack2(kLog2e, kLog2e));
    float p, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(low(r)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(high(r)));
    return pack2(p, q);
}

// (m, s) += (m2, s2): sums of exponentials relative to their maxima; a maximum of -inf has sum 0.
__device__ inline void add_sums(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    if (top == -INFINITY) return;
    s = (m == -INFINITY ? 0.f : s * exp_diff(m, top)) + (m2 == -INFINITY ? 0.f : s2 * exp_diff(m2, top));
    m = top;
}

// The warp's (m, s) in every lane.
__device__ inline void warp_sums(float& m, float& s) {
    float top;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(m));
    s = m == -INFINITY ? 0.f : s * exp_diff(m, top);
    m = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
}

__device__ inline bool row_ended(const lucetree_beam_args& a, int row) {
    return a.finished && a.finished[row] != 0;
}

// The best keys of all warps' sorted lists in s_list[0] (kWarps lists of 32).
__device__ inline void merge_warps(u64 (*s_list)[32], u64 mine) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    s_list[warp][lane] = mine;
#pragma unroll
    for (int half = kWarps / 2; half > 0; half >>= 1) {
        __syncthreads();
        if (warp < half) s_list[warp][lane] = mine = merge32(mine, s_list[warp + half][lane]);
    }
}

// ALIGNED: every row starts on a 16-byte boundary.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) beam_scan_kernel(BeamLaunch L) {
    constexpr int kE = Vec<T>::kE;
    __shared__ u64 s_list[kWarps][32];
    __shared__ u64 s_buf[kWarps][32 + 32 * kE];  // what one vector of every lane may add to 31 waiting keys
    __shared__ float2 s_sum[kWarps];
    __shared__ int s_left[kWarps];
    const lucetree_beam_args& a = L.a;
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int row = blockIdx.y, chunk = blockIdx.x, t = threadIdx.x;
    // rows that ended or are dead (at -inf or NaN) need no logits (launch 2 knows their candidates)
    if (row_ended(a, row) || !(a.cum[row] > -INFINITY)) return;
    const int warp = t >> 5, lane = t & 31;
    const T* x = reinterpret_cast<const T*>(a.logits) + (long long)row * a.row_stride;
    // vectors of kE elements by index, so that a row's sum does not depend on where
    // it lies (equal rows tie exactly); the last vocab % kE belong to the last chunk
    const int nv = a.vocab / kE;
    auto fetch = [&](int v) { return load_vector<T, ALIGNED>(x + (long long)v * kE); };
    const int v0 = (int)((long long)nv * chunk / L.chunks), v1 = (int)((long long)nv * (chunk + 1) / L.chunks);

    // thread t's vectors are v0 + t, v0 + t + kThreads, ..
    float m = -INFINITY;
    uint64_t s2 = 0;  // two sums of exp(x - m)
    int best = v0 + t;
    // kU vectors, kThreads apart, the first of them v; `all`: they all lie in the chunk
    // (those that do not count as vectors of -inf)
    auto batch = [&](auto all, int v) {
        constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
        uint4 u[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k)
            u[k] = all.value || v + k * kThreads < v1 ? fetch(v + k * kThreads) : make_uint4(kNone, kNone, kNone, kNone);
        float mb = m;
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            const float vm = vector_max<T>(u[k]);
            if (vm > mb) {
                mb = vm;
                best = v + k * kThreads;
            }
        }
        if (mb > m) {
            const float f = exp_diff(m, mb);  // 0 for the first
            s2 = mul2(s2, pack2(f, f));
            m = mb;
        }
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t minus_m = pack2(-mm, -mm);
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            float f[kE];
            unpack<T>(u[k], f);
#pragma unroll
            for (int e = 0; e < kE; e += 2) s2 = add2(s2, exp_diff2(f[e], f[e + 1], minus_m));
        }
    };
    int base = v0;
    for (; base + kU * kThreads <= v1; base += kU * kThreads) batch(std::true_type{}, base + t);
    if (base < v1) batch(std::false_type{}, base + t);
    float s = low(s2) + high(s2);
    // the threads with the best maxima
    merge_warps(s_list, sort32(v0 + t < v1 ? pack_key(m, (unsigned)best) : 0));
    __syncthreads();
    const u64 threads = s_list[0][lane];
    const u64 limit = __shfl_sync(0xffffffffu, threads, a.beams_out - 1);  // 0: fewer threads than that have a vector
    // A warp goes through one thread's vectors at a time; keys that count wait in shared
    // memory until 32 of them are sorted and merged into the warp's list.  Most
    // warps never have 32: what is left over is put together and ranked.
    u64 list = 0;
    int waiting = 0;
    bool listed = false;
    for (int i = warp; i < a.beams_out; i += kWarps) {
        const u64 key = __shfl_sync(0xffffffffu, threads, i);
        if (key == 0) break;
        const int first = v0 + (int)((key_index(key) - (unsigned)v0) % kThreads);
        for (int v = first + lane * kThreads; __any_sync(0xffffffffu, v < v1); v += 32 * kThreads) {
            float f[kE];
            unpack<T>(v < v1 ? fetch(v) : make_uint4(0, 0, 0, 0), f);
            // no element of a vector below the limit is among the best (keys of vectors order as their elements' do)
            unsigned pass = 0;
#pragma unroll
            for (int e = 0; e < kE; ++e) pass |= v < v1 && pack_key(f[e], (unsigned)v) >= limit ? 1u << e : 0u;
            int upto = __popc(pass);
            const int mine = upto;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            int at = waiting + upto - mine;
#pragma unroll
            for (int e = 0; e < kE; ++e)
                if ((pass >> e) & 1u) s_buf[warp][at++] = pack_key(f[e], (unsigned)(v * kE + e));
            waiting += __shfl_sync(0xffffffffu, upto, 31);
            __syncwarp();
            for (; waiting >= 32; waiting -= 32) {
                list = merge32(list, sort32(s_buf[warp][waiting - 32 + lane]));
                listed = true;
            }
            __syncwarp();
        }
    }
    if (chunk == L.chunks - 1 && warp == 0) {
        const bool in = lane < a.vocab - nv * kE;  // (nv * kE + lane may pass 2^31)
        const int i = nv * kE + (in ? lane : 0);
        const float f = in ? scalar(x + i) : -INFINITY;
        if (in) add_sums(m, s, f, f == -INFINITY ? 0.f : 1.f);
        if (waiting + kE > 32) {  // (the tail has fewer than kE elements)
            list = merge32(list, sort32(lane < waiting ? s_buf[warp][lane] : 0));
            listed = true;
            waiting = 0;
        }
        __syncwarp();
        if (in) s_buf[warp][waiting + lane] = pack_key(f, (unsigned)i);
        waiting += __popc(__ballot_sync(0xffffffffu, in));
        __syncwarp();
    }
    // the CTA's sum and list
    warp_sums(m, s);
    if (lane == 0) {
        s_sum[warp] = make_float2(m, s);
        s_left[warp] = waiting;
    }
    const bool any_listed = __syncthreads_or(listed);  // (every warp has read the threads' list)
    int at = 0, left = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        at += w < warp ? s_left[w] : 0;
        left += s_left[w];
    }
    u64* all = &s_list[0][0];  // fewer than 32 keys of each warp
    if (lane < waiting) all[at + lane] = s_buf[warp][lane];
    __syncthreads();
    const size_t place = (size_t)row * L.chunks + chunk;
    u64* out = L.keys + place * 32;
    if (!any_listed && left <= 64) {
        const u64 k0 = lane < left ? all[lane] : 0, k1 = lane + 32 < left ? all[lane + 32] : 0;
#pragma unroll 1
        for (int i = warp; i < left; i += kWarps) {
            const u64 d = all[i];
            const int ahead = __popc(__ballot_sync(0xffffffffu, k0 > d)) + __popc(__ballot_sync(0xffffffffu, k1 > d));
            if (lane == 0 && ahead < a.beams_out) out[ahead] = d;
        }
        if (t >= left && t < a.beams_out) out[t] = 0;
    } else {
        if (warp == 0) {
#pragma unroll 1
            for (int g = 0; g < left; g += 32) list = merge32(list, sort32(g + lane < left ? all[g + lane] : 0));
        }
        if (any_listed) {
            __syncthreads();
            merge_warps(s_list, list);
            list = s_list[0][lane];
        }
        if (warp == 0) out[lane] = list;
    }
    if (warp == 0) {
        m = lane < kWarps ? s_sum[lane].x : -INFINITY;
        s = lane < kWarps ? s_sum[lane].y : 0.f;
        warp_sums(m, s);
        if (lane == 0) L.sums[place] = make_float2(m, s);
    }
}

// A float as an ordered integer.
__device__ inline unsigned order_float(float x) {
    const unsigned u = __float_as_uint(x == 0.f ? 0.f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// x + y as a float and its rounding error (Knuth's two-sum).
__device__ inline float2 two_sum(float x, float y) {
    const float s = __fadd_rn(x, y), z = __fsub_rn(s, x);
    return make_float2(s, __fadd_rn(__fsub_rn(x, __fsub_rn(s, z)), __fsub_rn(y, z)));
}

// Scores are sums of two floats, some 48 bits (neighbouring candidates of different
// rows are closer than fp32 keeps beside a long sum; fp64 runs at 1/64 of its rate),
// and a quarter of their value, so that three finite terms cannot overflow.
constexpr float kQuarter = 0.25f;

// A quarter of m + log(s): s = 2^k f with f in [3/4, 3/2), the logarithm of f, at most 0.41,
// in fp32 and k log 2 in two parts, of which the first has 16 bits (Cody and Waite).
__device__ inline float2 quarter_lse(float m, float s) {
    int k;
    float f = frexpf(s, &k);  // in [1/2, 1)
    if (f < 0.75f) {
        f *= 2.f;
        --k;
    }
    constexpr float kHigh = 45426.f / 65536.f, kLow = (float)(0.6931471805599453 - 45426.0 / 65536.0);
    const float2 t = two_sum(m * kQuarter, kQuarter * (kHigh * k));
    const float low = kQuarter * fmaf(kLow, (float)k, log1pf(f - 1.f));
    const float2 u = two_sum(t.x, low);
    return two_sum(u.x, u.y + t.y);
}

// A candidate of the request: its score as an ordered integer, and beam * vocab + token.
struct Cand {
    u64 score;
    unsigned index;
};
constexpr u64 kNoScore = 0;  // of no candidate; below that of -inf

// (no branches)
__device__ inline bool better(const Cand& p, const Cand& q) {
    return (p.score > q.score) | ((p.score == q.score) & (p.index < q.index));
}
__device__ inline Cand better_of(const Cand& p, const Cand& q) { return better(q, p) ? q : p; }
__device__ inline Cand shfl_xor(const Cand& c, int o) {
    return Cand{__shfl_xor_sync(0xffffffffu, c.score, o), __shfl_xor_sync(0xffffffffu, c.index, o)};
}
__device__ inline u64 order_score(float2 x) { return ((u64)order_float(x.x) << 32) | order_float(x.y); }
__device__ inline float score_value(u64 score) {
    const unsigned u = (unsigned)(score >> 32);
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u) * (1.f / kQuarter);
}

// One CTA per request.  A list of Kout keys lies across `width` lanes (a power of two),
// every eighth list in the same warp, so that the good ones are spread over the
// warps.  The Kout-th best of 32 candidates, the first ones of lists, is no better
// than the Kout-th best of all: what is behind it drops out, and the few that are left
// (some 20 of 576 for eight beams of nine chunks) are ranked by counting.
// The steps run over nothing while the scan is still at work: a cold instruction cache
// costs more than the work itself.  First each in a warp of its own: behind the scan's
// loads one miss after the other would take longer than the scan (up to 14 us).
__global__ void __launch_bounds__(kMergeThreads, kCtasPerSm) beam_merge_kernel(BeamLaunch L) {
    constexpr int kMergeWarps = kMergeThreads / 32;
    constexpr int kLeft = kMergeThreads;  // candidates that are ranked by counting
    constexpr int kHold = 4;              // lists of a lane that are loaded at once and kept
    static_assert(kMergeWarps * 4 == 32, "four candidates of each warp are compared");
    enum { kLive, kEnded, kDead };
    __shared__ Cand s_first[32], s_left[kLeft], s_limit;
    __shared__ float2 s_lse[LUCETREE_MAX_BEAMS];
    __shared__ float s_cum[LUCETREE_MAX_BEAMS];
    __shared__ int s_state[LUCETREE_MAX_BEAMS];
    __shared__ int s_n;
    const lucetree_beam_args& a = L.a;
    const int b = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int K = a.beams_in, Kout = a.beams_out, chunks = L.chunks;
    const int width = 1 << (32 - __clz(Kout - 1));  // (1 for Kout = 1)
    const int j = lane & (width - 1);
    const int lists = K * chunks, per_pass = kMergeThreads / width;
    const int first_list = j < Kout ? (lane / width) * kMergeWarps + warp : lists;
    const u64* keys = L.keys + (size_t)b * lists * 32 + j;
    int beam[kHold];  // of the lane's first lists
#pragma unroll
    for (int x = 0; x < kHold; ++x) beam[x] = min(first_list + x * per_pass, lists - 1) / chunks;
    // (the inputs are those that the scan has waited for)
    const float cum_t = t < K ? __ldcg(a.cum + b * K + t) : 0.f;
    const bool ended_t = t < K && a.finished && __ldcg(a.finished + b * K + t) != 0;

    auto key_of = [&](int l, int k) -> u64 { return l < lists && s_state[k] == kLive ? keys[(size_t)l * 32] : 0; };
    auto cand_of = [&](int l, int k, u64 key) -> Cand {
        if (l >= lists) return Cand{kNoScore, ~0u};
        const float2 lse = s_lse[k];
        const float cum = s_cum[k] * kQuarter, x = key_value(key) * kQuarter;
        const float2 d = two_sum(x, -lse.x), e = two_sum(d.x, cum);
        float2 score = two_sum(e.x, (d.y + e.y) - lse.y);
        int token = (int)key_index(key);
        bool have = key != 0;
        if (s_state[k] != kLive || !(lse.x > -INFINITY)) {
            // the row's tokens in order, all at -inf, but after the one candidate of a beam that has ended
            // (with a score: at -inf eos is a token like the others)
            const bool one = s_state[k] == kEnded && cum > -INFINITY && a.eos >= 0 && a.eos < a.vocab;
            have = l == k * chunks && j < a.vocab;
            token = one ? (j == 0 ? a.eos : (j - 1 < a.eos ? j - 1 : j)) : j;
            score = make_float2(one && j == 0 ? cum : -INFINITY, 0.f);
        }
        if (!(score.x > -INFINITY)) score = make_float2(-INFINITY, 0.f);  // (a masked logit: NaN in the errors)
        return have ? Cand{order_score(score), (unsigned)k * (unsigned)a.vocab + (unsigned)token} : Cand{kNoScore, ~0u};
    };
    auto write = [&](bool warm, int at, const Cand& c) {
        const int beam = (int)(c.index / (unsigned)a.vocab), token = (int)(c.index % (unsigned)a.vocab);
        const size_t o = (size_t)b * Kout + at;
        const float score = score_value(c.score);
        if (warm) return;
        a.out_score[o] = score;
        a.out_token[o] = token;
        a.out_row[o] = b * K + beam;
        if (a.out_finished) a.out_finished[o] = (s_state[beam] == kEnded || token == a.eos) ? 1 : 0;
    };

#pragma unroll 1
    for (int warm = 2; warm >= 0; --warm) {
        auto mine = [&](int w) { return warm < 2 || warp == w; };
        u64 key[kHold];
        if (!warm) {
            if (t < K) {
                s_cum[t] = cum_t;
                s_state[t] = ended_t ? kEnded : cum_t > -INFINITY ? kLive : kDead;
            }
            __syncthreads();
            pdl_wait();
            if (t == 0) {
                pdl_trigger();
                s_n = 0;
            }
#pragma unroll
            for (int x = 0; x < kHold; ++x) key[x] = key_of(first_list + x * per_pass, beam[x]);
        }
        // log-sum-exp of the rows from their chunks
        if (mine(0)) {
#pragma unroll 1
            for (int k = warp; k < K; k += kMergeWarps) {
                const float2* sums = L.sums + (size_t)(b * K + k) * chunks;
                if (!warm && s_state[k] != kLive) continue;
                float m = -INFINITY, s = 0.f;
#pragma unroll 1
                for (int c = lane; c < chunks; c += 32) {
                    const float2 x = warm ? make_float2(0.f, 1.f) : sums[c];
                    add_sums(m, s, x.x, x.y);
                }
                warp_sums(m, s);
                const float2 lse = m > -INFINITY ? quarter_lse(m, s) : make_float2(-INFINITY, 0.f);
                if (lane == 0) s_lse[k] = lse;
            }
        }
        if (!warm) __syncthreads();
        // the best candidate of every lane, and of the lists that share a lane's eighth
        Cand c[kHold];
        if (mine(1)) {
            Cand top{kNoScore, ~0u};
#pragma unroll
            for (int x = 0; x < kHold; ++x) {
                c[x] = cand_of(first_list + x * per_pass, beam[x], warm ? (u64)t << 32 : key[x]);
                top = better_of(top, c[x]);
            }
#pragma unroll 1
            for (int l = first_list + kHold * per_pass; l < lists && !warm; l += per_pass)
                top = better_of(top, cand_of(l, l / chunks, key_of(l, l / chunks)));
            __syncwarp();
#pragma unroll 1
            for (int o = width; o < 8; o <<= 1) top = better_of(top, shfl_xor(top, o));
            const int group = width > 8 ? width : 8;  // lanes of which the first eighth is taken
            if ((lane & (group - 1)) < group / 8)
                s_first[warp * 4 + (lane / group) * (group / 8) + (lane & (group - 1))] = top;
        }
        if (!warm) __syncthreads();
        if (mine(2)) {
            const Cand one = s_first[lane];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int i = warp * 4 + x;
                const Cand d = s_first[i];
                // (several may be no candidate)
                const bool ahead = better(one, d) | ((one.score == d.score) & (one.index == d.index) & (lane < i));
                if (__popc(__ballot_sync(0xffffffffu, ahead)) == Kout - 1 && lane == 0) s_limit = d;
            }
        }
        if (!warm) __syncthreads();
        if (mine(3)) {
            const Cand limit = s_limit;
            auto keep = [&](const Cand& c) {
                if ((c.score == kNoScore) | better(limit, c)) return;
                const unsigned at = warm ? t : atomicAdd(&s_n, 1);  // (any order: they are ranked)
                if (at < kLeft) s_left[at] = c;
            };
#pragma unroll
            for (int x = 0; x < kHold; ++x) keep(warm ? Cand{limit.score | 1, 0} : c[x]);
#pragma unroll 1
            for (int l = first_list + kHold * per_pass; l < lists && !warm; l += per_pass)
                keep(cand_of(l, l / chunks, key_of(l, l / chunks)));
        }
        if (!warm) __syncthreads();
        const int n = warm ? 32 : s_n;
        if (n <= kLeft) {
            if (mine(4)) {
                // lane x of a warp ends up with the rank of its x-th candidate
                const Cand none{kNoScore, ~0u};
                const Cand d0 = lane < n ? s_left[lane] : none, d1 = lane + 32 < n ? s_left[lane + 32] : none;
                int rank = Kout;
#pragma unroll 2
                for (int i = warp, x = 0; i < n; i += kMergeWarps, ++x) {
                    const Cand d = s_left[i];
                    int ahead = __popc(__ballot_sync(0xffffffffu, better(d0, d))) + __popc(__ballot_sync(0xffffffffu, better(d1, d)));
#pragma unroll 1
                    for (int g = 64; g < n; g += 32)
                        ahead += __popc(__ballot_sync(0xffffffffu, g + lane < n && better(s_left[g + lane], d)));
                    if (lane == x) rank = ahead;
                }
                if (rank < Kout) write(warm, rank, s_left[warp + kMergeWarps * lane]);
                // (there are fewer than Kout candidates only after NaN logits)
                if (t >= n && t < Kout) write(warm, t, Cand{order_score(make_float2(-INFINITY, 0.f)), 0});
            }
        } else {
            // The good candidates share a few warps: one best after the other.
            Cand last{~0ull, 0};
#pragma unroll 1
            for (int r = 0; r < Kout; ++r) {
                Cand best{kNoScore, ~0u};
#pragma unroll 1
                for (int l = first_list; l < lists; l += per_pass) {
                    const Cand c = cand_of(l, l / chunks, key_of(l, l / chunks));
                    if (better(last, c)) best = better_of(best, c);
                }
#pragma unroll 1
                for (int o = 16; o > 0; o >>= 1) best = better_of(best, shfl_xor(best, o));
                if (lane == 0) s_first[warp] = best;
                __syncthreads();
#pragma unroll 1
                for (int w = 0; w < kMergeWarps; ++w) best = better_of(best, s_first[w]);
                if (t == 0) write(false, r, best);
                last = best;
                __syncthreads();
            }
        }
    }
}

// No more CTAs than run at once (four per SM), as long as there are no more rows
// than that, and no chunk of fewer than four elements a thread.
int beam_chunks(int rows, int vocab, int sms) {
    int chunks = kCtasPerSm * sms / rows;
    const int most = (int)((vocab + 4ll * kThreads - 1) / (4 * kThreads));
    if (chunks > most) chunks = most;
    return chunks < 1 ? 1 : chunks;
}

template <typename T>
cudaError_t launch_scan(const BeamLaunch& L, bool aligned, dim3 grid, cudaStream_t stream) {
    if (aligned) return launch_pdl(beam_scan_kernel<T, true>, grid, dim3(kThreads), 0, stream, L);
    return launch_pdl(beam_scan_kernel<T, false>, grid, dim3(kThreads), 0, stream, L);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t beam_workspace_bytes(int batch, int beams, int vocab, int device) {
    const size_t lists = (size_t)batch * beams * beam_chunks(batch * beams, vocab, device_sm_count(device));
    return align256(lists * 32 * sizeof(u64)) + align256(lists * sizeof(float2));
}

cudaError_t launch_beam_select(const lucetree_beam_args& a, void* workspace, int device, cudaStream_t stream) {
    BeamLaunch L;
    L.a = a;
    const int rows = a.batch * a.beams_in;
    L.chunks = beam_chunks(rows, a.vocab, device_sm_count(device));
    L.keys = reinterpret_cast<u64*>(workspace);
    L.sums = reinterpret_cast<float2*>(reinterpret_cast<char*>(workspace) +
                                       align256((size_t)rows * L.chunks * 32 * sizeof(u64)));
    const dim3 grid(L.chunks, rows);
    const int size = a.dtype == LUCETREE_F32 ? 4 : 2;
    const bool aligned = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && (rows == 1 || a.row_stride * size % 16 == 0);
    cudaError_t e;
    if (a.dtype == LUCETREE_F32) e = launch_scan<float>(L, aligned, grid, stream);
    else if (a.dtype == LUCETREE_BF16) e = launch_scan<__nv_bfloat16>(L, aligned, grid, stream);
    else e = launch_scan<__half>(L, aligned, grid, stream);
    if (e != cudaSuccess) return e;
    return launch_pdl(beam_merge_kernel, dim3(a.batch), dim3(kMergeThreads), 0, stream, L);
}

}  // namespace lucetree

using namespace lucetree;

extern "C" {

static lucetree_status beam_sizes(int batch, int beams_in, int beams_out, int vocab) {
    if (batch < 1 || beams_in < 1 || beams_out < 1 || vocab < 1) return LUCETREE_ERR_INVALID_ARG;
    if (beams_in > LUCETREE_MAX_BEAMS || beams_out > LUCETREE_MAX_BEAMS || (long long)batch * beams_in > 65535)
        return LUCETREE_ERR_UNSUPPORTED;
    if ((long long)beams_in * vocab > 0xfffffffell) return LUCETREE_ERR_UNSUPPORTED;  // candidates by a 32-bit index
    if (beams_out > (long long)beams_in * vocab) return LUCETREE_ERR_INVALID_ARG;  // fewer candidates than beams
    return LUCETREE_OK;
}

// An output under an input (but for the two updates in place) or under another output:
// a request's results would change what other requests still read.
static bool outputs_overlap(const lucetree_beam_args& a) {
    const long long before = 4ll * a.batch * a.beams_in, after = 4ll * a.batch * a.beams_out;
    const void* in[2] = {a.cum, a.finished};
    const void* out[4] = {a.out_score, a.out_finished, a.out_token, a.out_row};
    for (int o = 0; o < 4; ++o) {
        if (!out[o]) continue;
        for (int i = 0; i < 2; ++i)
            if (i != o && in[i] && bytes_overlap(in[i], before, out[o], after)) return true;
        for (int p = 0; p < o; ++p)
            if (out[p] && bytes_overlap(out[p], after, out[o], after)) return true;
    }
    return false;
}

lucetree_status lucetree_beam_select_workspace(int batch, int beams_in, int beams_out, int vocab, size_t* bytes) {
    if (!bytes) return LUCETREE_ERR_INVALID_ARG;
    const lucetree_status st = beam_sizes(batch, beams_in, beams_out, vocab);
    if (st != LUCETREE_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    *bytes = beam_workspace_bytes(batch, beams_in, vocab, dev);
    return LUCETREE_OK;
}

lucetree_status lucetree_beam_select(const lucetree_beam_args* a, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    if (!a) return LUCETREE_ERR_INVALID_ARG;
    if (a->dtype != LUCETREE_F16 && a->dtype != LUCETREE_BF16 && a->dtype != LUCETREE_F32)
        return LUCETREE_ERR_UNSUPPORTED;
    const lucetree_status st = beam_sizes(a->batch, a->beams_in, a->beams_out, a->vocab);
    if (st != LUCETREE_OK) return st;
    const uintptr_t elem = a->dtype == LUCETREE_F32 ? 4 : 2;
    if (!a->logits || !a->cum || !a->out_score || !a->out_token || !a->out_row || a->row_stride < a->vocab ||
        (reinterpret_cast<uintptr_t>(a->logits) & (elem - 1)) != 0)
        return LUCETREE_ERR_INVALID_ARG;
    // a request's own beams may be updated in place; other overlaps mix up requests
    const long long before = 4ll * a->batch * a->beams_in, after = 4ll * a->batch * a->beams_out;
    const bool same = a->beams_in == a->beams_out;
    if (bytes_overlap(a->cum, before, a->out_score, after) && !(same && (const void*)a->cum == a->out_score))
        return LUCETREE_ERR_INVALID_ARG;
    if (a->finished && a->out_finished && bytes_overlap(a->finished, before, a->out_finished, after) &&
        !(same && a->finished == a->out_finished))
        return LUCETREE_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    if (!workspace || workspace_bytes < beam_workspace_bytes(a->batch, a->beams_in, a->vocab, dev) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return LUCETREE_ERR_WORKSPACE;
    if (outputs_overlap(*a)) return LUCETREE_ERR_INVALID_ARG;
    if (launch_beam_select(*a, workspace, dev, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return LUCETREE_ERR_CUDA;
    return LUCETREE_OK;
}

}  // extern "C"
