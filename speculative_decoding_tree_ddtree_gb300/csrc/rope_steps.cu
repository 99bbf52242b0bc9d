// rope_steps.cu -- lucetree_rope_steps: the angles per position as whole multiples of 2^-64 of a turn.
//
// A step serves positions up to 2^31, so its last places count: in 64-bit floating point a power and the
// quotient by 2 pi leave it off by up to 2^-55 of a turn, 2^-24 after 2^31 positions.  So they are taken as sums of
// two doubles (about 104 bits): products and sums with their errors (Dekker, Knuth), the exponential by
// halving its argument and Taylor's series, the logarithm by one step of Newton's method from the 53-bit one.
// Every fused product is written as one: the same bits on every host.
#include <math.h>

#include "lucetree.h"

namespace lucetree {

namespace {

struct Two {
    double hi, lo;  // hi is the sum, rounded
};

Two sum2(double a, double b) {
    const double s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
Two tidy(double hi, double lo) {  // |lo| is small next to hi
    const double s = hi + lo;
    return {s, lo - (s - hi)};
}
Two add(Two a, Two b) {
    const Two s = sum2(a.hi, b.hi), t = sum2(a.lo, b.lo);
    const Two u = tidy(s.hi, s.lo + t.hi);
    return tidy(u.hi, u.lo + t.lo);
}
Two minus(Two a) { return {-a.hi, -a.lo}; }
Two mul(Two a, Two b) {
    const double p = a.hi * b.hi, e = fma(a.hi, b.hi, -p);
    return tidy(p, fma(a.hi, b.lo, fma(a.lo, b.hi, e)));
}
Two div(Two a, Two b) {
    const double q = a.hi / b.hi;
    const Two r = add(a, minus(mul(b, {q, 0.0})));
    const double q2 = r.hi / b.hi;
    const Two r2 = add(r, minus(mul(b, {q2, 0.0})));
    return add(tidy(q, q2), {r2.hi / b.hi, 0.0});
}

constexpr Two kLog2 = {0.6931471805599453, 2.3190468138462996e-17};
constexpr Two kTwoPi = {6.283185307179586, 2.4492935982947064e-16};

Two exp_two(Two x) {  // e^x
    const double k = nearbyint(x.hi / kLog2.hi);
    Two r = add(x, minus(mul(kLog2, {k, 0.0})));
    constexpr int kHalvings = 9;
    const double part = ldexp(1.0, -kHalvings);  // |r| <= 0.35 -> 0.0007
    r = {r.hi * part, r.lo * part};
    // e^r - 1 to r^11 / 11!, off by less than 2^-140
    Two y = {0.0, 0.0};
    for (int n = 11; n >= 1; --n) y = mul(div(r, {(double)n, 0.0}), add(y, {1.0, 0.0}));
    for (int n = 0; n < kHalvings; ++n) y = add(add(y, y), mul(y, y));  // (1 + y)^2 - 1
    y = add(y, {1.0, 0.0});
    return {ldexp(y.hi, (int)k), ldexp(y.lo, (int)k)};
}
Two ln_two(double x) {  // ln x
    const double y = log(x);
    // y + (x e^-y - 1); scaled by the power of two of x, so that neither factor leaves the range
    int e;
    const double m = frexp(x, &e);
    const Two f = exp_two(add({-y, 0.0}, mul(kLog2, {(double)e, 0.0})));
    return add({y, 0.0}, add(mul({m, 0.0}, f), {-1.0, 0.0}));
}

// (num / den) in [0, 1], clamped
Two clamp01(Two num, Two den) {
    const double w = num.hi / den.hi;
    if (!(w > -1.0)) return {0.0, 0.0};
    if (w > 2.0) return {1.0, 0.0};
    const Two q = div(num, den);
    if (q.hi < 0.0) return {0.0, 0.0};
    if (q.hi > 1.0 || (q.hi == 1.0 && q.lo > 0.0)) return {1.0, 0.0};
    return q;
}

// x >= 0, modulo 1, in units of 2^-64 (whole part, modulo 2^64, and rest in [0, 1))
uint64_t units(double x, double* rest) {
    constexpr double k64 = 18446744073709551616.0;
    *rest = 0.0;
    if (fabs(x) >= 9007199254740992.0) return 0;  // a whole number
    const double a = fmod(ldexp(x, 64), k64), w = floor(a);
    *rest = a - w;
    return w >= 0.0 ? (w < k64 ? (uint64_t)w : 0) : 0 - (uint64_t)(-w);
}
uint64_t fraction(Two x) {
    double a, b;
    const uint64_t hi = units(x.hi, &a), lo = units(x.lo, &b);
    return hi + lo + (uint64_t)nearbyint(a + b);
}

}  // namespace

}  // namespace lucetree

using namespace lucetree;

extern "C" lucetree_status lucetree_rope_steps(const lucetree_rope_config* c, uint64_t* steps, float* magnitude) {
    if (!c || !steps || !magnitude) return LUCETREE_ERR_INVALID_ARG;
    const int r = c->rot_dims;
    if (r < 2 || r > 1024 || r % 2 != 0 || c->scaling < LUCETREE_ROPE_NONE || c->scaling > LUCETREE_ROPE_YARN)
        return LUCETREE_ERR_INVALID_ARG;
    if (!(c->base > 1.0) || !isfinite(c->base)) return LUCETREE_ERR_INVALID_ARG;
    const bool scaled = c->scaling != LUCETREE_ROPE_NONE;
    if (scaled && (!(c->factor >= 1.0) || !isfinite(c->factor))) return LUCETREE_ERR_INVALID_ARG;
    if (c->scaling == LUCETREE_ROPE_NTK && r <= 2) return LUCETREE_ERR_INVALID_ARG;
    const bool banded = c->scaling == LUCETREE_ROPE_BANDS || c->scaling == LUCETREE_ROPE_YARN;
    if (banded && (!(c->orig_ctx > 0.0) || !isfinite(c->orig_ctx) || !(c->low > 0.0) || !(c->high > c->low) ||
                   !isfinite(c->high)))
        return LUCETREE_ERR_INVALID_ARG;
    const bool yarn = c->scaling == LUCETREE_ROPE_YARN;
    if (yarn && (!(c->magnitude >= 0.0) || !isfinite((float)c->magnitude))) return LUCETREE_ERR_INVALID_ARG;
    // (no angle is above 1 before its division, so that all of them stay finite)
    for (int i = 0; c->factors && i < r / 2; ++i)
        if (!(c->factors[i] > 0.0) || !isfinite(c->factors[i]) || !isfinite(1.0 / c->factors[i])) return LUCETREE_ERR_INVALID_ARG;
    const double s = scaled ? c->factor : 1.0;
    Two log_base = ln_two(c->base);
    if (c->scaling == LUCETREE_ROPE_NTK) log_base = add(log_base, mul(div({(double)r, 0.0}, {r - 2.0, 0.0}), ln_two(s)));
    double lo = 0.0, hi = 0.0;
    if (yarn) {
        auto dim = [&](double turns) { return r * log(c->orig_ctx / (kTwoPi.hi * turns)) / (2.0 * log(c->base)); };
        lo = fmax(floor(dim(c->high)), 0.0);
        hi = fmin(ceil(dim(c->low)), r - 1.0);
    }
    for (int i = 0; i < r / 2; ++i) {
        Two f = exp_two(mul(div({-2.0 * i, 0.0}, {(double)r, 0.0}), log_base));
        if (c->scaling == LUCETREE_ROPE_LINEAR) f = div(f, {s, 0.0});
        if (banded) {
            Two w;  // of the angle as it is
            if (yarn) {
                w = clamp01(sum2(i, -lo), {fmax(hi - lo, 0.001), 0.0});
                w = add({1.0, 0.0}, minus(w));
            } else {
                w = clamp01(add(div(mul({c->orig_ctx, 0.0}, f), kTwoPi), {-c->low, 0.0}), sum2(c->high, -c->low));
            }
            f = add(mul(w, f), mul(add({1.0, 0.0}, minus(w)), div(f, {s, 0.0})));
        }
        if (c->factors) f = div(f, {c->factors[i], 0.0});
        steps[i] = fraction(div(f, kTwoPi));
    }
    *magnitude = yarn ? (float)(c->magnitude > 0.0 ? c->magnitude : 0.1 * log(s) + 1.0) : 1.f;
    return LUCETREE_OK;
}
