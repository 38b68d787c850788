// token_math.cuh -- what the losses over given tokens do with a row's sums (sm_103a;
// the arithmetic also compiles for the host, where the tests compare it with long
// double).
//
// One token a against all others: with m_o the others' largest logit and
// s_o = sum_{v != a} exp((z_v - m_o) / T),
//   ln p = -ln(1 + s_o)                              a at the row's maximum, s_o relative to it
//   ln p = (z_a - m) / T - ln(s_o + e^((z_a - m) / T))   otherwise
//   1 - p = s_o / (s_o + e_a)
// The token's own weight never enters s_o, so ln p and 1 - p keep all their digits
// when the row is sure of the token (as 1 - q from the whole sum 1 - p would be
// rounded away from p = 1 - 2^-24 on, and the token's gradient with it).
#pragma once

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "dlm.h"
#include "token_rules.h"

#ifndef DLM_HD
#ifdef __CUDACC__
#define DLM_HD __device__ __forceinline__
#else
#define DLM_HD inline
#endif
#endif

namespace dlm {

DLM_HD bool is_finite(float x) { return fabsf(x) < INFINITY; }
DLM_HD float f32_nan() { return NAN; }

// A number as a sum of two floats, to about 2^-45.  (64-bit arithmetic has a 64th of the
// 32-bit rate here: with a dozen operations of it a row's slope took 2300 cycles, and the
// row's gradient waits for that.)
struct Two {
    float hi, lo;
};
DLM_HD Two two_sum(float a, float b) {
    const float s = a + b, x = s - a;
    const float e = (a - (s - x)) + (b - x);
    return Two{s, is_finite(s) ? e : 0.f};
}
DLM_HD Two two_prod(float a, float b) {
    const float p = a * b;
    return Two{p, is_finite(p) ? fmaf(a, b, -p) : 0.f};
}
DLM_HD Two plus(Two a, Two b) {
    Two s = two_sum(a.hi, b.hi);
    if (!is_finite(s.hi)) return s;
    return two_sum(s.hi, s.lo + (a.lo + b.lo));
}
DLM_HD Two minus(Two a) { return Two{-a.hi, -a.lo}; }
DLM_HD float rounded(Two a) { return a.hi + a.lo; }

// ln x for a normal x >= 1: the exponent's share exactly, so that what is left to the
// float logarithm is at most ln 2 / 2 (of x itself it is up to 14, and its last place
// 2^-20).
DLM_HD Two ln_split(float x) {
    uint32_t b;
    memcpy(&b, &x, 4);
    int e = (int)(b >> 23) - 127;
    b = (b & 0x7fffffu) | 0x3f800000u;
    float m;
    memcpy(&m, &b, 4);
    if (m > 1.41421354f) {
        m *= 0.5f;
        ++e;
    }
    // ln 2 to 12 bits (2839 / 4096), so that times e it is exact, and the rest of it
    return two_sum((float)e * (2839.f / 4096.f), fmaf((float)e, 3.1946184945e-5f, logf(m)));
}

// What follows from a row's sums: its maximum, 1 / sum, 1 - p of the token, and the
// log-probabilities.  A row that holds NaN or +inf, or -inf only, has NaN in all but
// m, and ok is 0.
struct TokenRow {
    float m, inv, away;
    int ok;
    Two logp, ln;  // ln: of the sum relative to m
};

// 2^-n, 0 <= n <= 126
DLM_HD float pow2_neg(int n) {
    const uint32_t b = (uint32_t)(127 - n) << 23;
    float x;
    memcpy(&x, &b, 4);
    return x;
}
// x 2^(-d (hi + lo)) to 2^-21 for d >= 0 of any size, err what d was rounded by.  (As one
// float the exponent would be off by 2^-24 of itself: 2^-17 at 115.)
DLM_HD float times_exp2(float x, float d, float err, float hi, float lo) {
    const float e = d * hi;
    if (!(e < 200.f)) return e != e ? f32_nan() : 0.f;
    const int n = (int)e, half = n >> 1;
    const float f = (e - (float)n) + fmaf(err, hi, fmaf(d, lo, fmaf(d, hi, -e)));
    return x * exp2f(-f) * pow2_neg(half) * pow2_neg(n - half);
}

// The hardware's 2^x, which the weights are made with, is a little too small on average
// (2^-25 over arguments in [-1, 0), 2^-22.7 at most): a row's sum of thousands of them by
// 2^-24.3 (4.0e-8 to 5.8e-8 over rows of 32000 and 152064 N(0, 4) logits of each type;
// its rounding scatters by as much).  A sequence's score is a sum of thousands of
// log-sum-exps, all off to that side, so it is put right where the weights are summed.
constexpr float kWeightsLow = 4.8e-8f;

// log2(e) / T and 1 / T, each as two floats.
struct Temper {
    float hi, lo;
    Two inv;
};

// The others' sum s_o relative to m_o (-inf: there are none, or all are -inf), and the
// token's logit.
DLM_HD TokenRow token_row(float m_o, float s_o, float z_a, const Temper& c) {
    TokenRow t;
    const bool top = z_a >= m_o;  // the token is at the maximum
    t.m = top ? z_a : m_o;
    const float low = top ? m_o : z_a;
    const Two d = two_sum(t.m, -low);  // the distance to the other one
    const float far = d.hi < INFINITY || d.hi != d.hi ? times_exp2(top ? s_o : 1.f, d.hi, d.lo, c.hi, c.lo) : 0.f;
    const float others = top ? far : s_o;
    const float total = top ? 1.f + others : far + others;
    // (total is 0 where nothing but -inf is)
    t.ok = is_finite(t.m) && s_o >= 0.f && total > 0.f && total < INFINITY && low == low;
    t.inv = 1.f / total;
    t.away = others * t.inv;
    Two ln = top && others < 0.5f ? Two{log1pf(others), 0.f} : ln_split(total);
    ln.lo = fmaf(kWeightsLow, t.away, ln.lo);
    t.logp = minus(ln);
    if (!top) {
        Two y = two_prod(d.hi, c.inv.hi);
        y.lo += is_finite(y.hi) ? fmaf(d.hi, c.inv.lo, d.lo * c.inv.hi) : 0.f;
        t.logp = plus(minus(y), t.logp);
    }
    t.ln = ln;
    if (!t.ok) {
        t.inv = t.away = f32_nan();
        t.logp = t.ln = Two{f32_nan(), 0.f};
    }
    return t;
}
// The row's log-sum-exp.
DLM_HD float token_lse(const TokenRow& t, const Temper& c) {
    Two y = two_prod(t.m, c.inv.hi);
    y.lo += is_finite(y.hi) ? t.m * c.inv.lo : 0.f;
    return rounded(plus(y, t.ln));
}

// e^y - 1 - y without its cancellation near 0.
DLM_HD float exp_past_line(float y) {
    if (!(fabsf(y) < 1.f)) {
        const float e = expm1f(y);
        return e == INFINITY ? e : e - y;
    }
    // y^2 (1/2! + y/3! + y^2/4! + ...), up to y^11/13!: the next term is below 2^-36
    float r = 1.f / 6227020800.f;
    r = fmaf(y, r, 1.f / 479001600);
    r = fmaf(y, r, 1.f / 39916800);
    r = fmaf(y, r, 1.f / 3628800);
    r = fmaf(y, r, 1.f / 362880);
    r = fmaf(y, r, 1.f / 40320);
    r = fmaf(y, r, 1.f / 5040);
    r = fmaf(y, r, 1.f / 720);
    r = fmaf(y, r, 1.f / 120);
    r = fmaf(y, r, 1.f / 24);
    r = fmaf(y, r, 1.f / 6);
    r = fmaf(y, r, 0.5f);
    return y * y * r;
}

// A loss and its derivative by the token's log-probability (or the score difference).
struct LossSlope {
    float loss, slope;
};

// A loss or a derivative that is not finite: the gradient is NaN.
DLM_HD LossSlope flagged(LossSlope x) {
    if (!is_finite(x.loss) || !is_finite(x.slope)) x.slope = f32_nan();
    return x;
}

// a - b and b - a of ln p and another log-probability.
DLM_HD float less(Two a, float b) {
    const Two s = two_sum(a.hi, -b);
    return s.hi + (is_finite(s.hi) ? s.lo + a.lo : 0.f);
}

DLM_HD LossSlope policy_row(const PolicyRule& p, Two logp, float weight, float advantage, bool has_old, float old_logp,
                            float ref_logp) {
    const float rho = has_old ? expf(less(logp, old_logp)) : 1.f;
    const float a = advantage;
    float gain = rho * a, slope = gain;
    if (a > 0.f && rho > p.hi) {
        gain = p.hi * a;
        slope = 0.f;
    } else if (a < 0.f && rho < p.lo) {
        gain = p.lo * a;
        slope = 0.f;
    } else if (a < 0.f && p.dual > 0.f && rho > p.dual) {
        gain = p.dual * a;
        slope = 0.f;
    } else if (a == 0.f && !(rho != rho)) {
        gain = slope = 0.f;  // also of a ratio beyond a float's range
    }
    LossSlope r{-gain, -slope};
    // (no ratio of its own: logp counts as old, and a row without one has no loss)
    if (!has_old && !(logp.hi > -INFINITY)) r.loss = r.slope = f32_nan();
    if (p.kl_weight != 0.f) {
        const float y = -less(logp, ref_logp);
        float kl, d;
        if (p.kl == DLM_KL_K1) {
            kl = -y;
            d = 1.f;
        } else if (p.kl == DLM_KL_K2) {
            kl = 0.5f * y * y;
            d = -y;
        } else {
            kl = exp_past_line(y);
            d = -expm1f(y);
        }
        r.loss = fmaf(p.kl_weight, kl, r.loss);
        r.slope = fmaf(p.kl_weight, d, r.slope);
    }
    r.loss *= weight;
    r.slope *= weight;
    return flagged(r);
}

// ln(1 + e^x)
DLM_HD float softplus(float x) { return log1pf(expf(-fabsf(x))) + fmaxf(x, 0.f); }
// 1 / (1 + e^-x)
DLM_HD float sigmoid(float x) {
    const float e = expf(-fabsf(x));
    return (x >= 0.f ? 1.f : e) / (1.f + e);
}

// A pair's loss, and its derivative by the difference of the two scores.
DLM_HD LossSlope preference_pair(const PreferenceRule& p, double chosen, double rejected, float margin, float weight) {
    const double h64 = p.beta * (chosen - rejected) - (double)margin;
    const float h = (float)h64;
    LossSlope r;
    if (p.kind == DLM_PREF_HINGE) {
        const float short_of = (float)(1.0 - h64);
        r.loss = short_of > 0.f ? short_of : (h != h ? h : 0.f);
        r.slope = short_of > 0.f ? -(float)p.beta : (h != h ? h : 0.f);
    } else if (p.kind == DLM_PREF_IPO) {
        const double x = (h64 - 0.5) / p.beta;
        r.loss = (float)(x * x);
        r.slope = (float)(2.0 * x);
    } else {
        // (a smoothing of 0 leaves its side out: 0 times an infinite loss is NaN)
        r.loss = p.smooth < 1.f ? (1.f - p.smooth) * softplus(-h) : 0.f;
        r.slope = -(1.f - p.smooth) * sigmoid(-h);
        if (p.smooth > 0.f) {
            r.loss += p.smooth * softplus(h);
            r.slope += p.smooth * sigmoid(h);
        }
        r.slope *= (float)p.beta;
    }
    r.loss *= weight;
    r.slope *= weight;
    return flagged(r);
}

}  // namespace dlm
