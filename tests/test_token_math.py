"""The arithmetic of the losses over given tokens (csrc/token_math.cuh) compiled for
the host and compared with long double.

Bounds: every float operation is off by at most 2^-24 of its result, and the host's
expf, logf, log1pf and expm1f by an ulp (2^-23)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r'''
#include "token_math.cuh"
#include <cstdio>
#include <cstdlib>
using namespace dlm;
static double off(double got, long double want) { return (double)(fabsl(got - want) / fabsl(want)); }
int main() {
    srand48(3);
    double ln = 0, line = 0, logp = 0, away = 0, pol = 0, pair = 0;
    for (long i = 0; i < 400000; ++i) {
        // ln x of 1 .. 2^24: one ulp of a logarithm of at most ln 2 / 2, absolute
        const float x = (float)exp(drand48() * 16.6);
        ln = fmax(ln, (double)fabsl((long double)ln_split(x).hi + ln_split(x).lo - logl((long double)x)));
        // e^y - 1 - y, both sides of 1
        const float y = (float)((drand48() - 0.5) * (i % 2 ? 12 : 2) * exp(-drand48() * (i % 3 ? 0 : 20)));
        if (y != 0) line = fmax(line, off(exp_past_line(y), expm1l((long double)y) - (long double)y));
        // a token at the maximum and below it, the others' sum from 2^-60 to 2^20
        const float m_o = (float)(drand48() * 8), z = m_o + (float)((drand48() - 0.5) * (i % 2 ? 40 : 1));
        const float s_o = (float)exp((drand48() - 0.75) * 50) + (i % 2 ? 1.f : 0.f);
        const double inv_t = i % 7 ? 1.0 : i % 2 ? 5.0 : 1.0 / 0.7;
        const float m = fmaxf(m_o, z);
        const double l2 = 1.4426950408889634 * inv_t;
        const float hi = nextafterf((float)l2, 0.f), lo = (float)(l2 - hi);
        const Temper temper{hi, lo, Two{(float)inv_t, (float)(inv_t - (float)inv_t)}};
        const TokenRow t = token_row(m_o, s_o, z, temper);
        const long double lp = (long double)t.logp.hi + t.logp.lo;
        // (the weights that s_o is the sum of are taken for this much too small)
        const long double a = expl(((long double)z - m) * inv_t),
                          o = (long double)s_o * (1 + (long double)kWeightsLow) * expl(((long double)m_o - m) * inv_t);
        const long double want = z >= m_o ? -log1pl(o) : ((long double)z - m) * inv_t - logl(a + o);
        if (o < 1.2e-38L) continue;  // below a normal float
        logp = fmax(logp, (double)(fabsl(lp - want) / fmaxl(fabsl(want) * 4, z >= m_o && o < 0.5L ? 0.L : 1.L)));
        away = fmax(away, off(t.away, o / (a + o)));
        if (!t.ok) return 2;
        // the policy: loss and slope relative to what they are sums of
        const PolicyRule p{0.8f, 1.28f, i % 4 ? 0.f : 3.f, i % 5 ? 0.1f : 0.f, (int)(1 + i % 3)};
        const float A = (float)(drand48() * 4 - 2), old = (float)(lp + drand48() - 0.5), ref = (float)(lp + drand48() - 0.5);
        const LossSlope l = policy_row(p, t.logp, 1.5f, A, true, old, ref);
        const long double rho = expl(lp - old), yy = ref - lp;
        if (fabsl(rho - p.lo) < 1e-5L || fabsl(rho - p.hi) < 1e-5L || fabsl(rho - 3) < 1e-5L) continue;
        long double gain = rho * A, slope = gain, c = rho < p.lo ? p.lo : rho > p.hi ? p.hi : rho;
        if (c * A < gain) gain = c * A, slope = 0;
        if (p.dual && A < 0 && gain < p.dual * A) gain = p.dual * A, slope = 0;
        const long double kl = p.kl == 1 ? -yy : p.kl == 2 ? yy * yy / 2 : expm1l(yy) - yy;
        const long double d = p.kl == 1 ? 1 : p.kl == 2 ? -yy : -expm1l(yy);
        const long double size = fabsl(gain) + p.kl_weight * fabsl(kl), tall = fabsl(slope) + p.kl_weight * fabsl(d);
        pol = fmax(pol, (double)(fabsl(l.loss / 1.5L - (p.kl_weight * kl - gain)) / size));
        if (tall > 0) pol = fmax(pol, (double)(fabsl(l.slope / 1.5L - (p.kl_weight * d - slope)) / tall));
        // the pair
        const PreferenceRule r{i % 2 ? 0.1 : 1.0, i % 3 ? 0.f : 0.125f, i % 3 ? (int)(i % 3) : 0};
        const double u = (drand48() - 0.5) * 60, v = (drand48() - 0.5) * 60;
        const float g = (float)drand48();
        const LossSlope q = preference_pair(r, u, v, g, 2.f);
        const long double h = (long double)r.beta * ((long double)u - v) - g, b = r.beta;
        long double w, k, part = 0;
        if (r.kind == DLM_PREF_HINGE) {
            if (fabsl(1 - h) < 1e-5L) continue;
            w = h < 1 ? 1 - h : 0, k = h < 1 ? -b : 0;
        } else if (r.kind == DLM_PREF_IPO) {
            w = (h - 0.5L) / b * ((h - 0.5L) / b), k = 2 * (h - 0.5L) / b;
            if (fabsl(h - 0.5L) < 1e-6L) continue;
        } else {
            const long double s = r.smooth;
            w = (1 - s) * log1pl(expl(-h)) + s * log1pl(expl(h));
            k = b * (s / (1 + expl(-h)) - (1 - s) / (1 + expl(h)));
            part = b * (s / (1 + expl(-h)) + (1 - s) / (1 + expl(h)));
        }
        // (h itself, as a float, is off by 2^-24 of up to 61, and so is e^h relatively)
        if (w != 0) pair = fmax(pair, off(q.loss / 2, w) / (1 + fabsl(h) / 4));
        if (k != 0) pair = fmax(pair, (double)(fabsl(q.slope / 2.L - k) / (part ? part : fabsl(k))) / (double)(1 + fabsl(h) / 4));
    }
    printf("ln %.3g line %.3g logp %.3g away %.3g policy %.3g pair %.3g\n", ln, line, logp, away, pol, pair);
    const float u = 5.9604645e-8f;  // 2^-24
    // ln: half of the values' ulp (|.| <= 0.35: 2^-26) and logf's; line: series of 13 roundings or expm1f - y;
    // logp: of o (5 roundings: e^n and its product) and log1pf, a quarter of it, or absolute; away: 10 roundings; policy: expf and 6; pair: 8 and e^h's
    int bad = ln > u || line > 8 * u || logp > 4 * u || away > 10 * u || pol > 10 * u || pair > 12 * u;
    // what is not finite
    const LossSlope n1 = policy_row(PolicyRule{0.8f, 1.2f, 0.f, 0.f, 1}, Two{-INFINITY, 0.f}, 1.f, -2.f, true, -3.f, 0.f);
    bad |= n1.loss != 1.6f || n1.slope != 0.f;                                     // ratio 0, clipped from below
    const LossSlope n2 = policy_row(PolicyRule{0.8f, 1.2f, 0.f, 0.f, 1}, Two{-1.0, 0.f}, 1.f, 0.f, true, -200.f, 0.f);
    bad |= n2.loss != 0.f || n2.slope != 0.f;                                      // advantage 0, ratio beyond a float
    const LossSlope n3 = policy_row(PolicyRule{0.8f, 1.2f, 0.f, 0.1f, 3}, Two{-INFINITY, 0.f}, 1.f, 1.f, true, -3.f, -2.f);
    bad |= n3.loss != INFINITY || n3.slope == n3.slope;
    const LossSlope n4 = policy_row(PolicyRule{0.8f, 1.2f, 0.f, 0.f, 1}, Two{NAN, 0.f}, 1.f, 1.f, true, -3.f, 0.f);
    bad |= n4.loss == n4.loss || n4.slope == n4.slope;
    const LossSlope n5 = policy_row(PolicyRule{0.f, INFINITY, 0.f, 0.f, 1}, Two{-1.0, 0.f}, 1.f, 3.f, true, -3.f, 0.f);
    bad |= fabsf(n5.loss + 22.167168f) > 1e-5f;                                    // no clip
    const LossSlope n6 = policy_row(PolicyRule{0.8f, 1.2f, 0.f, 0.f, 1}, Two{-7.0, 0.f}, 2.f, 3.f, false, 0.f, 0.f);
    bad |= n6.loss != -6.f || n6.slope != -6.f;                                    // the rollout's own policy
    const LossSlope p1 = preference_pair(PreferenceRule{1.0, 0.f, 0}, -INFINITY, 0.0, 0.f, 1.f);
    bad |= p1.loss != INFINITY || p1.slope == p1.slope;
    const LossSlope p2 = preference_pair(PreferenceRule{1.0, 0.f, 0}, 0.0, -INFINITY, 0.f, 1.f);
    bad |= p2.loss != 0.f || p2.slope != 0.f;
    const LossSlope p3 = preference_pair(PreferenceRule{1.0, 0.f, 1}, NAN, 0.0, 0.f, 1.f);
    bad |= p3.loss == p3.loss || p3.slope == p3.slope;
    const LossSlope p4 = preference_pair(PreferenceRule{1.0, 0.f, 1}, 1.0, 0.0, 0.f, 1.f);
    bad |= p4.loss != 0.f || p4.slope != 0.f;                                      // the hinge's corner
    const LossSlope p5 = preference_pair(PreferenceRule{1.0, 1.f, 0}, -INFINITY, 0.0, 0.f, 1.f);
    bad |= p5.loss != 0.f || p5.slope != 0.f;                                      // labels turned round
    const Temper one{1.44269502f, 1.93e-8f, Two{1.f, 0.f}};
    const TokenRow r1 = token_row(-INFINITY, 0.f, 3.f, one);
    bad |= !r1.ok || rounded(r1.logp) != 0.f || r1.away != 0.f || token_lse(r1, one) != 3.f;            // the only token
    const TokenRow r2 = token_row(-3.4028235e38f, 0.f, -INFINITY, one);
    bad |= r2.ok || r2.logp.hi == r2.logp.hi || r2.inv == r2.inv;                        // nothing but -inf
    const TokenRow r3 = token_row(1.f, 2.f, -INFINITY, one);
    bad |= !r3.ok || rounded(r3.logp) != -INFINITY || r3.away != 1.f;
    const TokenRow r4 = token_row(1.f, NAN, 0.f, one), r5 = token_row(1.f, 1.f, NAN, one),
                   r6 = token_row(INFINITY, 1.f, 0.f, one), r7 = token_row(1.f, 1.f, INFINITY, one);
    const TokenRow r8 = token_row(0.f, 1.f, 2000.f, one), r9 = token_row(2000.f, 1.f, 0.f, one);
    bad |= rounded(r8.logp) != 0.f || r8.away != 0.f || r9.away != 1.f || rounded(r9.logp) > -2000.f || rounded(r9.logp) < -2000.001f;
    bad |= r4.ok || r5.ok || r6.ok || r7.ok;
    return bad;
}
'''


@pytest.mark.parametrize("flags", [[], ["-ffp-contract=off"]])
def test_token_math_against_long_double(tmp_path, flags):
    src = tmp_path / "t.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "t"
    subprocess.run(["g++", "-O1", "-std=c++17", *flags, "-I", os.path.join(ROOT, "diffusion_decoding_token_gb300", "csrc"),
                    "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
