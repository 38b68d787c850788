"""64-bit restatements of the losses over given tokens, written from their
definitions in include/dlm.h."""
import math

import numpy as np


def row(z, token, temperature=1.0):
    """(ln q_token, ln sum exp(z / T), q, 1 - q_token) of a row of 64-bit logits.
    1 - q_token is the others' share, not a difference."""
    y = z / float(temperature)
    top = y.max()
    w = np.exp(y - top)
    lse = top + math.log(w.sum())
    others = w.copy()
    others[token] = 0.0
    rest = math.fsum(others)
    if y[token] == top:
        logp = -math.log1p(rest)
    else:
        logp = y[token] - lse
    return logp, lse, w / w.sum(), rest / (rest + w[token])


def row_grad(z, token, slope, temperature=1.0):
    """slope * d ln q_token / d z, and the magnitudes whose relative error it has:
    q's error grows with a token's distance from the maximum (see off below)."""
    t = float(temperature)
    _, _, q, away = row(z, token, t)
    g = -q
    g[token] = away
    # q = 2^-e / sum: 2^-22 (ex2), three roundings of e at 2^-24 each times ln 2, and
    # 2^-18 (the sum), in units of 2^-17; below 2^-126 ex2 gives 0
    off = np.maximum(1.0, 0.53 + 0.0165 * np.minimum((z.max() - z) / t / math.log(2), 1e4))
    scale = np.abs(g) * off + 2.0 ** (17 - 126)
    return slope / t * g, abs(slope) / t * scale


def policy(logp, advantage, old, ref, clip_low, clip_high, dual_clip, kl_weight, kl):
    """(loss, d loss / d logp) of a row of weight 1."""
    a = float(advantage)
    rho = 1.0 if old is None else math.exp(logp - old)
    lo, hi = 1.0 - clip_low, 1.0 + clip_high
    free, cut = rho * a, min(max(rho, lo), hi) * a
    gain, slope = (free, free) if free <= cut else (cut, 0.0)
    if dual_clip and a < 0 and gain < dual_clip * a:
        gain, slope = dual_clip * a, 0.0
    loss, slope = -gain, -slope
    if kl_weight:
        y = ref - logp
        k, d = {"k1": (-y, 1.0), "k2": (y * y / 2, -y), "k3": (math.expm1(y) - y, -math.expm1(y))}[kl]
        loss, slope = loss + kl_weight * k, slope + kl_weight * d
    return loss, slope


def pair(chosen, rejected, margin, beta, kind, smooth):
    """(loss, d loss / d (chosen - rejected)) of a pair of weight 1."""
    h = beta * (chosen - rejected) - margin
    if kind == "hinge":
        return max(0.0, 1.0 - h), (-beta if h < 1 else 0.0)
    if kind == "ipo":
        return ((h - 0.5) / beta) ** 2, 2.0 * (h - 0.5) / beta
    soft = lambda v: math.log1p(math.exp(-abs(v))) + max(v, 0.0)  # noqa: E731
    sig = lambda v: (1.0 if v >= 0 else math.exp(v)) / (1.0 + math.exp(-abs(v)))  # noqa: E731
    return (1 - smooth) * soft(-h) + smooth * soft(h), beta * (smooth * sig(h) - (1 - smooth) * sig(-h))
