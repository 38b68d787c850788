"""64-bit numpy restatements of the top-logit, sampling and distillation
operators, written from their definitions in include/dlm.h."""
import math

import numpy as np
import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rows(n, vocab, kind, seed, sigma=2.0, boosted=0.6, pad=0):
    """Logit rows on the CPU, [n, vocab] at a stride of whole 16-byte vectors
    (plus ``pad`` vectors): N(0, sigma^2), some rows with one raised token."""
    g = np.random.default_rng(seed)
    z = g.normal(0.0, sigma, (n, vocab)).astype(np.float32)
    if vocab > 1:
        for r in np.nonzero(g.random(n) < boosted)[0]:
            z[r, g.integers(vocab)] = math.log(vocab) + sigma * sigma / 2 + g.uniform(2, 10)
    epv = 4 if kind == "f32" else 8
    wide = torch.full((n, ((vocab + epv - 1) // epv + pad) * epv), float("nan"), dtype=TYPES[kind])
    wide[:, :vocab] = torch.from_numpy(z).to(TYPES[kind])
    return wide[:, :vocab]


def host(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def order(row):
    """Positions of the finite logits, largest first, ties to the lower one."""
    o = np.argsort(-row, kind="stable")
    return o[row[o] > -np.inf]


def topk(row, k, temperature=1.0):
    o = order(row)[:k]
    ids = np.full(k, -1, np.int64)
    values = np.full(k, -np.inf)
    ids[:len(o)], values[:len(o)] = o, row[o]
    y = row / np.float64(np.float32(temperature))
    return values, ids, y.max() + math.log(np.exp(y - y.max()).sum())


def kept(row, temperature, top_k, top_p, min_p):
    """(positions that stay in vocabulary order, their weights)."""
    o = order(row)
    if temperature == 0:
        return o[:1], np.ones(1)
    t, p, least = (float(np.float32(x)) for x in (temperature, top_p, min_p))
    if top_k > 0:
        o = o[:top_k]
    w = np.exp((row[o] - row[o[0]]) / t)
    ends = np.cumsum(w)
    n = len(o)
    if p < 1:
        n = 1 + int(np.searchsorted(ends[:-1], p * ends[-1], side="left"))
    if least > 0:
        n = min(n, int((w >= least).sum()))
    at = np.sort(o[:n])
    return at, np.exp((row[at] - row[o[0]]) / t)


def sample(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    at, w = kept(row, temperature, top_k, top_p, min_p)
    ends = np.cumsum(w)
    j = min(int(np.searchsorted(ends, float(np.float32(u)) * ends[-1], side="right")), len(at) - 1)
    return int(at[j]), w[j] / ends[-1]


def distill(row, ids, teacher, weight=1.0, temperature=1.0, teacher_lse=None):
    """(loss, gradient, per-token error scale of the gradient): the scale is
    what a relative error of 1 in q (more for far tokens, see below), p and
    the factor of the unlisted tokens together would change, for tolerances."""
    t = float(temperature)
    held = (ids >= 0) & (ids < len(row))
    ids, a = ids[held], teacher[held] / t
    y = row / t
    log_q = y - (y.max() + math.log(np.exp(y - y.max()).sum()))
    q = np.exp(log_q)
    # q = 2^-e / sum, e = (max - s) log2(e) / T: relative error 2^-22 (ex2),
    # 2.1 2^-24 e (three roundings of e, times ln 2) and 2^-18 (the sum), which
    # is 2^-17 (0.53 + 0.0165 e); in units of 2^-17.  Below 2^-126 of the
    # largest weight ex2 gives 0 for what is not (1 / sum <= 1): 2^-126 more
    off = np.maximum(1.0, 0.53 + 0.0165 * np.minimum((y.max() - y) / math.log(2), 1e4))
    if teacher_lse is None:
        if len(a) == 0 or a.max() == -np.inf:
            return 0.0, np.zeros_like(row), np.zeros_like(row)
        log_p = a - (a.max() + math.log(np.exp(a - a.max()).sum()))
    else:
        log_p = np.minimum(a - teacher_lse, 0.0)
    p = np.exp(log_p)
    loss = sum(p[j] * (log_p[j] - log_q[ids[j]]) for j in range(len(p)) if p[j] > 0)
    slope, scale = q.copy(), q * off + 2.0 ** (17 - 126)
    if teacher_lse is not None:
        out = np.ones(len(row), bool)
        out[ids] = False
        p_rest, q_rest = max(0.0, 1 - p.sum()), q[out].sum()
        if p_rest > 0:
            loss += p_rest * (math.log(p_rest) - (math.log(q_rest) if q_rest > 0 else -math.inf))
        if q_rest > 0:
            slope[out] *= 1 - p_rest / q_rest
            scale[out] *= 1 + p_rest / q_rest
    np.subtract.at(slope, ids, p)
    np.add.at(scale, ids, p)
    return weight * loss, weight / t * slope, abs(weight) / t * scale
