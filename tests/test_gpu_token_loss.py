"""Log-probabilities of given tokens, the policy loss and the preference loss, with
their gradients, against 64-bit numpy and against differences.

Tolerances.  The sum of all other tokens' weights comes from 32-bit sums within 2^-18
(ex2 2^-22, an exponent of up to ~20 rounded three times at 2^-24, additions).  With
it ln p = -ln(1 + others / own) is off by at most 2^-18 (1 - p), the log-sum-exp by
2^-18, and each by its own rounding (2^-24, and 2^-23 for the logarithm).  A loss is
off by what its derivative makes of that (d below) and 2^-20 of the terms that it is
the sum of (expf, expm1f and log1pf at 2 ulps, a handful of float operations); its
derivative likewise.  A gradient element is off by 2^-17 of itself (q 2^-18 of the sum,
the rest as in token_ref.row_grad), by the derivative's error, and by half a step of its type.
"""
import math

import numpy as np
import pytest
import torch

import row_ref
import token_ref as ref

pytestmark = pytest.mark.gpu
F32 = np.float32


@pytest.fixture(scope="module")
def dlm():
    import diffusion_decoding_token_gb300 as d
    d.lib()
    return d


def on_gpu(z):
    """The same rows at the same stride, NaN between them."""
    wide = torch.full((z.shape[0], z.stride(0) if z.shape[0] > 1 else (z.shape[1] + 7) // 8 * 8), float("nan"),
                      dtype=z.dtype, device="cuda")
    d = wide[:, :z.shape[1]]
    d.copy_(z)
    return d


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def half_step(x, dtype):
    f = torch.finfo(dtype)
    return np.maximum(np.abs(x) * f.eps / 2, f.tiny * f.eps / 2)


def tokens_of(z, seed):
    """A token per row: the largest, one at random, or the one before the largest."""
    g = np.random.default_rng(seed)
    zz = row_ref.host(z)
    top = zz.argmax(1)
    pick = g.integers(0, 3, len(zz))
    return np.where(pick == 0, top, np.where(pick == 1, g.integers(0, z.shape[1], len(zz)), np.maximum(top - 1, 0))).astype(np.int32)


def d_logp(away, logp):
    return 2.0 ** -18 * away + 2.0 ** -23 * abs(logp)


def near(got, want, tol, what):
    if math.isnan(want):
        assert math.isnan(got), what
    elif math.isinf(want):
        assert got == want, (what, got, want)
    else:
        assert abs(got - want) <= tol, (what, got, want, tol)


def check_grad(got, z, token, slope, d_slope, temperature, dtype, what):
    want, scale = ref.row_grad(z, token, slope, temperature)
    unit, _ = ref.row_grad(z, token, 1.0, temperature)
    tol = scale * 2.0 ** -17 + d_slope * np.abs(unit) + half_step(want, dtype) * 1.01
    bad = ~(np.abs(row_ref.host(got) - want) <= tol)
    assert not bad.any(), (what, np.nonzero(bad)[0][:5], row_ref.host(got)[bad][:5], want[bad][:5], tol[bad][:5])


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- log-probabilities ------------------------------------------------------

def check_logprob(dlm, z, token, temperature=1.0, weights=None, up=None, status_want=0):
    n, vocab = z.shape
    d, t, status = on_gpu(z), cuda(token), dlm.new_status()
    kw = dict(temperature=temperature, status=status)
    out = dlm.row_logprob(d, t, with_state=True, **kw)
    g1 = dlm.row_logprob_grad(d, t, out.state, cuda(up), **kw)
    logp2, g2 = dlm.row_logprob_step(d, t, cuda(weights), **kw)
    inplace = on_gpu(z)
    logp3, g3 = dlm.row_logprob_step(inplace, t, cuda(weights), grad=inplace, **kw)
    assert int(status.item()) == status_want
    assert same_bits(logp2, logp3) and same_bits(g2, g3)
    zz = row_ref.host(z)
    for r in range(n):
        w = 1.0 if weights is None else float(weights[r])
        u = 1.0 if up is None else float(up[r])
        if not 0 <= token[r] < vocab:
            assert float(out.logp[r]) == float(out.lse[r]) == float(logp2[r]) == 0.0
            assert (g1[r] == 0).all() and (g2[r] == 0).all()
            continue
        logp, lse, _, away = ref.row(zz[r], token[r], temperature)
        near(float(out.logp[r]), logp, d_logp(away, logp), ("logp", r))
        near(float(out.lse[r]), lse, 2.0 ** -18 + 2.0 ** -23 * abs(lse), ("lse", r))
        near(float(logp2[r]), logp if w else 0.0, d_logp(away, logp), ("logp of the step", r))
        for got, slope in ((g1, u), (g2, w)):
            if slope == 0:
                assert (got[r] == 0).all()
            else:
                check_grad(got[r], zz[r], token[r], slope, 2.0 ** -22 * abs(slope), temperature, z.dtype, r)


SHAPES = [(1, 1), (2, 9), (3, 130), (4, 1025), (5, 5003), (2, 32003), (330, 2051), (700, 257), (2, 126464), (41, 16383), (3, 262147)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,vocab", SHAPES)
def test_logprob(dlm, kind, n, vocab):
    z = row_ref.rows(n, vocab, kind, n + vocab, pad=n % 2)
    check_logprob(dlm, z, tokens_of(z, n))


@pytest.mark.parametrize("kind,n,vocab", [("f32", 2, 500001), ("bf16", 1, 1000003), ("f32", 1, 1048575), ("f16", 3, 600001)])
def test_logprob_of_long_rows(dlm, kind, n, vocab):
    z = row_ref.rows(n, vocab, kind, vocab)
    check_logprob(dlm, z, tokens_of(z, n))


@pytest.mark.parametrize("kind,rows,vocab", [("bf16", 900, 20011), ("f32", 401, 30001)])
def test_more_rows_than_run_at_once(dlm, kind, rows, vocab):
    # all rows equal: every row has to have the same answer
    z = row_ref.rows(1, vocab, kind, 77)
    wide = torch.empty((rows, (vocab + 7) // 8 * 8), dtype=z.dtype)
    wide[:, :vocab] = z
    d = on_gpu(wide[:, :vocab])
    t = torch.full((rows,), int(tokens_of(z, 1)[0]), dtype=torch.int32, device="cuda")
    w = torch.arange(rows, device="cuda", dtype=torch.float32) % 5  # every fifth is not read
    logp, grad = dlm.row_logprob_step(d, t, w)
    check_grad(grad[1], row_ref.host(z)[0], int(t[0]), 1.0, 2.0 ** -22, 1.0, z.dtype, "row 1")
    assert (logp == torch.where(w > 0, logp[1], 0.0)).all()
    for v in range(5):
        assert same_bits(grad[v::5], grad[v].expand(grad[v::5].shape))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("temperature", [0.3, 2.0, 17.0])
def test_logprob_temperature_weights_and_tokens_that_are_none(dlm, kind, temperature):
    n, vocab = 13, 4001
    g = np.random.default_rng(3)
    z = row_ref.rows(n, vocab, kind, 5)
    token = tokens_of(z, 2)
    token[[1, 8]] = -1
    token[3] = -2 ** 31
    weights, up = (g.normal(0, 1, n).astype(F32) for _ in range(2))
    weights[[2, 7]] = 0.0
    up[5] = 0.0
    check_logprob(dlm, z, token, temperature, weights, up)


def test_tokens_outside_the_vocabulary(dlm):
    z = row_ref.rows(4, 1000, "bf16", 6)
    token = np.array([5, 1000, 2 ** 31 - 1, 999], np.int32)
    check_logprob(dlm, z, token, status_want=dlm.DEV_BAD_INDEX)


@pytest.mark.parametrize("temperature", [1e-4, 1e30])
def test_extreme_temperatures(dlm, temperature):
    z = row_ref.rows(5, 3001, "f32", 8)
    token = tokens_of(z, 1)
    out = dlm.row_logprob(on_gpu(z), cuda(token), temperature=temperature)
    _, grad = dlm.row_logprob_step(on_gpu(z), cuda(token), temperature=temperature)
    for r, row in enumerate(row_ref.host(z)):
        logp, lse, _, away = ref.row(row, token[r], temperature)
        near(float(out.logp[r]), logp, d_logp(away, logp), r)
        near(float(out.lse[r]), lse, 2.0 ** -18 + 2.0 ** -23 * abs(lse), r)
        check_grad(grad[r], row, token[r], 1.0, 2.0 ** -22, temperature, z.dtype, r)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gap", [12.0, 30.0, 80.0, 2000.0])
def test_rows_that_are_sure(dlm, kind, gap):
    # the token far above the rest: ln p and 1 - p keep their digits; and far below
    n, vocab = 6, 2500
    z = row_ref.rows(n, vocab, kind, 9, boosted=0.0)
    token = np.arange(n, dtype=np.int32) * 300
    for r in range(n):
        z[r, token[r]] = gap if r % 2 == 0 else -gap
    z[4, 7] = z[4, token[4]]  # two tokens at the maximum
    check_logprob(dlm, z, token)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_masked_rows(dlm, kind):
    z = row_ref.rows(6, 3000, kind, 7)
    token = np.array([3, 5, 2999, 11, 20, 2000], np.int32)
    z[0, 1500:] = -math.inf
    z[1] = -math.inf
    z[1, 5] = 1.0                      # only the token is left: ln p = 0, gradient 0
    z[2] = torch.finfo(z.dtype).min
    z[2, 2999] = 0.0                   # masked with the type's lowest value
    z[3] = torch.finfo(z.dtype).min    # nothing but the lowest value: uniform
    z[4, 20] = -math.inf               # the token itself is masked
    z[5, 100:] = torch.finfo(z.dtype).min
    d, status = on_gpu(z), dlm.new_status()
    out = dlm.row_logprob(d, cuda(token), with_state=True, status=status)
    g1 = dlm.row_logprob_grad(d, cuda(token), out.state)
    _, g2 = dlm.row_logprob_step(d, cuda(token), status=status)
    assert int(status.item()) == 0
    zz = row_ref.host(z)
    for r in (0, 1, 2, 3, 5):
        logp, lse, _, away = ref.row(zz[r], token[r])
        near(float(out.logp[r]), logp, d_logp(away, logp), r)
        near(float(out.lse[r]), lse, 2.0 ** -18 + 2.0 ** -23 * abs(lse), r)
        for g in (g1, g2):
            check_grad(g[r], zz[r], token[r], 1.0, 2.0 ** -22, 1.0, z.dtype, r)
    assert float(out.logp[4]) == -math.inf
    other = zz[4].copy()
    other[20] = -1e9
    for g in (g1, g2):
        check_grad(g[4], other, 20, 1.0, 2.0 ** -22, 1.0, z.dtype, 4)
        assert (g[0, 1500:] == 0).all() and (g[1] == 0).all()


def test_rows_that_are_not_finite(dlm):
    z = row_ref.rows(6, 2000, "bf16", 8)
    z[0, 11] = math.nan
    z[1, 12] = math.inf
    z[2] = -math.inf
    z[3, 7] = math.nan                 # the token itself
    z[4, 7] = math.inf
    token = np.full(6, 7, np.int32)
    for r in range(5):
        status = dlm.new_status()
        dlm.row_logprob(on_gpu(z[r:r + 1]), cuda(token[:1]), status=status)
        assert int(status.item()) == dlm.DEV_NONFINITE, r
    out = dlm.row_logprob(on_gpu(z), cuda(token), with_state=True)
    logp, grad = dlm.row_logprob_step(on_gpu(z), cuda(token))
    apart = dlm.row_logprob_grad(on_gpu(z), cuda(token), out.state)
    assert torch.isnan(out.logp[:5]).all() and torch.isnan(out.lse[:5]).all() and torch.isnan(logp[:5]).all()
    assert torch.isnan(grad[:5]).all() and torch.isnan(apart[:5]).all()
    assert torch.isfinite(out.logp[5]) and torch.isfinite(grad[5]).all() and torch.isfinite(apart[5]).all()


@pytest.mark.parametrize("gather", [False, True])
def test_picked_rows(dlm, gather):
    n, vocab = 40, 3001
    z = row_ref.rows(n, vocab, "f16", 21)
    every = tokens_of(z, 4)
    index = np.array([39, 3, 17, -1, 0, 40, 22, 2 ** 31 - 1], np.int32)
    m = len(index) if gather else n
    token = np.where((index >= 0) & (index < n), every[np.clip(index, 0, n - 1)], 0).astype(np.int32) if gather else every
    out = dlm.RowLogprob(torch.full((m,), 7.0, device="cuda"), torch.full((m,), 7.0, device="cuda"), None)
    status = dlm.new_status()
    dlm.row_logprob(on_gpu(z), cuda(token), row_index=cuda(index), gather=gather, out=out, status=status)
    assert int(status.item()) == dlm.DEV_BAD_INDEX
    left = set(range(m))
    zz = row_ref.host(z)
    for i, q in enumerate(index):
        if 0 <= q < n:
            o = i if gather else int(q)
            left.discard(o)
            logp, lse, _, away = ref.row(zz[q], every[q])
            near(float(out.logp[o]), logp, d_logp(away, logp), i)
            near(float(out.lse[o]), lse, 2.0 ** -18 + 2.0 ** -23 * abs(lse), i)
    left = sorted(left)
    assert (out.logp[left] == 7.0).all() and (out.lse[left] == 7.0).all()


def test_the_same_row_picked_twice(dlm):
    z = row_ref.rows(9, 20001, "bf16", 23)
    token = tokens_of(z, 4)
    index = np.array([4, 4, 4, 8, 4], np.int32)
    out = dlm.row_logprob(on_gpu(z), cuda(token[index]), row_index=cuda(index), gather=True)
    want = dlm.row_logprob(on_gpu(z), cuda(token))
    near(float(out.logp[0]), float(want.logp[4]), 2.0 ** -17, 0)
    assert (out.logp[[1, 2, 4]] == out.logp[0]).all() and (out.lse[[1, 2, 4]] == out.lse[0]).all()


def test_rows_far_apart(dlm):
    # offsets of elements that pass 2^31
    vocab = 1001
    wide = torch.empty((3, 1 << 30), dtype=torch.bfloat16, device="cuda")
    z = row_ref.rows(3, vocab, "bf16", 30)
    d = wide[:, 4096:4096 + vocab]
    d.copy_(z)
    token = cuda(tokens_of(z, 5))
    logp, grad = dlm.row_logprob_step(d, token, grad=d)
    want_logp, want = dlm.row_logprob_step(on_gpu(z), token)
    assert torch.equal(logp, want_logp) and torch.equal(grad, want)
    del wide


def test_what_lies_past_the_rows_is_left(dlm):
    for vocab in (1003, 20001):
        z = row_ref.rows(5, vocab, "bf16", 11, pad=2)
        token, wide = tokens_of(z, 1), torch.full((5, z.stride(0)), 7.0, dtype=torch.bfloat16, device="cuda")
        token[3] = -1
        dlm.row_logprob_step(on_gpu(z), cuda(token), grad=wide[:, :vocab])
        assert (wide[:, vocab:] == 7.0).all() and not (wide[:, :vocab] == 7.0).any()


# ---- the policy loss --------------------------------------------------------

RULES = [dict(), dict(clip_low=0.2, clip_high=0.28, kl_weight=0.04, kl="k3"), dict(dual_clip=3.0, kl_weight=0.5, kl="k2"),
         dict(clip_low=1.0, clip_high=math.inf, kl_weight=1.0, kl="k1"), dict(clip_low=0.0, clip_high=0.0, dual_clip=1.0)]


def policy_inputs(z, token, seed, temperature=1.0):
    g = np.random.default_rng(seed)
    n = len(token)
    logp = np.array([ref.row(row, max(0, t), temperature)[0] for row, t in zip(row_ref.host(z), token)])
    # ratios away from every border (ln 0.8, ln 1.2, ln 1.28, ln 3 and 0) by far more than they are off
    x = g.choice([-1.5, -0.4, -0.1, 0.1, 0.15, 0.4, 1.5], n)
    old = (logp - x).astype(F32)
    refs = (logp + g.normal(0, 0.5, n)).astype(F32)
    refs[::4] = (logp[::4] + g.normal(0, 1e-3, len(refs[::4]))).astype(F32)
    adv = g.normal(0, 1.5, n).astype(F32)
    adv[::5] = 0.0
    return adv, old, refs


def check_policy(dlm, z, token, rule, temperature=1.0, weights=None, up=None, with_old=True, seed=1):
    n, vocab = z.shape
    adv, old, refs = policy_inputs(z, token, seed, temperature)
    d, t, status = on_gpu(z), cuda(token), dlm.new_status()
    kw = dict(old=cuda(old) if with_old else None, ref=cuda(refs) if rule.get("kl_weight") else None, temperature=temperature,
              weights=cuda(weights), status=status, **rule)
    out = dlm.policy_loss(d, t, cuda(adv), **kw)
    g1 = dlm.policy_grad(d, t, out.state, cuda(up), temperature=temperature, status=status)
    two = dlm.policy_step(d, t, cuda(adv), **kw)
    inplace = on_gpu(z)
    three = dlm.policy_step(inplace, t, cuda(adv), out=dlm.PolicyStep(torch.empty(n, device="cuda"), torch.empty(n, device="cuda"),
                                                                      inplace), **kw)
    assert int(status.item()) == 0
    assert all(same_bits(a, b) for a, b in zip(two, three))
    full = dict(clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_weight=0.0, kl="k3") | rule
    f = {k: (v if isinstance(v, str) else float(F32(v))) for k, v in full.items()}
    zz = row_ref.host(z)
    for r in range(n):
        w = 1.0 if weights is None else float(weights[r])
        u = 1.0 if up is None else float(up[r])
        if not 0 <= token[r] < vocab or w == 0:
            for x in (out.loss, out.logp, two.loss, two.logp):
                assert float(x[r]) == 0.0
            assert (g1[r] == 0).all() and (two.grad[r] == 0).all()
            continue
        logp, _, _, away = ref.row(zz[r], token[r], temperature)
        loss, slope = ref.policy(logp, adv[r], float(old[r]) if with_old else None, float(refs[r]), **f)
        rho, y = math.exp(logp - old[r]) if with_old else 1.0, float(refs[r]) - logp
        cut = min(max(rho, 1 - f["clip_low"]), 1 + f["clip_high"])
        big = (abs(rho) + abs(cut)) * abs(adv[r]) + f["kl_weight"] * (abs(y) + abs(math.expm1(y)))
        d1 = d_logp(away, logp)
        steep = abs(rho * adv[r]) + f["kl_weight"] * max(1.0, math.exp(y))  # |d slope / d logp|
        for got in (out, two):
            near(float(got.logp[r]), logp, d1, ("logp", r))
            near(float(got.loss[r]), w * loss, abs(w) * ((abs(slope) + steep * d1) * d1 + 2.0 ** -20 * big), ("loss", r))
        d_slope = abs(w) * (steep * d1 + 2.0 ** -20 * big)
        for got, k in ((g1, u), (two.grad, 1.0)):
            check_grad(got[r], zz[r], token[r], k * w * slope, abs(k) * d_slope, temperature, z.dtype, r)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("kind,n,vocab", [("f32", 37, 1025), ("bf16", 21, 5003), ("f16", 40, 130), ("bf16", 3, 126464)])
def test_policy(dlm, kind, n, vocab, rule):
    z = row_ref.rows(n, vocab, kind, n + vocab, pad=n % 2)
    check_policy(dlm, z, tokens_of(z, n), rule)


@pytest.mark.parametrize("rule", RULES[:2])
@pytest.mark.parametrize("temperature", [0.6, 1.7])
def test_policy_temperature_weights_and_upstream(dlm, temperature, rule):
    n = 24
    g = np.random.default_rng(5)
    z = row_ref.rows(n, 2003, "f32", 6)
    token = tokens_of(z, 6)
    token[[4, 9]] = -100
    weights, up = (g.normal(0, 1, n).astype(F32) for _ in range(2))
    weights[[1, 2, 23]] = 0.0
    up[7] = 0.0
    check_policy(dlm, z, token, rule, temperature, weights, up)


@pytest.mark.parametrize("rule", RULES[:2])
def test_policy_without_old_is_the_rollouts_own(dlm, rule):
    z = row_ref.rows(17, 3001, "bf16", 7)
    check_policy(dlm, z, tokens_of(z, 7), rule, with_old=False)


def test_policy_of_long_rows(dlm):
    z = row_ref.rows(2, 500001, "f32", 8)
    check_policy(dlm, z, tokens_of(z, 8), RULES[1])


def test_policy_rows_that_are_not_finite(dlm):
    z = row_ref.rows(5, 2000, "f32", 8)
    z[0, 3] = math.nan
    z[1, 7] = -math.inf                # the token: ratio 0, and with a KL term an infinite loss
    token = np.full(5, 7, np.int32)
    adv, old = np.full(5, -1.0, F32), np.full(5, -3.0, F32)
    old[2] = -300.0                    # a ratio beyond a float's range
    adv[3], old[3] = 0.0, -300.0       # which an advantage of 0 makes nothing of
    d, t = on_gpu(z), cuda(token)
    status = dlm.new_status()
    r = dlm.policy_step(d, t, cuda(adv), old=cuda(old), status=status)
    assert int(status.item()) == dlm.DEV_NONFINITE
    assert math.isnan(r.loss[0]) and float(r.loss[1]) == pytest.approx(0.8, rel=1e-6) and float(r.loss[2]) == math.inf
    assert float(r.loss[3]) == 0.0 and math.isfinite(r.loss[4])
    assert torch.isnan(r.grad[0]).all() and (r.grad[1] == 0).all() and torch.isnan(r.grad[2]).all() and (r.grad[3] == 0).all()
    status = dlm.new_status()
    r = dlm.policy_loss(d[1:2], t[:1], cuda(adv[1:2]), old=cuda(old[1:2]), ref=cuda(old[1:2]), kl_weight=0.1, status=status)
    assert float(r.loss[0]) == math.inf and int(status.item()) == dlm.DEV_NONFINITE
    assert torch.isnan(dlm.policy_grad(d[1:2], t[:1], r.state)).all()


def test_policy_gradient_against_differences(dlm):
    # central differences of the 64-bit loss: their error is h^2 / 6 times a third
    # derivative of at most ~4, and 1e-16 / h
    z = row_ref.rows(6, 60, "f32", 10)
    token, rule = tokens_of(z, 10), dict(dual_clip=3.0, kl_weight=0.3, kl="k3")
    adv, old, refs = policy_inputs(z, token, 3, 1.5)
    r = dlm.policy_step(on_gpu(z), cuda(token), cuda(adv), old=cuda(old), ref=cuda(refs), temperature=1.5, **rule)
    h = 1e-4
    for i, row in enumerate(row_ref.host(z)):
        f = lambda x: ref.policy(ref.row(x, token[i], 1.5)[0], adv[i], float(old[i]), float(refs[i]), 0.2, 0.2, 3.0,  # noqa: E731,B023
                                 float(F32(0.3)), "k3")[0]
        for v in range(60):
            e = np.zeros(60)
            e[v] = h
            assert abs(float(r.grad[i, v]) - (f(row + e) - f(row - e)) / (2 * h)) <= 2.0 ** -16 * (1 + abs(adv[i])) * 6 + h * h


# ---- the preference loss ----------------------------------------------------

def check_preference(dlm, z, token, offsets, kind="sigmoid", beta=0.1, smooth=0.0, temperature=1.0, with_ref=True,
                     weights=None, margins=None, pair_weights=None, up=None, seed=2, clean=None, status_want=0):
    n, vocab = z.shape
    offsets = np.asarray(offsets, np.int32)
    pairs = len(offsets) // 2
    zz = row_ref.host(z)
    g = np.random.default_rng(seed)
    rows = [ref.row(zz[r], token[r], temperature) if 0 <= token[r] < vocab else None for r in range(n)]
    refs = np.array([x[0] if x else 0.0 for x in rows]) + g.normal(0, 0.3, n)
    refs = refs.astype(F32)
    d, t, status = on_gpu(z), cuda(token), dlm.new_status()
    kw = dict(ref=cuda(refs) if with_ref else None, beta=beta, kind=kind, label_smoothing=smooth, margins=cuda(margins),
              weights=cuda(weights), pair_weights=cuda(pair_weights), temperature=temperature, status=status)
    out = dlm.preference_loss(d, t, cuda(offsets), **kw)
    g1 = dlm.preference_grad(d, t, out.state, cuda(up), temperature=temperature, status=status)
    two = dlm.preference_step(d, t, cuda(offsets), **kw)
    inplace = on_gpu(z)
    f = lambda k: torch.empty(k, device="cuda")  # noqa: E731
    three = dlm.preference_step(inplace, t, cuda(offsets), out=dlm.PreferenceStep(f(pairs), f(2 * pairs), f(n), inplace),
                                workspace=dlm.preference_workspace(n, pairs, "cuda"), **kw)
    assert int(status.item()) == status_want
    assert all(same_bits(a, b) for a, b in zip(two, three))
    at = offsets if clean is None else np.asarray(clean)
    w = np.ones(n) if weights is None else weights.astype(np.float64)
    b64 = float(F32(beta))
    slope, d_slope = np.zeros(n), np.zeros(n)
    pair_of = np.full(n, -1)
    for i in range(pairs):
        pair_of[at[2 * i]:at[2 * i + 2]] = i
        score, off = [], 0.0
        for s in (2 * i, 2 * i + 1):
            terms = [(w[r] * (rows[r][0] - (float(refs[r]) if with_ref else 0.0)), abs(w[r]) * d_logp(rows[r][3], rows[r][0]))
                     for r in range(at[s], at[s + 1]) if rows[r] and w[r]]
            score.append(math.fsum(x for x, _ in terms))
            one = sum(x for _, x in terms)
            off += one
            for got in (out, two):
                near(float(got.score[s]), score[-1], one + 2.0 ** -23 * abs(score[-1]), ("score", s))
        m = 0.0 if margins is None else float(margins[i])
        pw = 1.0 if pair_weights is None else float(pair_weights[i])
        loss, k = ref.pair(score[0], score[1], m, b64, kind, float(F32(smooth)))
        h = b64 * (score[0] - score[1]) - m
        bend = 2.0 if kind == "ipo" else b64 * b64 / 4       # |l''| by the difference of scores
        # (a float h is off by 2^-24 of itself, which e^h turns into as much of loss and slope)
        tol = abs(pw) * ((abs(k) + bend * off) * off + 2.0 ** -20 * (abs(loss) + abs(h) * abs(k)) + 2.0 ** -24 * abs(h) * b64)
        for got in (out, two):
            near(float(got.loss[i]), pw * loss, tol, ("loss", i))
        for s, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
            for r in range(at[s], at[s + 1]):
                if rows[r]:
                    slope[r] = sign * pw * k * w[r]
                    d_slope[r] = abs(pw * w[r]) * (bend * off + 2.0 ** -20 * (b64 if kind == "sigmoid" else abs(k)) * (1 + abs(h) / 16))
    for r in range(n):
        for got in (out, two):
            if rows[r] is None or not w[r]:
                assert float(got.logp[r]) == 0.0
            else:
                near(float(got.logp[r]), rows[r][0], d_logp(rows[r][3], rows[r][0]), ("logp", r))
        u = 1.0 if up is None else float(up[pair_of[r]])
        for got, f in ((g1, u), (two.grad, 1.0)):
            if slope[r] == 0 and d_slope[r] == 0 or f == 0:
                assert (got[r] == 0).all(), r
            else:
                check_grad(got[r], zz[r], token[r], f * slope[r], abs(f) * d_slope[r], temperature, z.dtype, r)


@pytest.mark.parametrize("pref,smooth", [("sigmoid", 0.0), ("sigmoid", 0.1), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("kind,vocab,offsets", [
    ("f32", 1025, [0, 7, 15]), ("bf16", 3001, [0, 4, 9, 10, 20, 26, 31]), ("f16", 130, [0, 20, 37, 60, 70]),
    ("bf16", 126464, [0, 2, 3])])
def test_preference(dlm, kind, vocab, offsets, pref, smooth):
    z = row_ref.rows(offsets[-1], vocab, kind, vocab, pad=1)
    check_preference(dlm, z, tokens_of(z, 3), offsets, pref, smooth=smooth)


@pytest.mark.parametrize("pref", ["sigmoid", "hinge", "ipo"])
def test_preference_weights_margins_and_upstream(dlm, pref):
    offsets = [0, 9, 12, 20, 33, 34, 40]
    n = 40
    g = np.random.default_rng(8)
    z = row_ref.rows(n, 2003, "f32", 15)
    token = tokens_of(z, 9)
    token[[3, 30]] = -1
    weights = (0.2 + g.random(n)).astype(F32)
    weights[[0, 10, 33]] = 0.0         # the fifth sequence has nothing left
    check_preference(dlm, z, token, offsets, pref, beta=0.5, temperature=0.8, weights=weights,
                     margins=g.random(3).astype(F32), pair_weights=np.array([0.5, 0.0, 2.0], F32),
                     up=np.array([1.5, -1.0, -0.25], F32))


def test_preference_without_a_reference(dlm):
    z = row_ref.rows(24, 1500, "bf16", 16)
    check_preference(dlm, z, tokens_of(z, 1), [0, 5, 12, 20, 24], with_ref=False, beta=2.0,
                     weights=np.full(24, 1 / 6, F32), margins=np.array([0.3, 0.0], F32))


def test_preference_of_empty_sequences_and_rows_in_none(dlm):
    z = row_ref.rows(30, 2051, "f16", 17)
    token = tokens_of(z, 2)
    # rows 0-3 and 25-29 belong to no sequence; the second pair has no rows, the third none on one side
    check_preference(dlm, z, token, [4, 10, 15, 15, 15, 15, 25])
    check_preference(dlm, z, token, [30, 30, 30])
    check_preference(dlm, z, token, [7])


def test_preference_without_rows(dlm):
    z = torch.empty((0, 1000), device="cuda")
    t, off, m = torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda"), cuda(np.array([0.0, 1.0], F32))
    for r in (dlm.preference_loss(z, t, off, margins=m), dlm.preference_step(z, t, off, margins=m)):
        np.testing.assert_allclose(r.loss.cpu().numpy(), [math.log(2), math.log1p(math.e)], rtol=2.0 ** -20)
        assert (r.score == 0).all()


@pytest.mark.parametrize("given,clean", [([0, -3, 9, 40, 22], [0, 0, 9, 30, 30]), ([5, 2, 9, 8, 2 ** 31 - 1], [5, 5, 9, 9, 30]),
                                         ([-(2 ** 31), 30, 4, 5, 6], [0, 30, 30, 30, 30])])
def test_offsets_out_of_order_are_put_right(dlm, given, clean):
    z = row_ref.rows(30, 1001, "f32", 18)
    check_preference(dlm, z, tokens_of(z, 2), given, clean=clean, status_want=dlm.DEV_BAD_INDEX)


def test_many_short_pairs_and_one_long_one(dlm):
    n = 1500
    z = row_ref.rows(n, 300, "bf16", 19)
    g = np.random.default_rng(4)
    cuts = np.sort(g.integers(0, 500, 399))
    offsets = np.concatenate([[0], cuts, [500, 1000, 1500]])  # 200 pairs of 2.5 rows, then one of 1000
    assert len(offsets) % 2 == 1
    check_preference(dlm, z, tokens_of(z, 3), offsets, beta=0.02)


def test_preference_of_long_rows(dlm):
    z = row_ref.rows(3, 500001, "f32", 20)
    check_preference(dlm, z, tokens_of(z, 3), [0, 1, 3])


def test_preference_pairs_that_are_not_finite(dlm):
    z = row_ref.rows(8, 2000, "f32", 8)
    z[0, 3] = math.nan                 # pair 0: NaN
    z[3, 7] = -math.inf                # pair 1: a rejected token without probability: loss 0
    z[4, 7] = -math.inf                # pair 2: a chosen one: loss infinite
    token = np.full(8, 7, np.int32)
    off = cuda(np.arange(0, 9, 1, dtype=np.int32))
    for call in (dlm.preference_loss, dlm.preference_step):
        status = dlm.new_status()
        r = call(on_gpu(z), cuda(token), off, beta=1.0, status=status)
        assert int(status.item()) == dlm.DEV_NONFINITE
        grad = r.grad if call is dlm.preference_step else dlm.preference_grad(on_gpu(z), cuda(token), r.state)
        assert math.isnan(r.loss[0]) and float(r.loss[1]) == 0.0 and float(r.loss[2]) == math.inf and math.isfinite(r.loss[3])
        assert torch.isnan(grad[:2]).all() and (grad[2:4] == 0).all() and torch.isnan(grad[4:6]).all() and torch.isfinite(grad[6:]).all()


def test_preference_gradient_against_differences(dlm):
    z = row_ref.rows(7, 40, "f32", 22)
    token, offsets = tokens_of(z, 3), [0, 3, 7]
    w = np.linspace(0.5, 1.5, 7).astype(F32)
    r = dlm.preference_step(on_gpu(z), cuda(token), cuda(np.array(offsets, np.int32)), beta=0.7, weights=cuda(w), temperature=1.5)

    def loss(zz):
        s = [sum(float(w[i]) * ref.row(zz[i], token[i], 1.5)[0] for i in range(a, b)) for a, b in ((0, 3), (3, 7))]
        return ref.pair(s[0], s[1], 0.0, float(F32(0.7)), "sigmoid", 0.0)[0]

    zz, h = row_ref.host(z), 1e-4
    for i in range(7):
        for v in range(40):
            e = np.zeros_like(zz)
            e[i, v] = h
            # third derivatives below ~2; 1e-16 / h of losses around 1
            assert abs(float(r.grad[i, v]) - (loss(zz + e) - loss(zz - e)) / (2 * h)) <= 2.0 ** -16 + h * h


# ---- as they are used -------------------------------------------------------

def test_rollout_to_policy_step_to_preference_step(dlm):
    # tokens are sampled, scored under the rollout's and a reference policy, trained on by policy
    # steps on the masked positions, and two answers of each prompt become a pair
    n, vocab = 64, 3000
    z = on_gpu(row_ref.rows(n, vocab, "f32", 40))
    reference = on_gpu(row_ref.rows(n, vocab, "bf16", 41))
    token = dlm.row_sample(z, torch.rand(n, device="cuda"), temperature=0.9, top_p=0.95).token
    old, refs = dlm.row_logprob(z, token), dlm.row_logprob(reference, token)
    st = dlm.row_stats(z)
    np.testing.assert_allclose(old.lse.cpu().numpy(), st.lse.cpu().numpy(), rtol=2.0 ** -17, atol=2.0 ** -17)
    adv = torch.randn(2, device="cuda").repeat_interleave(32)
    weights = torch.rand(n, device="cuda")
    weights[::3] = 0.0
    kw = dict(old=old.logp, ref=refs.logp, kl_weight=0.01, kl="k2", weights=weights)
    first = dlm.policy_step(z, token, adv, **kw)
    # at the rollout's own point the ratio is 1: the loss is -A and the KL term
    want = [float(weights[r]) * ref.policy(float(old.logp[r]), float(adv[r]), float(old.logp[r]), float(refs.logp[r]), 0.2,
                                           0.2, 0.0, float(F32(0.01)), "k2")[0] for r in range(n)]
    np.testing.assert_allclose(first.loss.cpu().numpy(), want, rtol=2.0 ** -17, atol=2.0 ** -17)
    for _ in range(3):
        r = dlm.policy_step(z, token, adv, **kw)
        z -= 0.5 * r.grad
    now = dlm.row_logprob(z, token).logp
    loss = dlm.policy_loss(z, token, adv, **kw)
    for i in range(0, n, 7):
        near(float(loss.logp[i]) if weights[i] else float(now[i]), ref.row(row_ref.host(z[i]), int(token[i]))[0], 2.0 ** -17, i)
    offsets = torch.tensor([0, 16, 32, 48, 64], dtype=torch.int32, device="cuda")
    p = dlm.preference_step(z, token, offsets, ref=refs.logp, weights=weights)
    score = (weights.double() * (now.double() - refs.logp.double())).view(4, 16).sum(1)
    np.testing.assert_allclose(p.score.cpu().numpy(), score.cpu().numpy(), rtol=2.0 ** -16, atol=2.0 ** -14)
    assert torch.isfinite(p.grad).all() and (p.grad[::3] == 0).all()


def graph_of(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    return g


@pytest.mark.parametrize("n,vocab", [(40, 8000), (400, 40003)])
def test_captured_steps_replay_on_new_inputs(dlm, n, vocab):
    z = on_gpu(row_ref.rows(n, vocab, "bf16", 12))
    token = cuda(tokens_of(z.cpu(), 1))
    adv, w = torch.randn(n, device="cuda"), torch.rand(n, device="cuda")
    offsets = torch.tensor([0, n // 3, n // 2, n - 5, n], dtype=torch.int32, device="cuda")
    f = lambda k: torch.empty(k, device="cuda")  # noqa: E731
    one = dlm.PolicyStep(f(n), f(n), on_gpu(z))
    two = dlm.PreferenceStep(f(2), f(4), f(n), on_gpu(z))
    ws = dlm.preference_workspace(n, 2, "cuda")
    ws.fill_(255)                      # whatever a workspace holds before a call
    g = graph_of(lambda: dlm.policy_step(z, token, adv, weights=w, out=one))
    h = graph_of(lambda: dlm.preference_step(z, token, offsets, weights=w, out=two, workspace=ws))
    h2 = graph_of(lambda: dlm.preference_step(z, token, offsets, weights=w, out=two, workspace=ws))
    for scale in (0.5, 1.5):
        z.mul_(scale)
        adv.neg_()
        for graph in (g, h, h2, h):    # two graphs that share a workspace, one after the other
            graph.replay()
        ws.fill_(127)
        want, want2 = dlm.policy_step(z, token, adv, weights=w), dlm.preference_step(z, token, offsets, weights=w)
        assert all(same_bits(a, b) for a, b in zip(one, want))
        assert all(same_bits(a, b) for a, b in zip(two, want2))


def test_calls_on_two_streams_at_once(dlm):
    z = [on_gpu(row_ref.rows(300, 20000, "bf16", s)) for s in (1, 2)]
    token = [cuda(tokens_of(x.cpu(), 1)) for x in z]
    offsets = torch.tensor([0, 100, 180, 250, 300], dtype=torch.int32, device="cuda")
    want = [dlm.preference_step(a, t, offsets) for a, t in zip(z, token)]
    want_lp = [dlm.row_logprob_step(a, t) for a, t in zip(z, token)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in z]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got, got_lp = [[], []], [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(dlm.preference_step(z[i], token[i], offsets))
                got_lp[i].append(dlm.row_logprob_step(z[i], token[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same_bits(a, b) for r in got[i] for a, b in zip(r, want[i]))
        assert all(same_bits(a, b) for r in got_lp[i] for a, b in zip(r, want_lp[i]))


@pytest.mark.parametrize("n,vocab", [(60, 5000), (500, 30011)])
def test_a_call_sees_what_the_one_before_it_wrote(dlm, n, vocab):
    # launches begin while the one before them ends: a chain of calls, each on the last one's
    # outputs, and torch's kernels between them, with and without waiting in between
    start = on_gpu(row_ref.rows(n, vocab, "bf16", 60))
    token = cuda(tokens_of(start.cpu(), 1))
    adv, offsets = torch.randn(n, device="cuda"), torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")

    def chain(wait):
        z, out = on_gpu(start), []
        f = lambda k: torch.empty(k, device="cuda")  # noqa: E731
        grad = on_gpu(start)
        for i in range(6):
            lp = dlm.row_logprob(z, token)
            wait()
            r = dlm.policy_step(z, token, adv, old=lp.logp, ref=lp.lse, kl_weight=0.1, kl="k2",
                                out=dlm.PolicyStep(f(n), f(n), grad))
            wait()
            p = dlm.preference_step(r.grad, token, offsets, ref=r.loss, weights=r.logp,
                                    out=dlm.PreferenceStep(f(1), f(2), f(n), r.grad))
            wait()
            _, z = dlm.row_logprob_step(p.grad, token, p.logp, grad=z)
            wait()
            if i % 2:
                z.add_(start)
            out += [lp.logp, r.loss, p.loss, p.score, p.logp, z.clone()]
        return out

    assert all(same_bits(a, b) for a, b in zip(chain(lambda: None), chain(torch.cuda.synchronize)))


def test_refusals(dlm):
    z = on_gpu(row_ref.rows(4, 512, "f32", 1))
    t, w = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(4, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    bad = [lambda: dlm.row_logprob(z, t.long()), lambda: dlm.row_logprob(z, t[:3]), lambda: dlm.row_logprob(z.T, t),
           lambda: dlm.row_logprob(z, t.cpu()), lambda: dlm.row_logprob(z.cpu(), t.cpu()), lambda: dlm.row_logprob(z, t, gather=True),
           lambda: dlm.row_logprob(z.double(), t), lambda: dlm.row_logprob_step(z, t, w.double()),
           lambda: dlm.row_logprob_step(z, t, w, grad=torch.empty((4, 512), device="cuda", dtype=torch.bfloat16)),
           lambda: dlm.row_logprob_grad(z, t, torch.zeros((4, 3), device="cuda")),
           lambda: dlm.policy_loss(z, t, w[:2]), lambda: dlm.policy_loss(z, t, w, kl="k4"),
           lambda: dlm.policy_step(z, t, w, old=w.half()), lambda: dlm.preference_loss(z, t, off.long()),
           lambda: dlm.preference_loss(z, t, off[:2]), lambda: dlm.preference_loss(z, t, off, kind="none"),
           lambda: dlm.preference_loss(z, t, off, margins=w), lambda: dlm.preference_step(z, t, off, workspace=w)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    state = torch.zeros((4, 8), device="cuda")
    wide = torch.zeros((5, 512), device="cuda")
    index = torch.zeros(1, dtype=torch.int32, device="cuda")
    worse = [lambda: dlm.row_logprob(z, t, temperature=0.0), lambda: dlm.row_logprob(z, t, row_index=index, out=dlm.RowLogprob(
                 torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), state)),
             lambda: dlm.row_logprob_step(wide[:4], t, grad=wide[1:]),
             lambda: dlm.row_logprob_step(z, t, w, logp=w), lambda: dlm.row_logprob(z, t, out=dlm.RowLogprob(w, w, None)),
             lambda: dlm.row_logprob(z, t, out=dlm.RowLogprob(w, state.view(-1)[:4], state)),
             lambda: dlm.policy_loss(z, t, w, clip_low=1.5), lambda: dlm.policy_loss(z, t, w, clip_high=-0.1),
             lambda: dlm.policy_loss(z, t, w, dual_clip=0.5), lambda: dlm.policy_loss(z, t, w, kl_weight=0.1),
             lambda: dlm.policy_loss(z, t, w, clip_high=math.nan), lambda: dlm.policy_loss(z, t, w, kl_weight=-1.0, ref=w),
             lambda: dlm.policy_step(z, t, w, out=dlm.PolicyStep(w, torch.empty(4, device="cuda"), torch.empty_like(z))),
             lambda: dlm.preference_loss(z, t, off, beta=0.0), lambda: dlm.preference_loss(z, t, off, beta=math.inf),
             lambda: dlm.preference_loss(z, t, off, label_smoothing=1.5),
             lambda: dlm.preference_loss(z, t, off, kind="ipo", label_smoothing=0.1),
             lambda: dlm.preference_step(z, t, off, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for call in worse:
        with pytest.raises(dlm.DlmError):
            call()
