"""Distillation where a student's mass lies in its list by tens of nats, or in one
token: loss and gradient against 64-bit numpy that works with logarithms.

Tolerances.  A row's two sums of exponentials (listed, not listed) are each
within 2^-18 of themselves (ex2 2^-22, exponents of up to ~20 relative to the
sum's own largest rounded three times at 2^-24, additions), and logarithms of
them within that.  So the loss is within |w| 2^-17 sum p, and 2^-21 of itself for
its own roundings.  An unlisted token's gradient w / T (q_v - p_rest e_v / rest)
is within 2^-17 of its two terms, more where the token lies far below the largest
unlisted one (row_ref.distill has that factor).  A listed token's q - p is within
2^-17 of q + p, and where q is above 1/2 within 2^-17 of (1 - q) + |1 - p|, of
which it is the difference too.  Half a step of the gradient's type is added.
"""
import math

import numpy as np
import pytest
import torch

import row_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dlm():
    import diffusion_decoding_token_gb300 as d
    d.lib()
    return d


def log_sum_exp(y):
    return y.max() + math.log(np.exp(y - y.max()).sum()) if len(y) and y.max() > -np.inf else -np.inf


def definition(row, ids, teacher, t, lse):
    """(loss, gradient, the gradient's error scale) of a row of weight 1."""
    held = ids >= 0
    ids, a = ids[held], teacher[held] / t
    with np.errstate(divide="ignore"):
        y = row / t
        log_q = y - log_sum_exp(y)
        log_p = np.minimum(a - (log_sum_exp(a) if lse is None else lse), 8 * math.log(2))
        out = np.ones(len(row), bool)
        out[ids] = False
        p, q = np.exp(log_p), np.exp(log_q)
        loss = sum(p[j] * (log_p[j] - log_q[ids[j]]) for j in range(len(p)) if p[j] > 0)
        far = lambda e: np.maximum(1.0, 0.53 + 0.0165 * np.minimum(e / math.log(2), 1e4))  # noqa: E731
        grad, scale = q.copy(), q * far(y.max() - y)
        total = np.zeros(len(row))
        np.add.at(total, ids, p)
        grad -= total
        scale += total
        if q.max() > 0.5 and not out[q.argmax()]:  # one token holds the row: its complement counts
            v = int(q.argmax())
            others = math.exp(log_sum_exp(np.delete(y, v)) - log_sum_exp(y))  # 1 - q
            less = 1 - total[v] if lse is not None else math.fsum(p[ids != v])
            # (each of the other weights may be one below 2^-126, which counts as 0)
            grad[v], scale[v] = less - others, abs(less) + others + len(row) * 2.0 ** (17 - 126)
        if lse is not None:
            p_rest = max(0.0, 1 - math.fsum(p))
            log_rest = log_sum_exp(y[out])
            if p_rest > 0:
                loss += p_rest * (math.log(p_rest) - (log_rest - log_sum_exp(y)))
            if p_rest > 0 and log_rest > -np.inf:
                e = np.exp(y[out] - y[out].max())  # (the logarithm itself has no digits left at -3e38)
                e /= e.sum()
                grad[out] -= p_rest * e
                scale[out] += p_rest * e * far(y[out].max() - y[out])
    return loss, grad / t, (scale + 2.0 ** (17 - 126)) / t, max(1.0, p.sum())


def half_step(x, dtype):
    f = torch.finfo(dtype)
    return np.maximum(np.abs(x) * f.eps / 2, f.tiny * f.eps / 2)


def on_gpu(z):
    wide = torch.full((z.shape[0], z.stride(0)), float("nan"), dtype=z.dtype, device="cuda")
    d = wide[:, :z.shape[1]]
    d.copy_(z)
    return d


def check(dlm, z, ids, top, lse, t=1.0, w=1.0):
    d, cuda = on_gpu(z), lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    status = dlm.new_status()
    weights = torch.full((len(z),), w, device="cuda")
    kw = dict(teacher_lse=cuda(lse), temperature=t, weights=weights, status=status)
    out = dlm.distill_loss(d, cuda(ids), cuda(top), **kw)
    g1 = dlm.distill_grad(d, cuda(ids), cuda(top), out.state, temperature=t, weights=weights, status=status)
    loss2, g2 = dlm.distill_step(d, cuda(ids), cuda(top), **kw)
    assert int(status.item()) == 0
    zz = ref.host(z)
    for r in range(len(zz)):
        want, grad, scale, mass = definition(zz[r], ids[r], top[r].astype(np.float64), t, None if lse is None else float(lse[r]))
        want, grad, scale = w * want, w * grad, w * scale
        for name, got in (("loss", float(out.loss[r])), ("step", float(loss2[r]))):
            if math.isinf(want):
                assert got == want, (name, r, got, want)
            else:
                assert abs(got - want) <= 2.0 ** -17 * w * mass + 2.0 ** -21 * (w + abs(want)), (name, r, got, want)
        for name, g in (("grad", g1), ("step", g2)):
            x = ref.host(g[r])
            bad = ~(np.abs(x - grad) <= scale * 2.0 ** -17 + half_step(grad, z.dtype))
            assert not bad.any(), (name, r, np.nonzero(bad)[0][:5], x[bad][:5], grad[bad][:5])


def flat_teacher(n, vocab, kind, k, seed, gap, t=1.0, rest_mass=0.5, hole=0.0):
    """Students whose listed logits lie `gap` temperatures above all others, the
    list all over the row (one entry of a cluster's each slice at a height of its
    own), against a teacher that gives the others `rest_mass`."""
    g = np.random.default_rng(seed)
    z = ref.rows(n, vocab, kind, seed, sigma=0.5, boosted=0.0)
    ids = np.stack([np.linspace(0, vocab - 1, k).astype(np.int32) for _ in range(n)])
    host = ref.host(z)
    for r in range(n):
        host[r] = host[r] * t
        host[r, ids[r]] += gap * t * np.where(np.arange(k) % 3 == 1, 0.9, 1.0)
        if hole:
            gone = g.random(vocab) < hole
            gone[ids[r]] = False
            host[r, gone] = -np.inf
    z.copy_(torch.from_numpy(host.astype(np.float32)).to(z.dtype))
    top = g.normal(0, t, (n, k)).astype(np.float32)
    a = top.astype(np.float64) / t
    lse = np.array([log_sum_exp(x) - math.log1p(-rest_mass) for x in a], np.float32)
    return z, ids, top, lse


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gap", [20, 30, 40, 60])
@pytest.mark.parametrize("n,vocab,k", [(3, 3000, 12), (2, 40001, 64), (1, 126464, 200)])
def test_list_far_above_the_rest(dlm, kind, gap, n, vocab, k):
    check(dlm, *flat_teacher(n, vocab, kind, k, gap, gap))


@pytest.mark.parametrize("gap", [30, 60])
@pytest.mark.parametrize("kind,vocab", [("f32", 500001), ("bf16", 1000003)])
def test_list_far_above_the_rest_of_a_long_row(dlm, kind, vocab, gap):
    check(dlm, *flat_teacher(1, vocab, kind, 40, gap, gap))


def test_repeats_far_above_the_rest(dlm):
    z, ids, top, lse = flat_teacher(3, 5000, "f32", 20, 3, 45)
    ids[:, 3] = ids[:, 4]
    check(dlm, z, ids, top, lse)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("gap,t", [(83, 1.0), (86, 1.0), (88, 0.125), (100, 1.0), (1000, 0.25), (40000, 0.01)])
@pytest.mark.parametrize("n,vocab,k", [(3, 3000, 12), (1, 126464, 64)])
def test_rest_below_the_range_of_a_float(dlm, kind, gap, t, n, vocab, k):
    # the unlisted tokens' weights relative to the row's largest are subnormal, or
    # 0 in 32 bits; a third of these tokens is masked
    check(dlm, *flat_teacher(n, vocab, kind, k, 7, gap, t, hole=0.3), t=t)


@pytest.mark.parametrize("kind,vocab", [("f32", 500001), ("bf16", 1000003)])
@pytest.mark.parametrize("gap", [86, 100])
def test_rest_below_the_range_of_a_float_in_a_long_row(dlm, kind, vocab, gap):
    check(dlm, *flat_teacher(1, vocab, kind, 40, 9, gap, hole=0.3))


@pytest.mark.parametrize("w", [1e30, 1e-30])
def test_large_and_small_weights(dlm, w):
    z, ids, top, lse = flat_teacher(2, 3000, "f32", 12, 11, 80, 1e-3, hole=0.3)
    check(dlm, z, ids, top, lse, t=1e-3, w=float(np.float32(w)))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rest_at_the_lowest_value(dlm, kind):
    # every unlisted token is masked with the type's lowest value: the rest's
    # probability is e^-3e38, its tokens share its gradient
    z, ids, top, lse = flat_teacher(3, 3000, kind, 12, 13, 20)
    keep = z.clone()
    z[:] = torch.finfo(z.dtype).min
    for r in range(3):
        z[r, torch.from_numpy(ids[r]).long()] = keep[r, torch.from_numpy(ids[r]).long()]
    z[2, ids[2, 1:].tolist()] = torch.finfo(z.dtype).min  # and of the list all but one
    check(dlm, z, ids, top, lse)


def test_no_rest_at_all(dlm):
    # q_rest = 0 while the teacher has a rest: the loss is infinite, the listed
    # tokens' gradient is what it is
    z, ids, top, lse = flat_teacher(2, 3000, "f32", 12, 15, 20)
    keep = z.clone()
    z[0] = -float("inf")
    z[0, torch.from_numpy(ids[0]).long()] = keep[0, torch.from_numpy(ids[0]).long()]
    check(dlm, z, ids, top, lse)


def peaked(n, vocab, kind, k, seed, rest, sure):
    """Students and teachers sure of the same token of each row, 1 - q and 1 - p
    about e^-sure each and of the same order."""
    g = np.random.default_rng(seed)
    z = ref.rows(n, vocab, kind, seed, boosted=0.0)
    host = ref.host(z)
    at = g.integers(vocab, size=n)
    for r in range(n):
        host[r, at[r]] = log_sum_exp(host[r]) + sure
    z.copy_(torch.from_numpy(host.astype(np.float32)).to(z.dtype))
    t = ref.host(z) + g.normal(0, 0.5, (n, vocab))
    ids = np.argsort(-t, axis=1, kind="stable")[:, :k].astype(np.int32)
    ids = ids[:, g.permutation(k)]
    top = np.take_along_axis(t, ids.astype(np.int64), 1).astype(np.float32)
    # (a little more than the log-sum-exp, so that rounding leaves no p above 1)
    lse = np.array([log_sum_exp(x) + 6e-6 for x in t], np.float32) if rest else None
    return z, ids, top, lse


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sure", [5, 9, 13])
@pytest.mark.parametrize("n,vocab,k", [(6, 2000, 16), (3, 40001, 300), (2, 126464, 64)])
def test_rows_that_are_sure_of_a_token(dlm, kind, sure, rest, n, vocab, k):
    check(dlm, *peaked(n, vocab, kind, k, sure, rest, sure))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("kind,vocab", [("f32", 500001), ("bf16", 1000003)])
def test_long_rows_that_are_sure_of_a_token(dlm, kind, vocab, rest):
    check(dlm, *peaked(1, vocab, kind, 40, 5, rest, 11))


@pytest.mark.parametrize("rest", [False, True])
def test_sure_of_a_token_that_is_listed_in_parts(dlm, rest):
    # the token's probability in three entries that add up to it
    z, ids, top, lse = peaked(4, 3000, "f32", 20, 21, rest, 10)
    for r in range(4):
        j = int(top[r].argmax())
        i = [x for x in range(20) if x != j][5:7]
        ids[r, i] = ids[r, j]
        top[r, i] = top[r, j] - np.float32(3.0)
        top[r, j] += np.float32(math.log1p(-2 * math.exp(-3.0)))
    check(dlm, z, ids, top, lse)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("less", [0.0, 1e-6, 1e-3, 0.3, 1.0, 5.0, 5.6, 40.0])
def test_teacher_sums_below_their_logits(dlm, kind, less):
    # probabilities above 1 are what the formula makes of them (up to 256): a
    # rounded log-sum-exp of a teacher that is sure of a token gives 1 + 1e-6
    z, ids, top, _ = peaked(5, 3000, kind, 16, 23, True, 9)
    check(dlm, z, ids, top, (top.max(1) - less).astype(np.float32))
    ids[:, 4] = ids[:, 5]
    check(dlm, z, ids, top, (top.max(1) - less).astype(np.float32))


def test_gradient_rows_between_the_students(dlm):
    # memory that holds both in turn overlaps nowhere
    z, ids, top, lse = flat_teacher(6, 1003, "f32", 8, 25, 3)
    cuda = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    want = dlm.distill_step(on_gpu(z), cuda(ids), cuda(top), teacher_lse=cuda(lse))
    for first in (0, 1):
        both = torch.full((6, 2, 1004), 7.0, device="cuda")
        student, grad = both[:, first, :1003], both[:, 1 - first, :1003]
        student.copy_(z)
        loss, _ = dlm.distill_step(student, cuda(ids), cuda(top), teacher_lse=cuda(lse), grad=grad)
        assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])
        assert torch.equal(student.cpu(), z) and (both[:, :, 1003] == 7.0).all()
    with pytest.raises(dlm.DlmError):  # the same stride, one vector of each row shared
        wide = torch.zeros((6, 2, 1004), device="cuda").view(6, 2008)
        dlm.distill_step(wide[:, :1003], cuda(ids), cuda(top), grad=wide[:, 1000:2003])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sure,t", [(18, 1.0), (24, 1.0), (40, 0.5)])
@pytest.mark.parametrize("n,vocab,k", [(5, 2000, 16), (2, 40001, 700), (1, 500001, 40)])
def test_rows_that_are_all_but_certain(dlm, kind, sure, t, n, vocab, k):
    # 1 - p from 1e-8 to 1e-35: next to nothing in units of 2^-44
    z, ids, top, _ = peaked(n, vocab, kind, k, sure, False, sure)
    check(dlm, z, ids, top, None, t=t)
    ids[:, 2] = ids[:, 3]
    check(dlm, z, ids, top, None, t=t)


def test_one_less_p_next_to_nothing(dlm):
    # lse_t - t / T of 2^-18 to 2^-40 (a teacher whose logits lie around 0)
    z, ids, top, _ = peaked(23, 2000, "f32", 16, 31, True, 12)
    top -= top.max(1, keepdims=True)
    check(dlm, z, ids, top, (2.0 ** -np.arange(18, 41)).astype(np.float32))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("listed", [False, True])
def test_logarithms_beyond_a_float(dlm, kind, listed):
    # ln q of -3e38 / 0.5 times a probability of 1e-5: a loss of 1e33
    z, ids, top, lse = flat_teacher(3, 3000, kind, 12, 27, 20, t=0.5, rest_mass=0.0 if listed else 1e-5)
    low = torch.finfo(z.dtype).min
    if listed:
        top[:, 3] = top.max(1) - np.float32(5.5)
        z[torch.arange(3), torch.from_numpy(ids[:, 3]).long()] = low
        check(dlm, z, ids, top, None, t=0.5)
    keep = z.clone()
    z[:] = low
    for r in range(3):
        z[r, torch.from_numpy(ids[r]).long()] = keep[r, torch.from_numpy(ids[r]).long()]
    if not listed:
        check(dlm, z, ids, top, lse, t=0.5)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("kind,n,vocab,k", [("f32", 128, 2000, 700), ("bf16", 128, 2000, 64), ("f16", 16, 60000, 1000),
                                            ("f32", 3, 500001, 300)])
def test_repeats_give_the_same_bits_on_every_launch(dlm, kind, n, vocab, k, rest):
    g = np.random.default_rng(33)
    z, ids, top, lse = flat_teacher(n, vocab, kind, k, 29, 2, rest_mass=0.5)
    ids = np.take_along_axis(ids, g.integers(0, k, (n, k)), 1)  # a third of the tokens is listed twice or more
    d, cuda = on_gpu(z), lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    i, t, lse = cuda(ids), cuda(top), cuda(lse) if rest else None
    bits = lambda x: x.contiguous().view(torch.uint8)  # noqa: E731
    want = dlm.distill_loss(d, i, t, teacher_lse=lse), dlm.distill_step(d, i, t, teacher_lse=lse)
    want_grad = dlm.distill_grad(d, i, t, want[0].state)
    for _ in range(20):
        out = dlm.distill_loss(d, i, t, teacher_lse=lse)
        loss, grad = dlm.distill_step(d, i, t, teacher_lse=lse)
        assert torch.equal(bits(out.loss), bits(want[0].loss)) and torch.equal(bits(out.state), bits(want[0].state))
        assert torch.equal(bits(loss), bits(want[1][0])) and torch.equal(bits(grad), bits(want[1][1]))
        assert torch.equal(bits(dlm.distill_grad(d, i, t, out.state)), bits(want_grad))
