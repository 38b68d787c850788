"""Distillation from a teacher's top logits against 64-bit numpy and against
differences of the loss.

Tolerances.  The student's log-sum-exp comes from 32-bit sums within 2^-18
(ex2 2^-22, an exponent of up to ~20 rounded three times at 2^-24, additions),
and so does ln q_rest; p is within 2^-22.  So a row's loss is within
|w| (2^-17 + 2^-22 sum p |ln p - ln q|) and its own rounding.  A gradient
element is within 2^-17 of the magnitudes it is the difference of (q, p, and q
times the factor of the unlisted tokens), plus half a step of its type.  For
tokens whose exponent e is above 28 the roundings of e weigh more than that
(row_ref.distill has the sum), and below 2^-126 of the largest weight ex2 gives
0 for what is not, which the factor of the unlisted tokens multiplies too.
"""
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


def half_step(x, dtype):
    f = torch.finfo(dtype)
    return np.maximum(np.abs(x) * f.eps / 2, f.tiny * f.eps / 2)


def case(n, vocab, kind, k, seed, rest, temperature=1.0, pad=0):
    g = np.random.default_rng(seed)
    z = ref.rows(n, vocab, kind, seed, pad=pad)
    t = ref.host(z) + g.normal(0, 1.0, (n, vocab))
    ids = np.argsort(-t, axis=1, kind="stable")[:, :k].astype(np.int32)
    top = np.take_along_axis(t, ids.astype(np.int64), 1).astype(np.float32)
    if k >= 3:
        ids[::3, -(k // 3):] = -1
    y = t / temperature
    lse = (y.max(1) + np.log(np.exp(y - y.max(1, keepdims=True)).sum(1))).astype(np.float32) if rest else None
    return z, ids, top, lse


def on_gpu(z):
    wide = torch.full((z.shape[0], z.stride(0)), float("nan"), dtype=z.dtype, device="cuda")
    d = wide[:, :z.shape[1]]
    d.copy_(z)
    return d


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(dlm, z, ids, top, lse, temperature=1.0, weights=None, upstream=None, teacher_dtype=torch.float32,
          status_want=0):
    n, vocab = z.shape
    teacher = cuda(top).to(teacher_dtype)
    top = ref.host(teacher)
    d, status = on_gpu(z), dlm.new_status()
    kw = dict(teacher_lse=cuda(lse), temperature=temperature, weights=cuda(weights), status=status)
    out = dlm.distill_loss(d, cuda(ids), teacher, **kw)
    g1 = dlm.distill_grad(d, cuda(ids), teacher, out.state, cuda(upstream), temperature=temperature,
                          weights=cuda(weights), status=status)
    loss2, g2 = dlm.distill_step(d, cuda(ids), teacher, **kw)
    inplace = on_gpu(z)
    loss3, g3 = dlm.distill_step(inplace, cuda(ids), teacher, grad=inplace, **kw)
    assert int(status.item()) == status_want
    assert torch.equal(loss2, loss3)
    assert torch.equal(g2.contiguous().view(torch.uint8), g3.contiguous().view(torch.uint8))
    zz = ref.host(z)
    for r in range(n):
        w = 1.0 if weights is None else float(weights[r])
        up = 1.0 if upstream is None else float(upstream[r])
        want, grad, scale = ref.distill(zz[r], ids[r], top[r], w, temperature, None if lse is None else float(lse[r]))
        if w == 0:
            want, grad, scale = 0.0, grad * 0, scale * 0
        for got in (float(out.loss[r]), float(loss2[r])):
            if np.isfinite(want):
                assert abs(got - want) <= abs(w) * 2.0 ** -17 + abs(want) * 2.0 ** -21 + abs(w) * 2.0 ** -21, (r, got, want)
            else:
                assert got == want
        for g, f in ((g1, up), (g2, 1.0)):
            x = ref.host(g[r])
            tol = abs(f) * scale * 2.0 ** -17 + half_step(f * grad, z.dtype)
            bad = np.abs(x - f * grad) > tol
            assert not bad.any(), (r, np.nonzero(bad)[0][:5], x[bad][:5], (f * grad)[bad][:5])


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,vocab,k", [(1, 1, 1), (2, 9, 4), (3, 130, 7), (4, 1025, 1), (5, 5003, 64), (2, 32003, 1024),
                                       (330, 2051, 16), (2, 126464, 64)])
def test_distill(dlm, kind, n, vocab, k, rest):
    check(dlm, *case(n, vocab, kind, min(k, vocab), seed=n + vocab + k, rest=rest, pad=n % 2))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("kind,n,vocab", [("f32", 2, 500001), ("bf16", 1, 1000003), ("f32", 1, 1048575)])
def test_rows_too_long_to_be_held_on_chip(dlm, kind, n, vocab, rest):
    check(dlm, *case(n, vocab, kind, 40, seed=vocab, rest=rest))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("temperature", [0.3, 2.0, 5.0])
def test_temperature_weights_and_upstream(dlm, temperature, rest):
    n = 11
    g = np.random.default_rng(3)
    weights = g.uniform(0.2, 3.0, n).astype(np.float32)
    weights[[2, 7]] = 0.0
    upstream = g.normal(0, 1, n).astype(np.float32)
    upstream[5] = 0.0
    check(dlm, *case(n, 4001, "f32", 24, 9, rest, temperature), temperature=temperature, weights=weights,
          upstream=upstream)


@pytest.mark.parametrize("teacher_dtype", [torch.bfloat16, torch.float16])
def test_teacher_types(dlm, teacher_dtype):
    z, ids, top, _ = case(6, 3000, "bf16", 32, 4, False)
    check(dlm, z, ids, top, None, teacher_dtype=teacher_dtype)


@pytest.mark.parametrize("rest", [False, True])
def test_repeated_padded_and_empty_lists(dlm, rest):
    z, ids, top, lse = case(6, 2000, "f32", 12, 5, rest)
    ids[0] = ids[0, 0]                 # one id twelve times: its entries add up
    ids[1, 3] = ids[1, 0]
    ids[2] = -1                        # nothing listed
    top[3, 2:] = -np.inf               # entries that carry nothing
    ids[4, 1:] = -1                    # one entry
    ids[5, 5] = -2000000000
    if rest:                           # the repeats' mass stays a probability
        lse = lse + np.float32(3.0)
    check(dlm, z, ids, top, lse)


def test_ids_outside_the_vocabulary_are_skipped(dlm):
    z, ids, top, _ = case(3, 1000, "bf16", 8, 6, False)
    ids[1, 2], ids[2, 0] = 1000, 2 ** 31 - 1
    check(dlm, z, ids, top, None, status_want=dlm.DEV_BAD_INDEX)


@pytest.mark.parametrize("rest", [False, True])
def test_masked_students(dlm, rest):
    z, ids, top, lse = case(4, 3000, "f32", 10, 7, rest)
    z[0, 1500:] = -float("inf")        # not listed: no probability, gradient 0
    z[1] = torch.finfo(torch.float32).min
    z[1, ids[1, 0]] = 0.0
    z[2] = -float("inf")
    z[2, 5] = 1.0                      # one token left; a listed -inf makes the loss infinite
    ids[0] = np.arange(10)
    check_finite = [0, 3]
    d = on_gpu(z)
    loss, grad = dlm.distill_step(d, cuda(ids), cuda(top), teacher_lse=cuda(lse))
    zz = ref.host(z)
    for r in check_finite:
        want, g, scale = ref.distill(zz[r], ids[r], top[r].astype(np.float64), teacher_lse=None if lse is None else float(lse[r]))
        assert abs(float(loss[r]) - want) <= 2.0 ** -16 + abs(want) * 2.0 ** -21
        assert (np.abs(ref.host(grad[r]) - g) <= scale * 2.0 ** -17 + half_step(g, z.dtype)).all()
    assert (ref.host(grad[0])[1500:] == 0).all()
    assert float(loss[2]) == float("inf")
    assert not torch.isnan(grad[:4]).any()


@pytest.mark.parametrize("rest", [False, True])
def test_nan_rows_are_flagged_and_stay_in_their_rows(dlm, rest):
    z, ids, top, lse = case(5, 2000, "bf16", 8, 8, rest)
    z[0, 11] = float("nan")
    z[1, 12] = float("inf")
    z[2] = -float("inf")
    top[3, 0] = np.nan
    status = dlm.new_status()
    loss, grad = dlm.distill_step(on_gpu(z), cuda(ids), cuda(top), teacher_lse=cuda(lse), status=status)
    assert int(status.item()) == dlm.DEV_NONFINITE
    assert torch.isnan(loss[:4]).all() and torch.isnan(grad[:4]).any(1).all()
    assert torch.isfinite(loss[4]) and torch.isfinite(grad[4]).all()


@pytest.mark.parametrize("rest", [False, True])
def test_gradient_against_differences(dlm, rest):
    # central differences of the 64-bit loss at the f32 student's values: their
    # error is h^2 / 6 times a third derivative of at most ~1, and 1e-16 / h
    z, ids, top, lse = case(3, 60, "f32", 6, 10, rest, 1.5)
    _, grad = dlm.distill_step(on_gpu(z), cuda(ids), cuda(top), teacher_lse=cuda(lse), temperature=1.5)
    h = 1e-4
    for r, row in enumerate(ref.host(z)):
        f = lambda x: ref.distill(x, ids[r], top[r].astype(np.float64), 1.0, 1.5, None if lse is None else float(lse[r]))[0]  # noqa: E731,B023
        for v in range(60):
            e = np.zeros(60)
            e[v] = h
            d = (f(row + e) - f(row - e)) / (2 * h)
            assert abs(float(grad[r, v]) - d) <= 2.0 ** -16 + h * h


def test_out_of_place_leaves_what_lies_past_the_rows(dlm):
    z, ids, top, _ = case(4, 1003, "bf16", 8, 11, False, pad=2)
    wide = torch.full((4, z.stride(0)), 7.0, dtype=torch.bfloat16, device="cuda")
    dlm.distill_step(on_gpu(z), cuda(ids), cuda(top), grad=wide[:, :1003])
    assert (wide[:, 1003:] == 7.0).all() and not (wide[:, :1003] == 7.0).any()


def test_captured_step_replays_on_new_inputs(dlm):
    z, ids, top, lse = case(40, 8000, "bf16", 32, 12, True)
    d, i, t, l = on_gpu(z), cuda(ids), cuda(top), cuda(lse)
    loss = torch.empty(40, device="cuda")
    grad = torch.empty_like(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        dlm.distill_step(d, i, t, teacher_lse=l, loss=loss, grad=grad)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            dlm.distill_step(d, i, t, teacher_lse=l, loss=loss, grad=grad)
    torch.cuda.current_stream().wait_stream(side)
    d.mul_(0.5)
    g.replay()
    want_loss, want = dlm.distill_step(d, i, t, teacher_lse=l)
    assert torch.equal(loss, want_loss) and torch.equal(grad, want)


def test_teacher_rows_to_student_gradient_to_sampled_tokens(dlm):
    # the operators as they are used together: the teacher's top logits and
    # log-sum-exp are stored, a student's rows are trained on them by their
    # gradient, and its tokens are sampled and selected
    n, vocab = 64, 3000
    teacher = on_gpu(ref.rows(n, vocab, "bf16", 40))
    student = on_gpu(ref.rows(n, vocab, "f32", 41, boosted=0.0))
    top = dlm.row_topk(teacher, 32)
    first = dlm.distill_loss(student, top.ids, top.values, teacher_lse=top.lse).loss
    grad = None
    for _ in range(3):
        loss, grad = dlm.distill_step(student, top.ids, top.values, teacher_lse=top.lse, grad=grad)
        student -= 4.0 * grad
    want = [ref.distill(ref.host(student)[r], top.ids[r].cpu().numpy(), ref.host(top.values[r]),
                        teacher_lse=float(top.lse[r]))[0] for r in range(4)]
    last = dlm.distill_loss(student, top.ids, top.values, teacher_lse=top.lse).loss
    np.testing.assert_allclose(last[:4].cpu().numpy(), want, atol=2.0 ** -16, rtol=2.0 ** -20)
    assert torch.isfinite(first).all()
    st = dlm.row_stats(student)
    u = torch.rand(n, device="cuda")
    s = dlm.row_sample(student, u, temperature=0.7, top_p=0.9, lse=st.lse)
    masked = torch.ones((2, 32), dtype=torch.uint8, device="cuda")
    sel, count = dlm.select_threshold(s.conf.view(2, 32), masked, 0.3)
    want_token = [ref.sample(row, float(u[r]), 0.7, 0, 0.9)[0] for r, row in enumerate(ref.host(student))]
    np.testing.assert_array_equal(s.token.cpu().numpy(), want_token)
    np.testing.assert_array_equal(count.cpu().numpy(), np.maximum(1, (s.conf.view(2, 32) > 0.3).sum(1).cpu().numpy()))
    assert (sel.sum(1).cpu() == count.cpu()).all()


def test_refusals(dlm):
    z, ids, top, lse = case(4, 512, "f32", 8, 1, True)
    d, i, t = on_gpu(z), cuda(ids), cuda(top)
    with pytest.raises(ValueError):
        dlm.distill_loss(d, i.long(), t)
    with pytest.raises(ValueError):
        dlm.distill_loss(d, i, t[:, :4])
    with pytest.raises(ValueError):
        dlm.distill_loss(d, i, t, weights=torch.ones(3, device="cuda"))
    with pytest.raises(dlm.DlmError):
        dlm.distill_loss(d, i, t, temperature=0.0)
    with pytest.raises(ValueError):
        dlm.distill_step(d, i, t, grad=torch.empty((4, 512), device="cuda", dtype=torch.bfloat16))
    with pytest.raises(dlm.DlmError):  # overlaps the student without being it
        wide = torch.zeros((5, 512), device="cuda")
        dlm.distill_step(wide[:4], i, t, grad=wide[1:])
    with pytest.raises(ValueError):
        dlm.distill_grad(d, i, t, torch.zeros((4, 3), device="cuda"))
