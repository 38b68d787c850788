"""Host-side refusals of the calls over given tokens: status codes before anything
touches a GPU (no device needed)."""
import ctypes
import math

import pytest

INVALID, ALIGN, UNSUP, WS = 1, 2, 3, 4
P = ctypes.c_void_p
D = ctypes.c_double


@pytest.fixture(scope="module")
def L():
    from diffusion_decoding_token_gb300 import build
    build.build()
    import diffusion_decoding_token_gb300 as d
    return d.lib()


def at(k):
    return P(0x1000000 + 0x10000 * k)


T, STATE, LOGP, LOSS, LSE, A, W, REF, OLD = at(1), at(3), at(4), at(5), at(6), at(7), at(8), at(9), at(10)
OFF, MARGIN, PW, SCORE, WORK = at(11), at(12), at(13), at(14), at(15)
BIG = (P(0x80000000), P(0xc0000000))  # logits and gradient, far apart


def head(kw):
    a = dict(logits=BIG[0], dtype=1, n=4, vocab=100, stride=104) | kw
    return a["logits"], a["dtype"], a["n"], a["vocab"], a["stride"]


def logprob(L, tokens=T, t=1.0, logp=LOGP, lse=LSE, state=None, index=None, n_src=0, flags=0, **kw):
    return L.dlm_row_logprob(*head(kw), index, n_src, tokens, D(t), logp, lse, state, None, flags, None)


def logprob_grad(L, tokens=T, t=1.0, state=STATE, up=None, grad=BIG[1], gstride=104, **kw):
    return L.dlm_row_logprob_grad(*head(kw), tokens, D(t), state, up, grad, gstride, None, None)


def logprob_step(L, tokens=T, t=1.0, weights=W, logp=LOGP, grad=BIG[1], gstride=104, **kw):
    return L.dlm_row_logprob_step(*head(kw), tokens, D(t), weights, logp, grad, gstride, None, None)


def policy(L, step, tokens=T, t=1.0, adv=A, old=OLD, ref=REF, weights=W, prm=(0.2, 0.2, 0.0, 0.1, 3), loss=LOSS, logp=LOGP,
           state=STATE, grad=BIG[1], gstride=104, **kw):
    from diffusion_decoding_token_gb300._binding import PolicyParams
    p = ctypes.byref(PolicyParams(*prm)) if prm else None
    a = (*head(kw), tokens, D(t), adv, old, ref, weights, p, loss, logp)
    return L.dlm_policy_step(*a, grad, gstride, None, None) if step else L.dlm_policy_loss(*a, state, None, None)


def preference(L, step, tokens=T, t=1.0, off=OFF, pairs=2, ref=REF, weights=W, margins=MARGIN, pw=PW, prm=(0.1, 0.0, 0), loss=LOSS,
               score=SCORE, logp=LOGP, state=STATE, grad=BIG[1], gstride=104, work=WORK, nbytes=1 << 15, **kw):
    from diffusion_decoding_token_gb300._binding import PreferenceParams
    p = ctypes.byref(PreferenceParams(*prm)) if prm else None
    a = (*head(kw), tokens, D(t), off, pairs, ref, weights, margins, pw, p, loss, score, logp)
    return L.dlm_preference_step(*a, grad, gstride, work, nbytes, None, None) if step else \
        L.dlm_preference_loss(*a, state, None, None)


CALLS = {"logprob": logprob, "grad": logprob_grad, "step": logprob_step,
         "policy_loss": lambda L, **k: policy(L, False, **k), "policy_step": lambda L, **k: policy(L, True, **k),
         "preference_loss": lambda L, **k: preference(L, False, **k),
         "preference_step": lambda L, **k: preference(L, True, **k)}


@pytest.mark.parametrize("name", CALLS)
def test_rows(L, name):
    call = CALLS[name]
    if not name.startswith("preference"):
        assert call(L, n=0) == 0 and call(L, n=0, logits=None, tokens=None) == 0
    else:
        assert call(L, n=0, pairs=0) == 0
    assert call(L, dtype=3) == UNSUP
    for kw in (dict(logits=None), dict(tokens=None), dict(n=-1), dict(n=1 << 31), dict(vocab=0), dict(vocab=105),
               dict(vocab=1 << 20, stride=1 << 20), dict(t=0.0), dict(t=5e-5), dict(t=2e30), dict(t=math.nan), dict(t=-1.0)):
        assert call(L, **kw) == INVALID, kw
    assert call(L, logits=P(0x80000008)) == ALIGN
    assert call(L, stride=101) == ALIGN
    if "step" in name or name == "grad":
        for kw in (dict(grad=None), dict(gstride=99), dict(grad=P(0x80000010)), dict(grad=BIG[0], gstride=112)):
            assert call(L, **kw) == INVALID, kw
        assert call(L, grad=P(0xc0000008)) == ALIGN and call(L, gstride=107) == ALIGN


def test_logprob(L):
    for kw in (dict(logp=None), dict(flags=1), dict(flags=4), dict(n_src=-1), dict(n_src=3), dict(state=STATE, index=at(20)),
               dict(lse=LOGP), dict(logp=T), dict(state=LSE), dict(lse=P(0x1000000 + 0x10000 * 4 + 12)),
               dict(logp=at(20), index=at(20), n_src=9)):
        assert logprob(L, **kw) == INVALID, kw
    assert logprob(L, state=P(0x1030008)) == ALIGN
    assert logprob_grad(L, state=None) == INVALID and logprob_grad(L, state=P(0x1030004)) == ALIGN
    assert logprob_step(L, logp=None) == INVALID and logprob_step(L, logp=W) == INVALID and logprob_step(L, logp=T) == INVALID


@pytest.mark.parametrize("step", [False, True])
def test_policy(L, step):
    inf, nan = math.inf, math.nan
    for prm in ((-0.1, 0.2, 0, 0, 3), (1.1, 0.2, 0, 0, 3), (nan, 0.2, 0, 0, 3), (0.2, -0.1, 0, 0, 3), (0.2, nan, 0, 0, 3),
                (0.2, 0.2, 0.5, 0, 3), (0.2, 0.2, -3, 0, 3), (0.2, 0.2, inf, 0, 3), (0.2, 0.2, nan, 0, 3), (0.2, 0.2, 0, -1, 3),
                (0.2, 0.2, 0, inf, 3), (0.2, 0.2, 0, nan, 3), (0.2, 0.2, 0, 0, 0), (0.2, 0.2, 0, 0, 4), None):
        assert policy(L, step, prm=prm) == INVALID, prm
        assert policy(L, step, prm=prm, n=0) == INVALID, prm
    for kw in (dict(adv=None), dict(loss=None), dict(ref=None), dict(loss=A), dict(logp=OLD), dict(logp=LOSS), dict(loss=W),
               dict(loss=P(0x1000000 + 0x70000 + 4)), dict(logp=REF)):
        assert policy(L, step, **kw) == INVALID, kw
    if not step:
        assert policy(L, step, state=P(0x1030004)) == ALIGN and policy(L, step, state=LOSS) == INVALID
    assert policy(L, step, n=0, prm=(0.2, inf, 1.0, 0, 1), adv=None) == 0


@pytest.mark.parametrize("step", [False, True])
def test_preference(L, step):
    for prm in ((0, 0, 0), (-1, 0, 0), (math.inf, 0, 0), (math.nan, 0, 0), (0.1, -0.1, 0), (0.1, 1.1, 0), (0.1, math.nan, 0),
                (0.1, 0.1, 1), (0.1, 0.1, 2), (0.1, 0, 3), (0.1, 0, -1), None):
        assert preference(L, step, prm=prm) == INVALID, prm
    for kw in (dict(pairs=-1), dict(pairs=1 << 31), dict(off=None), dict(loss=None), dict(loss=MARGIN), dict(loss=PW),
               dict(score=LOSS), dict(logp=REF), dict(score=OFF), dict(logp=P(0x1000000 + 0x50000 + 4))):
        assert preference(L, step, **kw) == INVALID, kw
    if step:
        need = L.dlm_preference_workspace_size(4, 2)
        assert need > 0 and preference(L, step, nbytes=need - 1) == WS and preference(L, step, work=None) == WS
        assert preference(L, step, work=P(0x10f0004)) == ALIGN
        for kw in (dict(work=W), dict(work=LOSS), dict(work=OFF), dict(work=LOGP)):
            assert preference(L, step, **kw) == INVALID, kw
    else:
        assert preference(L, step, state=None) == INVALID and preference(L, step, state=P(0x1030008)) == ALIGN
        assert preference(L, step, state=LOGP) == INVALID
    assert L.dlm_preference_workspace_size(-1, 0) == 0 and L.dlm_preference_workspace_size(0, -1) == 0


def test_gradients_pairs(L):
    call = L.dlm_preference_grad
    assert call(*head({}), T, D(1.0), -1, STATE, None, BIG[1], 104, None, None) == INVALID
    assert call(*head({}), T, D(1.0), 2, None, None, BIG[1], 104, None, None) == INVALID
    assert call(*head(dict(n=0)), T, D(1.0), 2, STATE, None, BIG[1], 104, None, None) == 0
