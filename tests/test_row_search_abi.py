"""Host-side refusals of the row search and distillation calls: status codes
before anything touches a GPU (no device needed)."""
import ctypes

import pytest

INVALID, ALIGN, UNSUP = 1, 2, 3
P = ctypes.c_void_p
F = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    from diffusion_decoding_token_gb300 import build
    build.build()
    import diffusion_decoding_token_gb300 as d
    return d.lib()


X = P(0x100000)
Y = P(0x10000000)
U = P(0x400000)


def topk(L, logits=X, dtype=1, n=4, vocab=100, stride=104, index=None, n_src=0, k=8, t=1.0, values=X, ids=X, flags=0):
    return L.dlm_row_topk(logits, dtype, n, vocab, stride, index, n_src, k, F(t), values, ids, X, None, flags, None)


def test_topk(L):
    assert topk(L, n=0) == 0
    assert topk(L, dtype=5) == UNSUP
    for kw in (dict(logits=None), dict(n=-1), dict(vocab=0), dict(vocab=105), dict(vocab=1 << 20, stride=1 << 20),
               dict(n_src=-1), dict(n_src=3), dict(k=0), dict(k=1025), dict(t=0.0), dict(t=5e-5), dict(t=float("inf")),
               dict(t=float("nan")), dict(t=-1.0), dict(t=2e30), dict(values=None), dict(ids=None), dict(flags=1), dict(flags=4),
               dict(n=1 << 31)):
        assert topk(L, **kw) == INVALID, kw
    assert topk(L, logits=P(0x100008)) == ALIGN
    assert topk(L, stride=101) == ALIGN


def sample(L, u=U, t=1.0, k=0, p=1.0, m=0.0, lse=None, conf=None, token=P(0x200000), prob=P(0x300000), n=4, rows=None, params=True, **kw):
    from diffusion_decoding_token_gb300._binding import SampleParams
    prm = SampleParams(t, k, p, m, *(rows or (None,) * 4))
    a = dict(dtype=1, vocab=100, stride=104, flags=0) | kw
    return L.dlm_row_sample(X, a["dtype"], n, a["vocab"], a["stride"], None, 0, u, ctypes.byref(prm) if params else None,
                            lse, token, prob, conf, None, a["flags"], None)


def test_sample(L):
    assert sample(L, n=0) == 0 and sample(L, n=0, t=0.0) == 0
    assert sample(L, dtype=3) == UNSUP
    for kw in (dict(params=False), dict(u=None), dict(t=-0.1), dict(t=1e-5), dict(t=2e30), dict(t=float("nan")), dict(k=-1),
               dict(p=0.0), dict(p=1.01), dict(p=float("nan")), dict(m=-0.1), dict(m=1.01), dict(lse=X), dict(conf=X),
               dict(token=None), dict(prob=None), dict(vocab=200), dict(flags=2 | 8), dict(prob=U), dict(token=U),
               dict(rows=(None, None, None, 0x200000)), dict(rows=(None, 0x300000, None, None))):
        assert sample(L, **kw) == INVALID, kw
    # a setting that comes per row is not checked here
    assert sample(L, n=0, t=-1.0, k=-1, p=7.0, m=7.0, rows=(0x1000,) * 4) == 0
    assert sample(L, stride=102) == ALIGN


def distill(L, call="loss", student=X, dtype=1, n=4, vocab=100, stride=104, ids=X, teacher=X, tdtype=0, k=8, t=1.0,
            loss=X, state=X, grad=Y, gstride=104):
    head = (student, dtype, n, vocab, stride, ids, teacher, tdtype, k)
    if call == "loss":
        return L.dlm_distill_loss(*head, None, ctypes.c_double(t), None, loss, state, None, None)
    if call == "grad":
        return L.dlm_distill_grad(*head, ctypes.c_double(t), None, state, None, grad, gstride, None, None)
    return L.dlm_distill_step(*head, None, ctypes.c_double(t), None, loss, grad, gstride, None, None)


@pytest.mark.parametrize("call", ["loss", "grad", "step"])
def test_distill(L, call):
    assert distill(L, call, n=0) == 0
    assert distill(L, call, dtype=3) == UNSUP and distill(L, call, tdtype=9) == UNSUP
    for kw in (dict(student=None), dict(ids=None), dict(teacher=None), dict(k=0), dict(k=1025), dict(t=0.0), dict(t=2e30),
               dict(t=float("nan")), dict(n=-1), dict(vocab=0), dict(vocab=105), dict(vocab=1 << 20, stride=1 << 20)):
        assert distill(L, call, **kw) == INVALID, kw
    assert distill(L, call, student=P(0x100002)) == ALIGN
    assert distill(L, call, stride=103) == ALIGN
    if call != "grad":
        assert distill(L, call, loss=None) == INVALID
    if call == "grad":
        assert distill(L, call, state=None) == INVALID
    if call != "loss":
        assert distill(L, call, grad=None) == INVALID
        assert distill(L, call, gstride=96) == INVALID
        assert distill(L, call, gstride=101) == ALIGN
        assert distill(L, call, grad=P(0x10000008)) == ALIGN
        # memory that overlaps the student without being the same rows
        assert distill(L, call, grad=P(0x100000 + 208)) == INVALID
        assert distill(L, call, grad=P(0x100000 - 208)) == INVALID
        assert distill(L, call, grad=X, gstride=112) == INVALID


def test_the_gradient_takes_its_own_memory_only():
    # the student as one position of a model's [batch, positions, vocabulary]
    import torch
    from diffusion_decoding_token_gb300 import _binding
    for dtype, vocab, padded in ((torch.float32, 1001, 1004), (torch.bfloat16, 1000, 1000), (torch.float16, 1001, 1008)):
        student = torch.empty((4, 50, padded), dtype=dtype)[:, 7, :vocab]
        grad = _binding._grad_out(student, None)
        assert grad.shape == student.shape and grad.dtype == dtype and grad.stride() == (padded, 1)
        assert grad.untyped_storage().nbytes() <= 4 * padded * grad.element_size()


def test_a_status_word_is_on_the_kernels_device():
    # (a host address would be written by the GPU)
    import torch
    from diffusion_decoding_token_gb300 import _binding
    here, word = torch.device("cpu"), torch.zeros(1, dtype=torch.int32)
    assert _binding._status_ptr(None, here) is None
    assert _binding._status_ptr(word, here) == word.data_ptr()
    for bad, device in ((word, torch.device("cuda", 0)), (word[:0], here), (word.long(), here), (word.float(), here)):
        with pytest.raises(ValueError):
            _binding._status_ptr(bad, device)


def test_sampled_tokens_and_their_inputs_do_not_overlap(L):
    # n = 1000 entries of 4 bytes each; token at 0x200000, prob at 0x300000
    at = lambda x: P(x)  # noqa: E731
    for kw in (dict(u=at(0x200000 + 3996)), dict(u=at(0x200000 - 3996)), dict(u=at(0x300000 + 4)),
               dict(prob=at(0x200000)), dict(prob=at(0x200000 + 2000)), dict(lse=X, conf=at(0x200000 + 4)),
               dict(lse=X, conf=at(0x300000)), dict(lse=at(0x300000 + 3996), conf=Y),
               dict(rows=(None, 0x200000 + 3996, None, None)), dict(rows=(0x300000 - 3996, None, None, None))):
        assert sample(L, n=1000, **kw) == INVALID, kw
