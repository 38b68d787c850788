"""row_sample at the ends of its documented range: rows whose mass fills 64 bits,
and masked rows whose every finite logit is the lowest float.

Tokens are compared exactly.  Every weight of these rows is 1 or 0, so prob is
1 / n, to 2^-20 and where a nucleus' end may stay open to 2^-17 more.
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


def check(dlm, z, picks, u, **f):
    """Row picks[i] of z with u[i], stored at i; the kept weights are all 1."""
    wide = torch.full((z.shape[0], (z.shape[1] + 7) // 8 * 8), float("nan"), dtype=z.dtype, device="cuda")
    d = wide[:, :z.shape[1]]
    d.copy_(z)
    status, u = dlm.new_status(), u.astype(np.float32)
    r = dlm.row_sample(d, torch.from_numpy(u).cuda(), row_index=torch.from_numpy(picks.astype(np.int32)).cuda(),
                       gather=True, status=status, **f)
    assert int(status.item()) == 0
    token, prob = r.token.cpu().numpy(), r.prob.cpu().numpy()
    for q, row in enumerate(ref.host(z)):
        at, w = ref.kept(row, f.get("temperature", 1.0), f.get("top_k", 0), f.get("top_p", 1.0), f.get("min_p", 0.0))
        assert (w == 1).all()
        mine = np.nonzero(picks == q)[0]
        want = at[(u[mine].astype(np.float64) * len(at)).astype(np.int64)]
        np.testing.assert_array_equal(token[mine], want)
        np.testing.assert_allclose(prob[mine], 1 / len(at), rtol=2.0 ** -20 + 2.0 ** -17)


@pytest.mark.parametrize("n", [2, 400])  # a cluster per row; a CTA per row and a second launch
@pytest.mark.parametrize("f", [dict(), dict(top_p=0.9), dict(top_p=float(np.float32(1 - 2 ** -24))), dict(top_p=0.01),
                               dict(min_p=1.0), dict(top_p=0.9, min_p=0.9999999), dict(top_p=0.9, min_p=1.0),
                               dict(top_k=1000000, top_p=0.9), dict(top_k=1000000)], ids=str)
def test_mass_that_fills_64_bits(dlm, f, n):
    # 2^20 - 1 weights of 2^44 each; the margin of a first pass is 1.3 2^44
    z = ref.rows(2, 1048575, "f32", seed=5, boosted=0.0)
    g = np.random.default_rng(9)
    check(dlm, z, np.arange(n) % 2, g.random(n), temperature=1e30, **f)


@pytest.mark.parametrize("n", [3, 400])
@pytest.mark.parametrize("f", [dict(top_k=3000, top_p=0.9), dict(top_k=3000, top_p=0.5), dict(top_k=3000),
                               dict(top_k=3000, top_p=0.9, min_p=0.5), dict(top_k=2400, top_p=0.9),
                               dict(top_k=9999, top_p=0.9), dict(top_p=0.9), dict()], ids=str)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rows_masked_with_the_lowest_value(dlm, kind, f, n):
    g = np.random.default_rng(3)
    z = torch.full((3, 40000), -float("inf"), dtype=ref.TYPES[kind])
    for q, m in enumerate((2500, 2049, 30000)):
        z[q, torch.from_numpy(g.permutation(40000)[:m])] = torch.finfo(z.dtype).min
    check(dlm, z, np.arange(n) % 3, g.random(n), **f)


def test_status_words_elsewhere_are_refused(dlm):
    z, word = torch.zeros((2, 104), device="cuda"), torch.zeros(1, dtype=torch.int32)
    i, t = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros((2, 4), device="cuda")
    for call in (lambda s: dlm.row_topk(z, 4, status=s), lambda s: dlm.row_sample(z, z[:, 0].contiguous(), status=s),
                 lambda s: dlm.distill_loss(z, i, t, status=s), lambda s: dlm.distill_step(z, i, t, status=s),
                 lambda s: dlm.distill_grad(z, i, t, torch.zeros((2, 8), device="cuda"), status=s)):
        for bad in (word, torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")):
            with pytest.raises(ValueError):
                call(bad)
        call(dlm.new_status())
