"""row_topk and row_sample against 64-bit numpy, over the sizes, filters and
masks where they can go wrong.

Tolerances.  Tokens and ids are compared exactly.  prob is one weight over the
kept mass: exp2f (2 ulp), a product, a 64-bit sum rounded to float and a
division, 2^-20 in all; where a nucleus is too long for a list, which token ends
it may stay open while the mass of the open ones is at most 2^-17 of the kept
mass, so there prob is within 2^-17 more.  lse: the 32-bit sum of exponentials is within 2^-18
(ex2 2^-22, an exponent of up to ~20 rounded three times at 2^-24, ten levels
of additions), and the float result and m / T round at 2^-23 of their value.
"""
import numpy as np
import pytest
import torch

import row_ref as ref

pytestmark = pytest.mark.gpu

PROB_RTOL = 2.0 ** -20
LIST = 64  # shorter nuclei always fit a candidate list


@pytest.fixture(scope="module")
def dlm():
    import diffusion_decoding_token_gb300 as d
    d.lib()
    return d


def check_topk(dlm, z, k, temperature=1.0, **kw):
    d = z.cuda()
    if z.stride(0) != z.shape[1]:
        wide = torch.empty((z.shape[0], z.stride(0)), dtype=z.dtype, device="cuda")
        d = wide[:, :z.shape[1]]
        d.copy_(z)
    status = dlm.new_status()
    r = dlm.row_topk(d, k, temperature=temperature, status=status, **kw)
    assert int(status.item()) == 0
    zz = ref.host(z)
    for i, row in enumerate(zz):
        values, ids, lse = ref.topk(row, k, temperature)
        np.testing.assert_array_equal(r.ids[i].cpu().numpy(), ids, err_msg=f"row {i}")
        np.testing.assert_array_equal(r.values[i].cpu().numpy().astype(np.float64), values)
        assert abs(float(r.lse[i]) - lse) <= 2.0 ** -18 + 2.0 ** -22 * (abs(lse) + abs(row.max() / temperature))


def on_gpu(z):
    """The same rows at the same stride."""
    wide = torch.full((z.shape[0], z.stride(0)), float("nan"), dtype=z.dtype, device="cuda")
    d = wide[:, :z.shape[1]]
    d.copy_(z)
    return d


def check_sample(dlm, z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mixed=False):
    status = dlm.new_status()
    n = z.shape[0]
    dev = lambda v, t: torch.as_tensor(v, dtype=t).cuda() if mixed else v  # noqa: E731
    r = dlm.row_sample(on_gpu(z), torch.from_numpy(u.astype(np.float32)).cuda(),
                       temperature=dev(temperature, torch.float32), top_k=dev(top_k, torch.int32),
                       top_p=dev(top_p, torch.float32), min_p=dev(min_p, torch.float32), status=status)
    assert int(status.item()) == 0
    at = lambda v, i: v[i] if mixed else v  # noqa: E731
    token, prob = r.token.cpu().numpy(), r.prob.cpu().numpy()
    for i, row in enumerate(ref.host(z)):
        want, p = ref.sample(row, u[i], at(temperature, i), at(top_k, i), at(top_p, i), at(min_p, i))
        assert token[i] == want, (i, token[i], want)
        kept = len(ref.kept(row, *(at(v, i) for v in (temperature, top_k, top_p, min_p)))[0])
        open_end = 2.0 ** -17 if kept > LIST and at(top_p, i) < 1 else 0.0
        assert abs(prob[i] - p) <= (PROB_RTOL + open_end) * p, (i, prob[i], p)
    return r


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,vocab,k", [(1, 1, 1), (3, 2, 5), (2, 7, 7), (5, 129, 16), (4, 1000, 1000), (3, 1024, 64),
                                       (2, 4097, 1024), (6, 5003, 3), (3, 32003, 128), (2, 126464, 1024),
                                       (330, 2050, 20)])
def test_topk(dlm, kind, n, vocab, k):
    check_topk(dlm, ref.rows(n, vocab, kind, seed=vocab + k, pad=n % 3), k)


@pytest.mark.parametrize("temperature", [0.1, 0.7, 3.0])
def test_topk_tempered_lse(dlm, temperature):
    check_topk(dlm, ref.rows(4, 9001, "f32", seed=5), 10, temperature)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_topk_ties(dlm, kind):
    z = torch.zeros((4, 20000), dtype=ref.TYPES[kind])      # every logit equal: positions 0 .. k-1
    z[1, 15000:] = 1.0                                      # the top lies in one half
    z[2, ::7] = 2.0                                         # more ties than a candidate list holds
    z[3] = -0.0
    z[3, 5::11] = 0.0                                       # -0 and +0 are equal
    for k in (1, 100, 1024):
        check_topk(dlm, z, k)


def test_topk_few_finite(dlm):
    z = ref.rows(4, 6000, "f32", seed=9)
    z[0, 1:] = -float("inf")
    z[1, 40:] = -float("inf")
    z[2] = torch.finfo(torch.float32).min
    z[2, 17] = -1e30
    z[3, :5990] = torch.finfo(torch.float32).min
    check_topk(dlm, z, 64)
    check_topk(dlm, z, 1024)


def test_topk_rows_that_have_no_maximum(dlm):
    z = ref.rows(4, 3000, "bf16", seed=2).contiguous()
    z[0] = -float("inf")
    z[1, 100] = float("nan")
    z[2, 7] = float("inf")
    status = dlm.new_status()
    r = dlm.row_topk(z.cuda(), 8, status=status)
    assert int(status.item()) == dlm.DEV_NONFINITE
    assert (r.ids[:3] == -1).all() and torch.isinf(r.values[:3]).all()
    assert float(r.lse[0]) == -float("inf") and torch.isnan(r.lse[1]) and float(r.lse[2]) == float("inf")
    np.testing.assert_array_equal(r.ids[3].cpu().numpy(), ref.topk(ref.host(z)[3], 8)[1])


@pytest.mark.parametrize("gather", [False, True])
def test_row_index(dlm, gather):
    z = ref.rows(9, 2000, "f16", seed=3)
    index = torch.tensor([8, 0, 5, -1, 3, 9, 5], dtype=torch.int32)
    status = dlm.new_status()
    m = len(index) if gather else 9
    out = dlm.RowTopk(torch.full((m, 4), 7.0, device="cuda"), torch.full((m, 4), -7, dtype=torch.int32, device="cuda"),
                      torch.full((m,), 7.0, device="cuda"))
    r = dlm.row_topk(on_gpu(z), 4, row_index=index.cuda(), gather=gather, out=out, status=status)
    assert int(status.item()) == dlm.DEV_BAD_INDEX
    u = torch.rand(m, generator=torch.Generator().manual_seed(1))
    tok = dlm.RowSample(torch.full((m,), -7, dtype=torch.int32, device="cuda"), torch.full((m,), 7.0, device="cuda"), None)
    s = dlm.row_sample(on_gpu(z), u.cuda(), top_p=0.9, row_index=index.cuda(), gather=gather, out=tok)
    zz, written = ref.host(z), set()
    for i, q in enumerate(index.tolist()):
        if not 0 <= q < 9:
            continue
        o = i if gather else q
        written.add(o)
        np.testing.assert_array_equal(r.ids[o].cpu().numpy(), ref.topk(zz[q], 4)[1])
        assert int(s.token[o]) == ref.sample(zz[q], float(u[o]), top_p=0.9)[0]
    for o in set(range(m)) - written:  # left as they were
        assert (r.ids[o] == -7).all() and (r.values[o] == 7.0).all() and float(r.lse[o]) == 7.0
        assert int(s.token[o]) == -7 and float(s.prob[o]) == 7.0


FILTERS = [dict(), dict(top_p=0.9), dict(top_p=0.5, temperature=0.7), dict(top_k=1), dict(top_k=50),
           dict(top_k=50, top_p=0.95, min_p=0.05, temperature=0.8), dict(min_p=0.1), dict(min_p=1.0),
           dict(min_p=1e-6), dict(top_p=0.999, min_p=0.02, temperature=1.3), dict(top_k=1500, top_p=0.97),
           dict(top_k=1024), dict(temperature=0.0), dict(temperature=0.2, top_p=0.9), dict(temperature=2.0),
           dict(top_k=3000, min_p=1e-4), dict(top_k=700, top_p=0.3, temperature=5.0), dict(top_p=1e-6)]


@pytest.mark.parametrize("f", FILTERS, ids=lambda f: ",".join(f"{k}={v}" for k, v in f.items()) or "none")
@pytest.mark.parametrize("kind,n,vocab", [("f32", 6, 1), ("f32", 7, 130), ("bf16", 12, 2500), ("f32", 9, 5001),
                                          ("bf16", 40, 40001), ("f16", 6, 126464)])
def test_sample(dlm, kind, n, vocab, f):
    z = ref.rows(n, vocab, kind, seed=vocab + n)
    check_sample(dlm, z, np.random.default_rng(n + vocab).random(n), **f)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("f", [dict(), dict(top_p=0.95), dict(top_p=0.99, temperature=1.5), dict(top_k=2000)],
                         ids=["none", "p95", "p99t15", "k2000"])
def test_sample_flat_rows(dlm, kind, f):
    # every row flat: borders lie within the error of 32-bit sums in many
    z = ref.rows(640, 20011, kind, seed=77, sigma=1.0, boosted=0.0)
    check_sample(dlm, z, np.random.default_rng(4).random(640), **f)


def test_sample_per_row_settings(dlm):
    n = 96
    g = np.random.default_rng(8)
    z = ref.rows(n, 9000, "bf16", seed=8)
    check_sample(dlm, z, g.random(n), temperature=g.choice(np.float32([0.0, 0.3, 0.7, 1.0, 1.4]), n),
                 top_k=g.choice([0, 1, 20, 1200, 9000], n), top_p=g.choice(np.float32([0.5, 0.9, 1.0]), n),
                 min_p=g.choice(np.float32([0.0, 0.05, 0.3]), n), mixed=True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("f", [dict(), dict(top_p=0.25), dict(top_k=1500), dict(top_k=10, top_p=0.35),
                               dict(min_p=0.9), dict(top_k=2500, top_p=0.9)], ids=str)
def test_sample_ties(dlm, kind, f):
    z = torch.zeros((5, 12000), dtype=ref.TYPES[kind])
    z[1, 6000:] = 0.5
    z[2, ::3] = 1.0
    z[3] = torch.finfo(ref.TYPES[kind]).min
    z[4, 100:] = -float("inf")
    check_sample(dlm, z, np.array([0.3, 0.71, 0.999, 0.5, 0.25]), **f)


@pytest.mark.parametrize("f", FILTERS, ids=str)
def test_sample_ends_of_u(dlm, f):
    # u = 0: the first kept position; the largest u: the last one with weight
    z = ref.rows(8, 3001, "f32", seed=31, sigma=1.0)
    z[4:, :50] = -float("inf")
    u = np.array([0.0, np.float32(1 - 2 ** -24), 2.0 ** -24, 1e-30] * 2)
    check_sample(dlm, z, u, **f)


def test_sample_conf(dlm):
    z = ref.rows(40, 7000, "bf16", seed=12)
    d = on_gpu(z)
    st = dlm.row_stats(d)
    u = torch.rand(40, device="cuda")
    r = dlm.row_sample(d, u, temperature=0.7, top_p=0.9, lse=st.lse)
    zz = ref.host(z)
    for i, row in enumerate(zz):
        p = np.exp(row - row.max())
        want = p[int(r.token[i])] / p.sum()
        # lse is held to 1e-4 elsewhere; here 2^-18 plus its own rounding, and expf
        assert abs(float(r.conf[i]) - want) <= want * (2.0 ** -18 + 2.0 ** -23 * abs(float(st.lse[i])) + 2.0 ** -21)


def test_sample_rows_out_of_range(dlm):
    n = 10
    z = ref.rows(n, 2100, "f32", seed=6).contiguous()
    z[7] = -float("inf")
    z[8, 3] = float("nan")
    z[9, 3] = float("inf")
    u = np.full(n, 0.5, np.float32)
    u[0], u[1], u[2] = 1.0, -0.1, np.nan
    t = np.ones(n, np.float32)
    t[3], t[4] = -1.0, np.inf
    p = np.full(n, 0.9, np.float32)
    p[5] = 0.0
    k = np.zeros(n, np.int32)
    k[6] = -1
    status = dlm.new_status()
    c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    r = dlm.row_sample(z.cuda(), c(u), temperature=c(t), top_p=c(p), top_k=c(k), status=status)
    assert (r.token == -1).all() and (r.prob == 0).all()
    assert int(status.item()) == dlm.DEV_BAD_PARAM | dlm.DEV_NONFINITE


def test_sample_is_the_same_on_every_launch_and_in_a_graph(dlm):
    z = on_gpu(ref.rows(64, 30011, "bf16", seed=21, boosted=0.3))
    u = torch.rand(64, device="cuda")
    first = dlm.row_sample(z, u, top_p=0.95)
    out = dlm.RowSample(torch.empty_like(first.token), torch.empty_like(first.prob), None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        dlm.row_sample(z, u, top_p=0.95, out=out)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            dlm.row_sample(z, u, top_p=0.95, out=out)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        out.token.fill_(-5)
        g.replay()
        assert torch.equal(out.token, first.token) and torch.equal(out.prob, first.prob)


@pytest.mark.parametrize("f", [dict(), dict(top_p=0.95), dict(top_p=0.9, temperature=0.7), dict(min_p=1e-3)], ids=str)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_sample_next_to_a_border(dlm, kind, f):
    # u chosen so that u * mass lies 1e-10 .. 1e-8 of the mass from a border of
    # the running sum, on both sides: 32-bit sums (1e-7) can not tell, the
    # integer weights (1e-11) can
    n = 24
    z = ref.rows(n, 20011, kind, seed=91, sigma=1.0, boosted=0.0)
    u, g = np.zeros(n, np.float32), np.random.default_rng(5)
    for r, row in enumerate(ref.host(z)):
        at, w = ref.kept(row, f.get("temperature", 1.0), 0, f.get("top_p", 1.0), f.get("min_p", 0.0))
        borders = np.cumsum(w)[:-1] / w.sum()
        near = borders.astype(np.float32)
        off = near.astype(np.float64) - borders
        ok = (np.abs(off) > 1e-10) & (np.abs(off) < 1e-8) & ((off > 0) == (r % 2 == 0))
        u[r] = g.choice(near[ok])
    check_sample(dlm, z, u.astype(np.float64), **f)


@pytest.mark.parametrize("gather", [False, True])
def test_sample_rows_listed_twice(dlm, gather):
    # enough rows for one CTA each, so that the open ones go to the second launch
    n, vocab = 700, 20011
    z = ref.rows(n, vocab, "bf16", seed=17, sigma=1.0, boosted=0.2)
    g = np.random.default_rng(6)
    index = g.integers(0, n, n).astype(np.int32)
    u = g.random(n).astype(np.float32)
    d = on_gpu(z)
    r = dlm.row_sample(d, torch.from_numpy(u).cuda(), top_p=0.95, row_index=torch.from_numpy(index).cuda(), gather=gather)
    zz = ref.host(z)
    for i in g.choice(n, 120, replace=False):
        o = i if gather else index[i]
        assert int(r.token[o]) == ref.sample(zz[index[i]], float(u[o]), top_p=0.95)[0]


def test_two_streams_at_once(dlm):
    z = [on_gpu(ref.rows(400, 20011, "bf16", seed=s, boosted=0.3)) for s in (1, 2)]
    u = torch.rand(400, device="cuda")
    want = [dlm.row_sample(x, u, top_p=0.95).token.clone() for x in z]
    streams = [torch.cuda.Stream() for _ in z]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for x, st in zip(z, streams):
            with torch.cuda.stream(st):
                got.append(dlm.row_sample(x, u, top_p=0.95).token)
    torch.cuda.synchronize()
    for i, t in enumerate(got):
        assert torch.equal(t, want[i % 2])


@pytest.mark.parametrize("n,vocab", [(6, 20012), (330, 20012), (330, 3000)])
@pytest.mark.parametrize("f", [dict(top_p=0.9, temperature=1e-4), dict(top_p=0.3, temperature=1e-4), dict(temperature=1e-4), dict(min_p=1e-6, temperature=1e-4),
                               dict(top_p=0.9, temperature=0.01), dict(top_p=0.5, temperature=1e30),
                               dict(min_p=0.5, temperature=1e30), dict(temperature=1e30),
                               dict(top_k=3000, temperature=1e-4)], ids=str)
def test_sample_far_from_zero(dlm, n, vocab, f):
    # logits whose place is far above the temperature: a step of the type is
    # many powers of e, and thousands of tokens share the maximum
    g = np.random.default_rng(11)
    z = torch.zeros((n, vocab), dtype=torch.float32)
    z[0::6] = 1e6 - torch.from_numpy((g.random((n // 6, vocab)) > 0.8).astype(np.float32))
    z[1::6] = -1e30
    z[1::6, ::3] = -0.999e30
    z[2::6] = 1e5 + torch.from_numpy(g.integers(0, 64, (n // 6, vocab)).astype(np.float32)) / 128
    z[3::6] = 1000 + torch.from_numpy(g.integers(0, 64, (n // 6, vocab)).astype(np.float32)) / 16384
    z[4::6] = torch.from_numpy(g.normal(0, 1e-4, (n // 6, vocab)).astype(np.float32))
    z[5::6] = 3e38
    z[5::6, 1::2] = -3e38
    check_sample(dlm, z, g.random(n), **f)


@pytest.mark.parametrize("kind,vocab", [("f32", 1048575), ("bf16", 1000001)])
def test_largest_vocabularies(dlm, kind, vocab):
    z = ref.rows(2, vocab, kind, seed=3)
    check_topk(dlm, z, 300)
    for f in (dict(), dict(top_p=0.9), dict(top_k=40, min_p=0.01)):
        check_sample(dlm, z, np.array([0.31, 0.87]), **f)


def test_refusals(dlm):
    z = on_gpu(ref.rows(4, 100, "f32", seed=1))
    u = torch.zeros(4, device="cuda")
    with pytest.raises(dlm.DlmError):
        dlm.row_topk(z, 0)
    with pytest.raises(dlm.DlmError):
        dlm.row_topk(z, dlm.MAX_TOPK + 1)
    with pytest.raises(dlm.DlmError):
        dlm.row_topk(z, 4, temperature=0.0)
    for bad in (dict(temperature=-1.0), dict(temperature=2e30), dict(temperature=float("nan")), dict(top_k=-1), dict(top_p=0.0),
                dict(top_p=1.5), dict(min_p=-0.1), dict(min_p=1.1)):
        with pytest.raises(dlm.DlmError):
            dlm.row_sample(z, u, **bad)
    with pytest.raises(ValueError):
        dlm.row_sample(z, u[:3])
    with pytest.raises(ValueError):
        dlm.row_sample(z, u, top_k=torch.zeros(4, device="cuda"))  # not int32
    with pytest.raises(ValueError):
        dlm.row_sample(z.double(), u)
    with pytest.raises(ValueError):
        dlm.row_sample(z.t(), u)
    with pytest.raises(dlm.DlmError):
        dlm.row_topk(torch.zeros((4, 101), device="cuda"), 4)   # rows not at 16 bytes
    assert dlm.row_topk(z[:0], 4).ids.shape == (0, 4)
