"""Measured cases of the sampling, top-logit and distillation operators over vocab-wide logit rows.

Each case names its operator, its sizes and its storage type.  ``run`` computes
it either in its plain form (elementary torch operations) or, with ``own`` set,
through the package's public calls.  ``exact`` restates the definitions in
numpy and 64 bits.

Logit rows follow the decoding workloads' recipe: background N(0, 2^2) (the
smallest case N(0, 1)) and, for 60 % of the rows, one token raised so that its
softmax confidence is about sigmoid(u), u ~ U(4, 12).  The other rows stay
flat, as positions whose context is still masked are.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one block of 32 positions over a small vocabulary: launch latency
        {"name": "topk_block", "op": "topk", "rows": 32, "vocab": 1024, "type": "f32", "k": 16, "temperature": 1.0},
        # a teacher's rows for a batch of 64 sequences: its 64 largest logits are what is stored for training
        {"name": "topk_teacher", "op": "topk", "rows": 2048, "vocab": 152064, "type": "bf16", "k": 64,
         "temperature": 1.0},
        # log-probabilities of many alternatives for a few rows, odd vocabulary, tempered
        {"name": "topk_many", "op": "topk", "rows": 61, "vocab": 100003, "type": "f32", "k": 1000,
         "temperature": 0.7},
        # unfiltered sampling of one small block: launch latency
        {"name": "sample_block", "op": "sample", "rows": 32, "vocab": 1024, "type": "f32", "temperature": 1.0,
         "top_k": 0, "top_p": 1.0, "min_p": 0.0, "mixed": False, "subset": False},
        # one sequence's block of 32 positions per step of a decode
        {"name": "sample_step", "op": "sample", "rows": 32, "vocab": 126464, "type": "bf16", "temperature": 0.7,
         "top_k": 0, "top_p": 0.9, "min_p": 0.0, "mixed": False, "subset": False},
        # serving: 64 sequences, every one with settings of its own
        {"name": "sample_serving", "op": "sample", "rows": 2048, "vocab": 152064, "type": "bf16",
         "temperature": 1.0, "top_k": 50, "top_p": 0.95, "min_p": 0.05, "mixed": True, "subset": False},
        # nucleus sampling at temperature 1: on flat rows tens of thousands of tokens stay
        {"name": "sample_nucleus", "op": "sample", "rows": 2048, "vocab": 126464, "type": "bf16",
         "temperature": 1.0, "top_k": 0, "top_p": 0.95, "min_p": 0.0, "mixed": False, "subset": False},
        # the positions that are still masked late in a decode, picked out of the batch's rows
        {"name": "sample_late", "op": "sample", "rows": 203, "vocab": 16383, "type": "f16", "temperature": 0.6,
         "top_k": 0, "top_p": 1.0, "min_p": 0.05, "mixed": False, "subset": True},
        # evaluation of a student on held-out positions
        {"name": "distill_eval", "op": "distill_loss", "rows": 512, "vocab": 126464, "type": "bf16", "k": 64,
         "temperature": 1.0, "rest": False, "skip": 0},
        # training where another loss is added first: the gradient of the row losses comes from outside
        {"name": "distill_train", "op": "distill_train", "rows": 250, "vocab": 32003, "type": "f32", "k": 32,
         "temperature": 2.0, "rest": False, "skip": 0},
        # training step over a whole batch, the teacher's remaining mass as one more class, every fourth
        # position not masked and so without a loss
        {"name": "distill_step", "op": "distill_step", "rows": 2048, "vocab": 152064, "type": "bf16", "k": 64,
         "temperature": 1.0, "rest": True, "skip": 4},
        # the same over one small block with many teacher logits
        {"name": "distill_block", "op": "distill_step", "rows": 32, "vocab": 16384, "type": "f16", "k": 256,
         "temperature": 1.0, "rest": True, "skip": 0},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    rows, vocab = _log_uniform(rng, 1, 2048), _log_uniform(rng, 1000, 152064)
    kind = rng.choice(["f32", "bf16", "bf16", "f16"])
    if kind == "f32":
        rows = max(1, rows // 2)
    case = {"op": rng.choice(["topk", "sample", "sample", "distill_loss", "distill_train", "distill_step"]),
            "rows": rows, "vocab": vocab, "type": kind}
    if case["op"] == "sample":
        case |= {"temperature": round(rng.uniform(0.2, 1.3), 2), "top_k": rng.choice([0, 0, _log_uniform(rng, 1, 2000)]),
                 "top_p": rng.choice([1.0, round(rng.uniform(0.5, 0.99), 3)]),
                 "min_p": rng.choice([0.0, 0.0, round(rng.uniform(0.01, 0.3), 3)]),
                 "mixed": rng.random() < 0.3, "subset": rng.random() < 0.3}
    else:
        case |= {"k": _log_uniform(rng, 1, min(1024, vocab)), "temperature": rng.choice([1.0, round(rng.uniform(0.5, 3.0), 2)])}
        if case["op"] != "topk":
            case |= {"rest": rng.random() < 0.5, "skip": rng.choice([0, 0, 2, 5])}
    return case


def _logits(case, g, sigma, dtype, boosted):
    """[rows, vocab] rows at a stride that is a multiple of 16 bytes."""
    rows, vocab = case["rows"], case["vocab"]
    z = torch.empty((rows, (vocab + 7) // 8 * 8), dtype=dtype, device="cuda")[:, :vocab]
    step = max(1, (1 << 27) // vocab)
    mass = math.log(vocab) + sigma * sigma / 2
    for a in range(0, rows, step):
        n = min(step, rows - a)
        x = torch.randn((n, vocab), device="cuda", generator=g).mul_(sigma)
        u = torch.rand((n, 3), device="cuda", generator=g)
        at = (u[:, 0] * vocab).long().clamp_(max=vocab - 1)
        raised = torch.where(u[:, 1] < boosted, mass + 4 + 8 * u[:, 2], x.gather(1, at[:, None])[:, 0])
        z[a:a + n] = x.scatter_(1, at[:, None], raised[:, None])
    return z


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, rows, vocab = _TYPES[case["type"]], case["rows"], case["vocab"]
    sigma = 1.0 if vocab <= 1024 else 2.0
    z = _logits(case, g, sigma, dtype, 0.6)
    s = dict(case, logits=z)
    if case["op"] == "sample":
        n = rows
        if case["subset"]:  # two rows of three, picked at random, in ascending order
            n = (2 * rows + 2) // 3
            s["index"] = torch.randperm(rows, device="cuda", generator=g)[:n].sort().values.to(torch.int32)
        s["u"] = torch.rand(n, device="cuda", generator=g)
        if case["mixed"]:  # settings per request, 32 rows each
            r = torch.rand((n // 32 + 1, 4), device="cuda", generator=g).repeat_interleave(32, 0)[:n]
            pick = lambda j, v, t: torch.tensor(v, device="cuda", dtype=t)[(r[:, j] * len(v)).long().clamp_(max=len(v) - 1)]  # noqa: E731
            s["temperature"] = pick(0, [0.2, 0.5, 0.7, 0.8, 1.0, case["temperature"]], torch.float32)
            s["top_k"] = pick(1, [0, 20, case["top_k"], 200], torch.int32)
            s["top_p"] = pick(2, [0.8, 0.9, case["top_p"], 1.0], torch.float32)
            s["min_p"] = pick(3, [0.0, 0.0, case["min_p"]], torch.float32)
    elif case["op"] != "topk":
        # the teacher: the same positions, other values; its top logits are stored, shorter lists are padded
        t = z.float()
        t += torch.randn(t.shape, device="cuda", generator=g)
        top = torch.topk(t, case["k"], dim=1)
        s["ids"], s["teacher"] = top.indices.to(torch.int32), top.values.contiguous()
        if case["k"] >= 4:
            s["ids"][::7, -(case["k"] // 4):] = -1
        s["teacher_lse"] = torch.logsumexp(t / case["temperature"], 1) if case["rest"] else None
        s["weights"] = 0.5 + torch.rand(rows, device="cuda", generator=g)
        if case["skip"]:
            s["weights"][case["skip"] - 1::case["skip"]] = 0.0
        s["upstream"] = torch.randn(rows, device="cuda", generator=g)
    return s


def _per_row(v, n, dtype):
    return v.to(dtype) if torch.is_tensor(v) else torch.full((n,), v, dtype=dtype, device="cuda")


def _plain_topk(s):
    z = s["logits"].float()
    values, ids = torch.sort(z, dim=1, descending=True, stable=True)
    y = z / s["temperature"]
    m = y.amax(1, keepdim=True)
    lse = m[:, 0].double() + torch.exp(y - m).sum(1, dtype=torch.float64).log()
    return {"values": values[:, :s["k"]].contiguous(), "ids": ids[:, :s["k"]].to(torch.int32), "lse": lse.float()}


def _plain_sample(s):
    # 64 bits: the running sums are compared with borders that lie next to them
    z = s["logits"][s["index"].long()] if s["subset"] else s["logits"]
    n = z.shape[0]
    order = torch.sort(z.float(), dim=1, descending=True, stable=True)
    t = _per_row(s["temperature"], n, torch.float32).double()[:, None]
    k = _per_row(s["top_k"], n, torch.int64)[:, None]
    p = _per_row(s["top_p"], n, torch.float32).double()[:, None]
    least = _per_row(s["min_p"], n, torch.float32).double()[:, None]
    x = order.values.double()
    w = torch.exp((x - x[:, :1]) / t)
    rank = torch.arange(z.shape[1], device="cuda")[None]
    w_k = torch.where((k <= 0) | (rank < k), w, 0.0)
    mass = torch.cumsum(w_k, 1)
    before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], 1)
    keep = (w_k > 0) & ((p >= 1) | (before < p * mass[:, -1:])) & (w >= least)
    kept = torch.zeros_like(w).scatter_(1, order.indices, torch.where(keep, w, 0.0))
    cdf = torch.cumsum(kept, 1)
    token = torch.searchsorted(cdf, s["u"].double()[:, None] * cdf[:, -1:], right=True)
    token = torch.minimum(token, z.shape[1] - 1 - kept.flip(1).gt(0).to(torch.uint8).argmax(1, keepdim=True))
    prob = kept.gather(1, token) / cdf[:, -1:]
    return {"token": token[:, 0].to(torch.int32), "prob": prob[:, 0].float()}


def _plain_distill(s, gradient):
    z, t, w = s["logits"].float(), s["temperature"], s["weights"]
    y = z / t
    m = y.amax(1, keepdim=True)
    e = torch.exp(y - m)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    held = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    a = (s["teacher"].double() / t).masked_fill(~held, -math.inf)
    ref = s["teacher_lse"].double()[:, None] if s["rest"] else torch.log(torch.exp(a - a[:, :1]).sum(1, keepdim=True)) + a[:, :1]
    p = torch.exp(a - ref)
    log_q = y.gather(1, ids).double() - (m.double() + total.log())
    loss = torch.where(held & (p > 0), p * ((a - ref) - log_q), 0.0).sum(1)
    if s["rest"]:
        outside = torch.ones_like(e).scatter_(1, torch.where(held, ids, ids[:, :1]), 0.0)
        p_rest = (1 - p.sum(1)).clamp(min=0)
        q_rest = (e * outside).sum(1, dtype=torch.float64) / total[:, 0]
        loss = loss + torch.where(p_rest > 0, p_rest * (torch.log(p_rest) - torch.log(q_rest)), 0.0)
    loss = torch.where(w != 0, w * loss, 0.0).float()
    if gradient is None:
        return {"loss": loss}
    scale = (w * gradient / t)[:, None]
    q = e / total.float()
    base = q * (1 - p_rest / q_rest).float()[:, None] if s["rest"] else q
    at_ids = torch.where(held, q.gather(1, ids) - p.float(), base.gather(1, ids))
    ids = torch.where(held, ids, ids[:, :1])
    at_ids = torch.where(held, at_ids, at_ids[:, :1])
    grad = torch.where(scale != 0, scale * base.scatter(1, ids, at_ids), 0.0)
    return {"loss": loss, "grad": grad.to(s["logits"].dtype)}


def run(s):
    if own:
        import diffusion_decoding_token_gb300 as dlm
        if s["op"] == "topk":
            r = dlm.row_topk(s["logits"], s["k"], temperature=s["temperature"])
            return {"values": r.values, "ids": r.ids, "lse": r.lse}
        if s["op"] == "sample":
            r = dlm.row_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"], row_index=s.get("index"), gather=s["subset"])
            return {"token": r.token, "prob": r.prob}
        given = dict(teacher_lse=s["teacher_lse"], temperature=s["temperature"], weights=s["weights"])
        if s["op"] == "distill_step":
            loss, grad = dlm.distill_step(s["logits"], s["ids"], s["teacher"], **given)
            return {"loss": loss, "grad": grad}
        r = dlm.distill_loss(s["logits"], s["ids"], s["teacher"], **given)
        if s["op"] == "distill_loss":
            return {"loss": r.loss}
        grad = dlm.distill_grad(s["logits"], s["ids"], s["teacher"], r.state, s["upstream"],
                                temperature=s["temperature"], weights=s["weights"])
        return {"loss": r.loss, "grad": grad}
    if s["op"] == "topk":
        return _plain_topk(s)
    if s["op"] == "sample":
        return _plain_sample(s)
    upstream = {"distill_loss": None, "distill_step": torch.ones_like(s["weights"]), "distill_train": s["upstream"]}
    return _plain_distill(s, upstream[s["op"]])


def work(case):
    size = 4 if case["type"] == "f32" else 2
    rows, vocab = case["rows"], case["vocab"]
    cells = rows * vocab
    if case["op"] == "topk":
        # the maximum search and the log-sum-exp: compare, scale, exponential, add
        return {"bytes": cells * size + rows * (8 * case["k"] + 4), "flops": 4 * cells}
    if case["op"] == "sample":
        if case["subset"]:
            rows = (2 * rows + 2) // 3
            cells = rows * vocab
        return {"bytes": cells * size + rows * (28 if case["mixed"] else 12), "flops": 4 * cells}
    read = cells - (rows // case["skip"] * vocab if case["skip"] else 0)
    lists = rows * case["k"] * 8 + rows * 12
    if case["op"] == "distill_loss":
        return {"bytes": read * size + lists, "flops": 4 * read}
    return {"bytes": read * size + cells * size + lists, "flops": 6 * read}


def exact(case, seed):
    if case["rows"] * case["vocab"] > 3e7:
        return None  # minutes of sorting and exponentials on the host
    s = prepare(case, seed)
    host = {k: (v.cpu() if torch.is_tensor(v) else v) for k, v in s.items()}
    z = host["logits"].float().numpy().astype(np.float64)
    if case["op"] == "topk":
        return _exact_topk(z, case)
    if case["op"] == "sample":
        return _exact_sample(z, host, case)
    return _exact_distill(z, host, case)


def _exact_topk(z, case):
    ids = np.argsort(-z, axis=1, kind="stable")[:, :case["k"]].astype(np.int32)
    y = z / case["temperature"]
    m = y.max(1)
    lse = m + np.log(np.exp(y - m[:, None]).sum(1))
    return {"values": np.take_along_axis(z, ids.astype(np.int64), 1), "ids": ids, "lse": lse}


def _exact_sample(z, host, case):
    if case["subset"]:
        z = z[host["index"].numpy()]
    at = lambda name, r: float(host[name][r]) if torch.is_tensor(host[name]) else host[name]  # noqa: E731
    token, prob = np.zeros(len(z), np.int32), np.zeros(len(z))
    for r, row in enumerate(z):
        t, p, least = (float(np.float32(at(n, r))) for n in ("temperature", "top_p", "min_p"))
        k = int(at("top_k", r))
        ranked = np.argsort(-row, kind="stable")[:k if k > 0 else None]
        w = np.exp((row[ranked] - row[ranked[0]]) / t)
        ends = np.cumsum(w)
        n = len(w) if p >= 1 else 1 + int(np.searchsorted(ends[:-1], p * ends[-1], side="left"))
        n = min(n, int((w >= least).sum()))
        kept = np.sort(ranked[:n])
        w = np.exp((row[kept] - row[ranked[0]]) / t)
        ends = np.cumsum(w)
        j = min(int(np.searchsorted(ends, float(host["u"][r]) * ends[-1], side="right")), n - 1)
        token[r], prob[r] = kept[j], w[j] / ends[-1]
    return {"token": token, "prob": prob}


def _exact_distill(z, host, case):
    t = case["temperature"]
    loss, grad = np.zeros(len(z)), np.zeros_like(z)
    for r, row in enumerate(z):
        weight = float(host["weights"][r])
        if weight == 0:
            continue
        ids = host["ids"][r].numpy()
        a = host["teacher"][r].numpy().astype(np.float64)[ids >= 0] / t
        ids = ids[ids >= 0]
        y = row / t
        log_q = y - (y.max() + math.log(np.exp(y - y.max()).sum()))
        q = np.exp(log_q)
        log_p = a - (float(host["teacher_lse"][r]) if case["rest"] else a.max() + math.log(np.exp(a - a.max()).sum()))
        p = np.exp(log_p)
        value, slope = (p * (log_p - log_q[ids])).sum(), q.copy()
        if case["rest"]:
            others = np.ones(len(row), bool)
            others[ids] = False
            p_rest, q_rest = max(0.0, 1 - p.sum()), q[others].sum()
            if p_rest > 0:
                value += p_rest * (math.log(p_rest) - (math.log(q_rest) if q_rest > 0 else -math.inf))
                slope[others] *= 1 - p_rest / q_rest
        slope[ids] -= p
        loss[r] = weight * value
        grad[r] = slope * weight / t * (float(host["upstream"][r]) if case["op"] == "distill_train" else 1.0)
    return {"loss": loss} if case["op"] == "distill_loss" else {"loss": loss, "grad": grad}
