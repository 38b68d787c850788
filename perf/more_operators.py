"""Measured cases of the operators that train or score given tokens over vocab-wide logit rows.

Three operators: the log-probability of one token per row, the clipped policy
loss with a KL term, and the preference loss of paired sequences, each alone and
with its gradient.  Each case names its operator, its sizes and its storage type.
``run`` computes it either in its plain form (elementary torch operations) or,
with ``own`` set, through the package's public calls.  ``exact`` restates the
definitions in 64 bits.

Logit rows follow the decoding workloads' recipe: background N(0, 2^2) (vocabularies
up to 1024: N(0, 1)) and, for 60 % of the rows, one token raised so that its softmax
confidence is about sigmoid(u), u ~ U(4, 12).  The tokens are samples of the rows, as
a rollout's are.  Their log-probabilities under the policy that made the rollout and
under the reference policy lie around those of the rows (N(0, 0.2^2), N(0, 0.3^2)).
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # log-probabilities of one block's tokens over a small vocabulary: launch latency
        {"name": "logprob_block", "op": "logprob", "rows": 32, "vocab": 1024, "type": "f32", "temperature": 1.0,
         "subset": False},
        # a whole batch of 64 sequences scored under the reference policy
        {"name": "logprob_score", "op": "logprob", "rows": 2048, "vocab": 152064, "type": "bf16", "temperature": 1.0,
         "subset": False},
        # the positions that are still masked late in a decode, picked out of the batch's rows, odd vocabulary
        {"name": "logprob_late", "op": "logprob", "rows": 203, "vocab": 16383, "type": "f16", "temperature": 0.6,
         "subset": True},
        # the likelihood bound's training step: tokens weighted by 1 / t, every fourth position not masked
        {"name": "logprob_step", "op": "logprob_step", "rows": 512, "vocab": 126464, "type": "bf16",
         "temperature": 1.0, "skip": 4},
        # policy step on one small block: launch latency
        {"name": "policy_block", "op": "policy_step", "rows": 32, "vocab": 16384, "type": "f16", "temperature": 1.0,
         "dual": 0.0, "kl_weight": 0.04, "kl": "k3", "skip": 0},
        # policy step over a whole batch, every fourth position not masked and so without a loss
        {"name": "policy_step", "op": "policy_step", "rows": 2048, "vocab": 152064, "type": "bf16",
         "temperature": 1.0, "dual": 0.0, "kl_weight": 0.04, "kl": "k3", "skip": 4},
        # loss and clipping statistics of held-out rollouts
        {"name": "policy_eval", "op": "policy_loss", "rows": 512, "vocab": 126464, "type": "bf16", "temperature": 1.0,
         "dual": 3.0, "kl_weight": 0.1, "kl": "k2", "skip": 0},
        # training where another loss is added first: the gradient of the row losses comes from outside
        {"name": "policy_train", "op": "policy_train", "rows": 250, "vocab": 32003, "type": "f32", "temperature": 0.8,
         "dual": 3.0, "kl_weight": 0.04, "kl": "k3", "skip": 5},
        # two pairs of short answers: launch latency
        {"name": "preference_block", "op": "preference_step", "rows": 48, "vocab": 16384, "type": "f16", "pairs": 2,
         "temperature": 1.0, "kind": "sigmoid", "smooth": 0.0, "free": False},
        # a batch of pairs of ragged length
        {"name": "preference_step", "op": "preference_step", "rows": 1024, "vocab": 126464, "type": "bf16", "pairs": 8,
         "temperature": 1.0, "kind": "sigmoid", "smooth": 0.1, "free": False},
        # two pairs of long answers
        {"name": "preference_long", "op": "preference_step", "rows": 2048, "vocab": 152064, "type": "bf16", "pairs": 2,
         "temperature": 1.0, "kind": "ipo", "smooth": 0.0, "free": False},
        # loss and gradient apart, the gradient of the pair losses coming from outside, odd vocabulary
        {"name": "preference_train", "op": "preference_train", "rows": 331, "vocab": 32003, "type": "f32", "pairs": 16,
         "temperature": 1.0, "kind": "hinge", "smooth": 0.0, "free": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    rows, vocab = _log_uniform(rng, 2, 2048), _log_uniform(rng, 1000, 152064)
    kind = rng.choice(["f32", "bf16", "bf16", "f16"])
    if kind == "f32":
        rows = max(2, rows // 2)
    case = {"op": rng.choice(["logprob", "logprob_step", "policy_loss", "policy_train", "policy_step",
                              "preference_step", "preference_step", "preference_train"]),
            "rows": rows, "vocab": vocab, "type": kind,
            "temperature": rng.choice([1.0, 1.0, round(rng.uniform(0.5, 1.5), 2)])}
    if case["op"] == "logprob":
        case |= {"subset": rng.random() < 0.4}
    elif case["op"].startswith("preference"):
        case |= {"pairs": _log_uniform(rng, 1, max(1, rows // 4)), "kind": rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"]),
                 "smooth": rng.choice([0.0, 0.1]), "free": rng.random() < 0.3}
    else:
        case |= {"skip": rng.choice([0, 0, 2, 4, 5])}
        if case["op"] != "logprob_step":
            case |= {"dual": rng.choice([0.0, 3.0]), "kl_weight": rng.choice([0.0, 0.04, 0.2]),
                     "kl": rng.choice(["k1", "k2", "k3", "k3"])}
    return case


def _logits(case, g):
    """[rows, vocab] rows at a stride that is a multiple of 16 bytes, one sampled token of each and its log-probability."""
    rows, vocab = case["rows"], case["vocab"]
    sigma = 1.0 if vocab <= 1024 else 2.0
    z = torch.empty((rows, (vocab + 7) // 8 * 8), dtype=_TYPES[case["type"]], device="cuda")[:, :vocab]
    token = torch.empty(rows, dtype=torch.int64, device="cuda")
    lp = torch.empty(rows, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // vocab)
    mass = math.log(vocab) + sigma * sigma / 2
    for a in range(0, rows, step):
        n = min(step, rows - a)
        x = torch.randn((n, vocab), device="cuda", generator=g).mul_(sigma)
        u = torch.rand((n, 3), device="cuda", generator=g)
        at = (u[:, 0] * vocab).long().clamp_(max=vocab - 1)
        raised = torch.where(u[:, 1] < 0.6, mass + 4 + 8 * u[:, 2], x.gather(1, at[:, None])[:, 0])
        z[a:a + n] = x.scatter_(1, at[:, None], raised[:, None])
        # the largest of y plus Gumbel noise is a sample of softmax(y)
        x = z[a:a + n].float() / case["temperature"]
        noise = torch.empty_like(x).exponential_(generator=g).clamp_(min=1e-30).log_()
        token[a:a + n] = (x - noise).argmax(1)
        lp[a:a + n] = x.gather(1, token[a:a + n, None])[:, 0] - x.logsumexp(1)
    return z, token, lp


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = case["rows"]
    z, token, lp = _logits(case, g)
    s = dict(case, logits=z, tokens=token.to(torch.int32))
    normal = lambda n, sigma: torch.randn(n, device="cuda", generator=g) * sigma  # noqa: E731
    if case["op"] == "logprob":
        if case["subset"]:  # two rows of three, picked at random, in ascending order
            n = (2 * rows + 2) // 3
            s["index"] = torch.randperm(rows, device="cuda", generator=g)[:n].sort().values.to(torch.int32)
            s["tokens"] = s["tokens"][s["index"].long()].contiguous()
        return s
    # an estimate of the likelihood bound weighs a masked token by 1 / t, t ~ U(0.2, 1) for each sequence of 32 rows
    s["weights"] = 1.0 / (0.2 + 0.8 * torch.rand(rows // 32 + 1, device="cuda", generator=g)).repeat_interleave(32)[:rows]
    if case.get("skip"):
        s["weights"][case["skip"] - 1::case["skip"]] = 0.0
    if case["op"].startswith("policy"):
        s["old"], s["ref"] = lp + normal(rows, 0.2), lp + normal(rows, 0.3)
        s["advantages"] = normal(rows // 32 + 1, 1.0).repeat_interleave(32)[:rows].contiguous()
        s["upstream"] = normal(rows, 1.0)
    elif case["op"].startswith("preference"):
        s["ref"] = None if case["free"] else lp + normal(rows, 0.3)
        # ragged sequences, chosen and rejected in turn; answers of one length on average
        ends = torch.cumsum(0.25 + torch.rand(2 * case["pairs"], device="cuda", generator=g), 0)
        s["offsets"] = torch.cat([torch.zeros(1, device="cuda"), ends / ends[-1] * rows]).round().to(torch.int32)
        s["margins"] = torch.rand(case["pairs"], device="cuda", generator=g) * 0.5
        s["pair_weights"] = 0.5 + torch.rand(case["pairs"], device="cuda", generator=g)
        s["upstream"] = normal(case["pairs"], 1.0)
        if case["free"]:  # without a reference the sequences' scores are means
            n = (s["offsets"][1:] - s["offsets"][:-1]).clamp(min=1)
            s["weights"] /= n[_sequence(s["offsets"], rows)]
    return s


def _sequence(offsets, rows):
    """The sequence that each row belongs to."""
    at = torch.arange(rows, device="cuda", dtype=torch.int32)
    return (offsets[None, 1:] <= at[:, None]).sum(1).clamp(max=len(offsets) - 2)


_BETA = 0.1
_CLIP = (0.2, 0.28)


def _plain_rows(z, token, temperature):
    """Weights relative to the maximum, their sum in 64 bits, and the token's log-probability."""
    y = z.float() / temperature
    m = y.amax(1, keepdim=True)
    e = torch.exp(y - m)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    lse = m.double() + total.log()
    return e, total, (y.gather(1, token[:, None]).double() - lse)[:, 0], lse[:, 0]


def _plain_grad(e, total, token, slope, temperature, dtype):
    """slope / T ([v = token] - q_v); 1 - q of the token itself from the other weights."""
    q = e / total.float()
    away = ((total - e.gather(1, token[:, None])) / total).float()
    k = (slope / temperature).float()[:, None]
    grad = (-k * q).scatter_(1, token[:, None], k * away)
    return torch.where(k != 0, grad, 0.0).to(dtype)


def _plain_policy(s, lp):
    """(loss, d loss / d log-probability) of each row, weights apart."""
    rho = torch.exp(lp - s["old"].double())
    a = s["advantages"].double()
    free, cut = rho * a, rho.clamp(1 - _CLIP[0], 1 + _CLIP[1]) * a
    gain, slope = torch.minimum(free, cut), torch.where(free <= cut, free, 0.0)
    if s["dual"]:
        floor = (a < 0) & (gain < s["dual"] * a)
        gain, slope = torch.where(floor, s["dual"] * a, gain), torch.where(floor, 0.0, slope)
    y = s["ref"].double() - lp
    kl, kl_slope = {"k1": (-y, torch.ones_like(y)), "k2": (y * y / 2, -y), "k3": (torch.expm1(y) - y, -torch.expm1(y))}[s["kl"]]
    return s["kl_weight"] * kl - gain, s["kl_weight"] * kl_slope - slope


def _plain_preference(s, lp):
    """Loss of each pair, score of each sequence; a row's slope is its pair's (third) times its sign and weight (fifth)."""
    rows, pairs = s["rows"], s["pairs"]
    seq = _sequence(s["offsets"], rows)
    term = s["weights"].double() * (lp if s["free"] else lp - s["ref"].double())
    score = torch.zeros(2 * pairs, dtype=torch.float64, device="cuda").index_add_(0, seq, term)
    h = _BETA * (score[0::2] - score[1::2]) - s["margins"].double()
    if s["kind"] == "sigmoid":
        eps, soft = s["smooth"], lambda v: torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)
        loss = (1 - eps) * soft(-h) + eps * soft(h)
        slope = eps / (1 + torch.exp(-h)) - (1 - eps) / (1 + torch.exp(h))
    elif s["kind"] == "hinge":
        loss, slope = (1 - h).clamp(min=0), -(h < 1).double()
    else:
        loss, slope = ((h - 0.5) / _BETA) ** 2, 2 * (h - 0.5) / _BETA ** 2
    per_pair = s["pair_weights"].double() * slope * _BETA
    sign = 1.0 - 2.0 * (seq % 2)
    return s["pair_weights"].double() * loss, score, per_pair, seq // 2, sign * s["weights"].double()


def _plain(s):
    token, t, dtype = s["tokens"].long(), s["temperature"], s["logits"].dtype
    z = s["logits"][s["index"].long()] if s.get("subset") else s["logits"]
    e, total, lp, lse = _plain_rows(z, token, t)
    if s["op"] == "logprob":
        return {"logp": lp.float(), "lse": lse.float()}
    w = s["weights"].double()
    if s["op"] == "logprob_step":
        return {"logp": torch.where(w != 0, lp, 0.0).float(), "grad": _plain_grad(e, total, token, w, t, dtype)}
    if s["op"].startswith("policy"):
        loss, slope = _plain_policy(s, lp)
        out = {"loss": (w * loss).float(), "logp": torch.where(w != 0, lp, 0.0).float()}
        if s["op"] != "policy_loss":
            up = s["upstream"].double() if s["op"] == "policy_train" else 1.0
            out["grad"] = _plain_grad(e, total, token, up * w * slope, t, dtype)
        return out
    loss, score, per_pair, pair, sign = _plain_preference(s, lp)
    if s["op"] == "preference_train":
        per_pair = per_pair * s["upstream"].double()
    return {"loss": loss.float(), "score": score.float(), "logp": lp.float(),
            "grad": _plain_grad(e, total, token, per_pair[pair] * sign, t, dtype)}


def _own(s):
    import diffusion_decoding_token_gb300 as dlm
    z, token, t = s["logits"], s["tokens"], s["temperature"]
    if s["op"] == "logprob":
        r = dlm.row_logprob(z, token, temperature=t, row_index=s.get("index"), gather=s["subset"])
        return {"logp": r.logp, "lse": r.lse}
    if s["op"] == "logprob_step":
        logp, grad = dlm.row_logprob_step(z, token, s["weights"], temperature=t)
        return {"logp": logp, "grad": grad}
    if s["op"].startswith("policy"):
        given = dict(old=s["old"], ref=s["ref"], clip_low=_CLIP[0], clip_high=_CLIP[1], dual_clip=s["dual"],
                     kl_weight=s["kl_weight"], kl=s["kl"], temperature=t, weights=s["weights"])
        if s["op"] == "policy_step":
            r = dlm.policy_step(z, token, s["advantages"], **given)
            return {"loss": r.loss, "logp": r.logp, "grad": r.grad}
        r = dlm.policy_loss(z, token, s["advantages"], **given)
        if s["op"] == "policy_loss":
            return {"loss": r.loss, "logp": r.logp}
        return {"loss": r.loss, "logp": r.logp, "grad": dlm.policy_grad(z, token, r.state, s["upstream"], temperature=t)}
    given = dict(ref=s["ref"], beta=_BETA, kind=s["kind"], label_smoothing=s["smooth"] if s["kind"] == "sigmoid" else 0.0,
                 margins=s["margins"], weights=s["weights"], pair_weights=s["pair_weights"], temperature=t)
    if s["op"] == "preference_step":
        r = dlm.preference_step(z, token, s["offsets"], **given)
        return {"loss": r.loss, "score": r.score, "logp": r.logp, "grad": r.grad}
    r = dlm.preference_loss(z, token, s["offsets"], **given)
    grad = dlm.preference_grad(z, token, r.state, s["upstream"], temperature=t)
    return {"loss": r.loss, "score": r.score, "logp": r.logp, "grad": grad}


def run(s):
    if own:
        return _own(s)
    return _plain(s)


def work(case):
    size = 4 if case["type"] == "f32" else 2
    rows, vocab = case["rows"], case["vocab"]
    if case.get("subset"):
        rows = (2 * rows + 2) // 3
    cells = rows * vocab
    if case["op"] == "logprob":  # the maximum, scale, exponential, add; a token in, two numbers out
        return {"bytes": cells * size + rows * (16 if case["subset"] else 12), "flops": 4 * cells}
    read = cells - (rows // case["skip"] * vocab if case.get("skip") else 0)
    if case["op"] == "policy_loss":
        return {"bytes": read * size + rows * 28, "flops": 4 * read}
    return {"bytes": read * size + cells * size + rows * 28, "flops": 6 * read}


def exact(case, seed):
    s = prepare(case, seed)
    t, op = case["temperature"], case["op"]
    index = s["index"].tolist() if case.get("subset") else range(case["rows"])
    tokens = s["tokens"].tolist()
    host = {k: v.double().tolist() for k, v in s.items() if torch.is_tensor(v) and v.dim() == 1}
    weights = host.get("weights")
    lp, lse, away = [], [], []
    # one token against all others: ln p = -ln(1 + sum of the others' odds)
    for r, row in enumerate(index):
        y = s["logits"][row].double() / t
        other = y.clone()
        other[tokens[r]] = -math.inf
        ln_others = torch.logsumexp(other, 0)
        pair = torch.stack([y[tokens[r]], ln_others])
        both = torch.logaddexp(pair[0], pair[1])
        lse.append(both)
        lp.append(-torch.nn.functional.softplus(ln_others - pair[0], threshold=700.0))
        away.append(torch.exp(ln_others - both))
    lp, lse, away = (torch.stack(v).tolist() for v in (lp, lse, away))
    pack = lambda v: torch.tensor(v, dtype=torch.float64)  # noqa: E731
    if op == "logprob":
        return {"logp": pack(lp), "lse": pack(lse)}
    masked = [w != 0 for w in weights]
    out, slope = {"logp": pack([x if m else 0.0 for x, m in zip(lp, masked)])}, []
    if op == "logprob_step":
        slope = list(weights)
    elif op.startswith("policy"):
        loss = []
        for r, w in enumerate(weights):
            one, d = _exact_policy(lp[r] - host["old"][r], host["ref"][r] - lp[r], host["advantages"][r], case)
            loss.append(w * one)
            slope.append(w * d * (host["upstream"][r] if op == "policy_train" else 1.0))
        out["loss"] = pack(loss)
    else:
        slope = [0.0] * case["rows"]
        out["loss"], out["score"] = [], []
        at = s["offsets"].tolist()
        for i in range(case["pairs"]):
            won, lost = (range(at[j], at[j + 1]) for j in (2 * i, 2 * i + 1))
            score = [math.fsum(weights[r] * (lp[r] - (0.0 if case["free"] else host["ref"][r])) for r in q) for q in (won, lost)]
            one, d = _exact_pair(_BETA * (score[0] - score[1]) - host["margins"][i], case)
            out["loss"].append(host["pair_weights"][i] * one)
            out["score"] += score
            d *= host["pair_weights"][i] * _BETA * (host["upstream"][i] if op == "preference_train" else 1.0)
            for q, sign in ((won, 1.0), (lost, -1.0)):
                for r in q:
                    slope[r] = sign * d * weights[r]
        out["loss"], out["score"] = pack(out["loss"]), pack(out["score"])
    if op != "policy_loss":
        grad = torch.zeros((case["rows"], case["vocab"]), dtype=torch.float64, device="cuda")
        for r, d in enumerate(slope):
            if d != 0:
                grad[r] = torch.exp(s["logits"][r].double() / t - lse[r]) * (-d / t)
                grad[r, tokens[r]] = d / t * away[r]
        out["grad"] = grad
    return out


def _exact_policy(x, y, a, case):
    rho = math.exp(x)
    lo, hi = 1 - _CLIP[0], 1 + _CLIP[1]
    if (a >= 0 and rho > hi) or (a < 0 and rho < lo):  # clipped, and no better for it
        gain, slope = (hi if a >= 0 else lo) * a, 0.0
    elif a < 0 and case["dual"] and rho > case["dual"]:
        gain, slope = case["dual"] * a, 0.0
    else:
        gain = slope = rho * a
    kl, d = {"k1": (-y, 1.0), "k2": (y * y / 2, -y), "k3": (math.expm1(y) - y, -math.expm1(y))}[case["kl"]]
    return case["kl_weight"] * kl - gain, case["kl_weight"] * d - slope


def _exact_pair(h, case):
    if case["kind"] == "sigmoid":
        eps, p = case["smooth"], 1 / (1 + math.exp(-h)) if h > 0 else math.exp(h) / (1 + math.exp(h))
        down = math.log1p(math.exp(-abs(h)))
        return (1 - eps) * (down + max(-h, 0.0)) + eps * (down + max(h, 0.0)), p - (1 - eps)
    if case["kind"] == "hinge":
        return max(0.0, 1 - h), -1.0 if h < 1 else 0.0
    return ((h - 0.5) / _BETA) ** 2, 2 * (h - 0.5) / _BETA ** 2
