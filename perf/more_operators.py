"""What the output head's scoring and training operators are measured on: cases, their inputs, and their plain forms.

``head_logprobs`` gives the log-probabilities of given ids, the entropy and the top alternatives of rows of logits,
``head_logprobs_backward`` the gradient of the first two; ``head_distill`` gives the divergence of rows of logits from a
teacher's top alternatives and, in the same call, its gradient.  ``run`` computes them in elementary torch operations, or,
where ``own`` is true, by the package's kernels.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
INF = float("inf")


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token of one request, with the alternatives that an answer lists: latency
        {"name": "logprobs 1x32256 top 20", "op": "logprobs", "rows": 1, "tokens": 32256, "type": "f32", "top": 20,
         "tempered": False, "padded": False},
        # a decoding batch over the largest vocabulary that merges can make, each row at its own temperature
        {"name": "logprobs 256x65536 top 20", "op": "logprobs", "rows": 256, "tokens": 65536, "type": "bf16", "top": 20,
         "tempered": True, "padded": False},
        # scoring a long text: every position, its own token alone
        {"name": "logprobs 8192x32256", "op": "logprobs", "rows": 8192, "tokens": 32256, "type": "bf16", "top": 0,
         "tempered": False, "padded": False},
        # a teacher's answers over the substring vocabulary, kept for distillation
        {"name": "logprobs 333x250000 top 64", "op": "logprobs", "rows": 333, "tokens": 250000, "type": "f16", "top": 64,
         "tempered": False, "padded": False},
        # odd sizes in 32 bits: rows that start anywhere, the entropy's gradient too
        {"name": "logprobs_grad 777x4351 f32 entropy", "op": "logprobs_grad", "rows": 777, "tokens": 4351, "type": "f32",
         "entropy": True, "tempered": True, "padded": False},
        # the loss of a training step: cross entropy over a vocabulary padded to a multiple of 128
        {"name": "logprobs_grad 8192x32156", "op": "logprobs_grad", "rows": 8192, "tokens": 32156, "type": "bf16",
         "entropy": False, "tempered": False, "padded": True},
        # a small evaluation batch
        {"name": "distill 16x4352 f32 8", "op": "distill", "rows": 16, "tokens": 4352, "type": "f32", "listed": 8,
         "rest": False, "tempered": False, "padded": False},
        # evaluation over the substring vocabulary, the unlisted tokens as one class
        {"name": "distill 900x250000 100 rest", "op": "distill", "rows": 900, "tokens": 250000, "type": "bf16", "listed": 100,
         "rest": True, "tempered": False, "padded": False},
        # a small training step with odd sizes in 32 bits
        {"name": "distill_grad 61x65535 f32 33 rest", "op": "distill_grad", "rows": 61, "tokens": 65535, "type": "f32",
         "listed": 33, "rest": True, "tempered": False, "padded": False},
        # the training step: loss and gradient of every position
        {"name": "distill_grad 8192x32256 64", "op": "distill_grad", "rows": 8192, "tokens": 32256, "type": "bf16",
         "listed": 64, "rest": False, "tempered": True, "padded": False},
        # the same over the substring vocabulary, in 16-bit floats
        {"name": "distill_grad 400x250000 f16 128 rest", "op": "distill_grad", "rows": 400, "tokens": 250000, "type": "f16",
         "listed": 128, "rest": True, "tempered": False, "padded": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "distill", "distill_grad"])
    tokens = _log(rng, 260, 250000)
    rows = max(1, min(_log(rng, 1, 8192), 8192 * 32156 // tokens))
    kind = rng.choice(["f32", "bf16", "bf16", "f16"])
    if kind == "f32":
        rows = (rows + 1) // 2
    case = {"op": op, "rows": rows, "tokens": tokens, "type": kind, "tempered": rng.random() < 0.5,
            "padded": rng.random() < 0.3}
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 20, rng.randint(2, 128)])
    elif op == "logprobs_grad":
        case["entropy"] = rng.random() < 0.5
    else:
        case["listed"] = _log(rng, 1, 128)
        case["rest"] = rng.random() < 0.5
    return case


def work(case):
    m, n, e = case["rows"], case["tokens"], SIZE[case["type"]]
    if case["op"] == "logprobs":   # the row once; id in, log-probability, entropy and norm out, the alternatives
        return {"bytes": m * n * e + m * (20 + 8 * case["top"]), "flops": 5 * m * n}
    if case["op"] == "logprobs_grad":
        return {"bytes": 2 * m * n * e + m * 24, "flops": (8 if case["entropy"] else 4) * m * n}
    if case["op"] == "distill":
        return {"bytes": m * n * e + m * (4 + 8 * case["listed"]), "flops": 4 * m * n}
    return {"bytes": 2 * m * n * e + m * (8 + 8 * case["listed"]), "flops": 8 * m * n}


# ----------------------------------------------------------------- inputs ---

def _rows_of(case, normal, rand, whole):
    """Logits [rows, tokens]: flat with a few tokens that the context makes likely; a view of wider rows where padded."""
    m, n = case["rows"], case["tokens"]
    wide = -(-n // 128) * 128 + 128 if case["padded"] else n
    logits = 2.0 * normal(m, n)
    likely = min(n // 6, 120)
    at = (whole(n, m, 1) + torch.arange(likely, device="cuda") * (n // (likely + 1))) % n
    logits.scatter_(1, at, 7 + 3 * normal(m, likely))
    full = torch.zeros(m, wide, device="cuda", dtype=TYPES[case["type"]])
    full[:, :n] = logits
    return full[:, :n], at


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    m, n = case["rows"], case["tokens"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def whole(most, *shape):
        return torch.randint(0, most, shape, generator=g, device="cuda")

    logits, at = _rows_of(case, normal, rand, whole)
    s = {"op": case["op"], "logits": logits, "temperature": 0.6 + 0.9 * rand(m) if case["tempered"] else 1.0}
    scale = 1024.0 if case["type"] == "f16" else 1.0   # losses of 16-bit floats are scaled
    if case["op"] in ("logprobs", "logprobs_grad"):
        ids = at.gather(1, whole(at.shape[1], m, 1))[:, 0]
        ids = torch.where(rand(m) < 0.2, whole(n, m), ids)
        s["ids"] = torch.where(rand(m) < 0.05, -1, ids).to(torch.int32)   # rows that pad a batch have none
    if case["op"] == "logprobs":
        s["top"] = case["top"]
    elif case["op"] == "logprobs_grad":
        s["grad_logprob"] = -scale / m * (0.5 + rand(m))
        s["grad_entropy"] = -0.01 * scale / m * (0.5 + rand(m)) if case["entropy"] else None
    else:
        # a teacher that agrees with the student but for noise; rows with fewer alternatives end in ids of -1
        k, rest = case["listed"], case["rest"]
        ids = torch.empty(m, k, device="cuda", dtype=torch.int32)
        values = torch.empty(m, k, device="cuda")
        for r in range(0, m, 512):
            t = logits[r:r + 512].float()
            t = t + 0.8 * normal(*t.shape)
            top = t.topk(k, dim=1)
            ids[r:r + 512] = top.indices.to(torch.int32)
            values[r:r + 512] = top.values - torch.logsumexp(t, 1, keepdim=True)
        count = torch.where(rand(m, 1) < 0.1, 1 + (rand(m, 1) * k).long(), k)
        s["top_ids"] = torch.where(torch.arange(k, device="cuda") < count, ids, -1)
        s["top_logprob"], s["rest"] = values, rest
        s["grad"] = scale / m * (0.5 + rand(m)) if case["op"] == "distill_grad" else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    m, op = case["rows"], case["op"]
    # the buffers that a loop keeps for the results
    if op == "logprobs":
        s["out"] = {"logprob": torch.empty(m, device="cuda"), "entropy": torch.empty(m, device="cuda"),
                    "norm": torch.empty(m, 2, device="cuda")}
        if s["top"]:
            s["out"]["top_ids"] = torch.empty(m, s["top"], device="cuda", dtype=torch.int32)
            s["out"]["top_logprob"] = torch.empty(m, s["top"], device="cuda")
        return s
    if op == "logprobs_grad":
        # what head_logprobs gave in the step's forward pass
        s["norm"], s["entropy"] = torch.empty(m, 2, device="cuda"), torch.empty(m, device="cuda")
        for r in range(0, m, 1024):
            some = slice(r, r + 1024)
            v = s["logits"][some].double()
            t = s["temperature"][some].double()[:, None] if case["tempered"] else 1.0
            top = v.amax(1, keepdim=True)
            z = (v - top) / t
            lse = z.exp().sum(1).log()
            s["norm"][some, 0], s["norm"][some, 1] = top[:, 0].float(), lse.float()
            s["entropy"][some] = (lse - (z * (z - lse[:, None]).exp()).sum(1)).float()
    if op == "distill":
        s["loss"] = torch.empty(m, device="cuda")
    else:
        s["out"] = torch.empty_strided(s["logits"].shape, s["logits"].stride(), dtype=s["logits"].dtype, device="cuda")
        if op == "distill_grad":
            s["loss"] = torch.empty(m, device="cuda")
    return s


# -------------------------------------------------------------- the plain ---

def _column(v):
    return v[:, None] if isinstance(v, torch.Tensor) else v


def _softmax(s):
    """(largest logit, z, log of the sum of exp(z)) of every row."""
    v = s["logits"].float()
    top = v.amax(dim=1, keepdim=True)
    z = (v - top) / _column(s["temperature"])
    return v, top, z, torch.exp(z).sum(dim=1, keepdim=True).log()


def _plain_logprobs(s):
    v, top, z, lse = _softmax(s)
    z -= lse
    ids = s["ids"].long()
    given = z.gather(1, ids.clamp_min(0)[:, None])[:, 0]
    logprob = torch.where(ids < 0, 0.0, given)
    entropy = -(torch.exp(z) * z).sum(dim=1)
    out = [logprob, entropy, torch.cat([top, lse], dim=1)]
    if s["top"]:
        order = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :s["top"]]
        out += [order.to(torch.int32), z.gather(1, order)]
    return out


def _plain_logprobs_grad(s):
    v, t = s["logits"].float(), _column(s["temperature"])
    lp = (v - s["norm"][:, :1]) / t - s["norm"][:, 1:]
    p = torch.exp(lp)
    ids = s["ids"].long()
    some = torch.where(ids < 0, 0.0, s["grad_logprob"])[:, None]
    d = -some * p
    d.scatter_add_(1, ids.clamp_min(0)[:, None], some)
    if s["grad_entropy"] is not None:
        d -= s["grad_entropy"][:, None] * p * (lp + s["entropy"][:, None])
    return (d / t).to(s["logits"].dtype)


def _plain_distill(s):
    _, _, z, lse = _softmax(s)
    z -= lse
    ids = s["top_ids"].long()
    given = ids >= 0
    ids = ids.clamp_min(0)
    t = torch.where(given, s["top_logprob"], -INF)
    if not s["rest"]:
        t = t - t.amax(dim=1, keepdim=True)
        t = t - torch.exp(t).sum(dim=1, keepdim=True).log()
    q = torch.exp(t)
    term = q * (t - z.gather(1, ids))
    loss = torch.where(q > 0, term, 0.0).sum(dim=1)
    factor = q.sum(dim=1)
    if s["rest"]:
        # the mass of the unlisted tokens is summed over them; ids of -1 mark a place beyond the last
        n = z.shape[1]
        left = torch.ones(z.shape[0], n + 1, dtype=torch.bool, device=z.device)
        left.scatter_(1, torch.where(given, ids, n), False)
        left = left[:, :n]
        q_rest = (1.0 - factor).clamp_min(0.0)
        p_rest = torch.where(left, torch.exp(z), 0.0).sum(dim=1)
        loss = loss + torch.where(q_rest > 0, q_rest * (torch.log(q_rest) - torch.log(p_rest)), 0.0)
        factor = factor + q_rest
    if s["grad"] is None:
        return loss
    d = torch.exp(z)
    if s["rest"]:
        d *= torch.where(left, (factor - q_rest / p_rest)[:, None], factor[:, None])
    else:
        d *= factor[:, None]
    d.scatter_add_(1, ids, -q)
    d *= s["grad"][:, None]
    return [loss, (d / _column(s["temperature"])).to(s["logits"].dtype)]


_context = None


def _own():
    global _context
    if _context is None:
        import bpe_trie_encode_gb300
        _context = bpe_trie_encode_gb300.Context()
    return _context


def run(state):
    s = state
    if not own:
        return {"logprobs": _plain_logprobs, "logprobs_grad": _plain_logprobs_grad, "distill": _plain_distill,
                "distill_grad": _plain_distill}[s["op"]](s)
    ctx = _own()
    if s["op"] == "logprobs":
        logprob, entropy, top_ids, top_logprob, norm = ctx.head_logprobs(
            s["logits"], s["ids"], temperature=s["temperature"], top=s["top"], **s["out"])
        return [logprob, entropy, norm] + ([top_ids, top_logprob] if s["top"] else [])
    if s["op"] == "logprobs_grad":
        return ctx.head_logprobs_backward(s["logits"], s["ids"], s["norm"], s["grad_logprob"], s["entropy"],
                                          s["grad_entropy"], temperature=s["temperature"], out=s["out"])
    if s["op"] == "distill":
        return ctx.head_distill(s["logits"], s["top_ids"], s["top_logprob"], temperature=s["temperature"], rest=s["rest"],
                                loss=s["loss"])[0]
    loss, grad = ctx.head_distill(s["logits"], s["top_ids"], s["top_logprob"], temperature=s["temperature"], rest=s["rest"],
                                  grad=s["grad"], loss=s["loss"], out=s["out"])
    return [loss, grad]


# -------------------------------------------------------------- in 64 bits ---

def _part(s, some):
    """The rows `some` of a state: its tensors of rows cut to them."""
    return {k: v[some] if isinstance(v, torch.Tensor) else v for k, v in s.items()}


def _log_p(s):
    """Log-probabilities by torch.logsumexp, and what the logits were divided by."""
    x = s["logits"].double()
    t = s["temperature"]
    t = t.double().unsqueeze(1) if isinstance(t, torch.Tensor) else torch.full((x.shape[0], 1), float(t), device="cuda").double()
    y = x / t
    return y, y - torch.logsumexp(y, 1, keepdim=True), t


def _exact_logprobs(s):
    y, lp, t = _log_p(s)
    m, n = y.shape
    wanted = s["ids"].long()
    logprob = torch.zeros(m, device="cuda", dtype=torch.float64)
    has = torch.nonzero(wanted >= 0)[:, 0]
    logprob[has] = lp[has, wanted[has]]
    entropy = torch.special.entr(lp.exp()).sum(1)
    top = s["logits"].amax(1).double()
    out = [logprob, entropy, torch.stack([top, -lp.amax(1)], 1)]
    if s["top"]:
        # one whole number for each token, larger for larger logits, then for lower ids
        bits = (s["logits"].float() + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -2147483648 - bits, bits) * n + (n - 1 - torch.arange(n, device="cuda"))
        best = n - 1 - torch.topk(order, s["top"], dim=1).values.remainder(n)
        out += [best.to(torch.int32), torch.take_along_dim(lp, best, 1)]
    return out


def _exact_logprobs_grad(s):
    _, lp, t = _log_p(s)
    p = lp.exp()
    onehot = torch.zeros_like(p)
    has = torch.nonzero(s["ids"] >= 0)[:, 0]
    onehot[has, s["ids"].long()[has]] = 1
    g = onehot.sub_(p * (s["ids"] >= 0).unsqueeze(1)).mul_(s["grad_logprob"].double().unsqueeze(1))
    if s["grad_entropy"] is not None:
        entropy = torch.special.entr(p).sum(1, keepdim=True)
        g += (torch.special.entr(p) - p * entropy) * s["grad_entropy"].double().unsqueeze(1)
    return [g / t]


def _exact_distill(s):
    _, lp, t = _log_p(s)
    m, n = lp.shape
    has = s["top_ids"] >= 0
    teacher = torch.zeros_like(lp)
    q = s["top_logprob"].double().exp() * has
    if not s["rest"]:
        q = q / q.sum(1, keepdim=True)
    at = torch.nonzero(has)
    places = s["top_ids"].long()[at[:, 0], at[:, 1]]
    teacher[at[:, 0], places] = q[at[:, 0], at[:, 1]]
    loss = (torch.xlogy(teacher, teacher) - teacher * lp).sum(1)
    g = lp.exp().mul_(teacher.sum(1, keepdim=True)) - teacher
    if s["rest"]:
        listed_ = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        listed_[at[:, 0], places] = True
        q_rest = (1 - q.sum(1, keepdim=True)).clamp_min(0)
        among = lp.masked_fill(listed_, -INF)
        log_rest = torch.logsumexp(among, 1, keepdim=True)
        loss += (torch.xlogy(q_rest, q_rest) - q_rest * log_rest)[:, 0]
        g += q_rest * (lp.exp() - (among - log_rest).exp())
    if s["grad"] is None:
        return [loss]
    return [loss, g * s["grad"].double().unsqueeze(1) / t]


def exact(case, seed):
    s = _inputs(case, seed)
    how = {"logprobs": _exact_logprobs, "logprobs_grad": _exact_logprobs_grad, "distill": _exact_distill,
           "distill_grad": _exact_distill}[case["op"]]
    step = max(1, 20_000_000 // case["tokens"])
    parts = [how(_part(s, slice(r, r + step))) for r in range(0, case["rows"], step)]
    out = [torch.cat(one) for one in zip(*parts)]
    return out[0] if case["op"] in ("logprobs_grad", "distill") else out
