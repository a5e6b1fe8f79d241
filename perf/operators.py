"""What the output head's operators are measured on: cases, their inputs, and their plain forms.

Three operators take a hidden state to a token id: ``head_norm`` (residual addition, root-mean-square
norm, 8-bit output with a scale per 128 columns), ``head_logits`` (8-bit matrix product with block
scales) and ``head_sample`` (the draw of ids).  ``run`` computes them in elementary torch operations,
or, where ``own`` is true, by the package's kernels.
"""
import math

import torch

own = False

BLOCK = 128          # columns (and vocabulary rows) that share a scale
E4M3_MAX = 448.0
TINY = 2.0 ** -126   # smallest scale and smallest temperature that is not greedy
ONE = 2.0 ** 40      # the weight of a row's largest logit in the draw

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token of one request: latency
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "dim": 4096, "type": "bf16", "residual": True},
        # odd width and rows, 32-bit activations, no residual stream
        {"name": "norm 777x1000 f32", "op": "norm", "rows": 777, "dim": 1000, "type": "f32", "residual": False},
        # scoring a long text: every position goes through the head
        {"name": "norm 8192x4096", "op": "norm", "rows": 8192, "dim": 4096, "type": "bf16", "residual": True},
        # one token of one request over the 32,256-token vocabulary of the large corpus
        {"name": "logits 1x32256x4096", "op": "logits", "rows": 1, "tokens": 32256, "dim": 4096, "type": "f32"},
        # a decoding batch over the largest vocabulary that merges can make
        {"name": "logits 64x65536x4096", "op": "logits", "rows": 64, "tokens": 65536, "dim": 4096, "type": "f32"},
        # a ragged batch over the substring vocabulary, a width that ends inside a block
        {"name": "logits 333x250000x1040", "op": "logits", "rows": 333, "tokens": 250000, "dim": 1040, "type": "bf16"},
        # scoring: the largest product
        {"name": "logits 4096x32256x4096", "op": "logits", "rows": 4096, "tokens": 32256, "dim": 4096, "type": "bf16"},
        # one request's next token
        {"name": "sample 1x32256", "op": "sample", "rows": 1, "tokens": 32256, "type": "f32", "filters": "top_p", "shape": "peaked"},
        # a decoding batch with every filter, each row with its own settings
        {"name": "sample 256x65536", "op": "sample", "rows": 256, "tokens": 65536, "type": "bf16", "filters": "all", "shape": "peaked"},
        # the substring vocabulary, flat rows: nuclei of many thousand tokens
        {"name": "sample 61x250000 flat", "op": "sample", "rows": 61, "tokens": 250000, "type": "f32", "filters": "top_p", "shape": "flat"},
        # many drafts over a small vocabulary, temperature alone
        {"name": "sample 4096x4352", "op": "sample", "rows": 4096, "tokens": 4352, "type": "bf16", "filters": "none", "shape": "peaked"},
        # a batch with top-k alone
        {"name": "sample 33x32256 top-k", "op": "sample", "rows": 33, "tokens": 32256, "type": "f16", "filters": "top_k", "shape": "flat"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "logits", "sample"])
    kind = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 8192), "dim": _log(rng, 200, 8000), "type": kind,
                "residual": rng.random() < 0.7}
    if op == "logits":
        dim = _log(rng, 256, 8000)
        if rng.random() < 0.75:
            dim = dim // 16 * 16
        rows, tokens = _log(rng, 1, 4096), _log(rng, 512, 250000)
        rows = max(1, min(rows, 4096 * 32256 * 4096 // (tokens * dim), 4096 * 32256 // tokens))
        return {"op": op, "rows": rows, "tokens": tokens, "dim": dim, "type": kind}
    tokens = _log(rng, 512, 250000)
    rows = max(1, min(_log(rng, 1, 4096), 24_000_000 // tokens))
    return {"op": op, "rows": rows, "tokens": tokens, "type": kind,
            "filters": rng.choice(["none", "top_k", "top_p", "min_p", "all"]), "shape": rng.choice(["peaked", "flat"])}


def work(case):
    m = case["rows"]
    if case["op"] == "norm":
        k, e = case["dim"], SIZE[case["type"]]
        stream = 3 if case["residual"] else 1
        return {"bytes": m * k * (stream * e + 1) + k * e + 4 * m * -(-k // BLOCK), "flops": 8 * m * k}
    n = case["tokens"]
    if case["op"] == "logits":
        k, kb = case["dim"], -(-case["dim"] // BLOCK)
        return {"bytes": (m + n) * k + 4 * kb * (m + -(-n // BLOCK)) + m * n * SIZE[case["type"]], "flops": 2 * m * n * k}
    return {"bytes": m * n * SIZE[case["type"]] + 28 * m, "flops": 4 * m * n}


# ----------------------------------------------------------------- inputs ---

def _blocks_of_rows(w):
    """An [N, K] matrix as e4m3 with one scale per 128 x 128 block, as a checkpoint stores it."""
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    full = torch.zeros(nb * BLOCK, kb * BLOCK, device=w.device)
    full[:n, :k] = w
    t = full.view(nb, BLOCK, kb, BLOCK)
    scale = (t.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(TINY)
    q = (t / scale[:, None, :, None]).reshape(nb * BLOCK, kb * BLOCK)[:n, :k].contiguous()
    return q.to(torch.float8_e4m3fn), scale


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    m, kind = case["rows"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        k = case["dim"]
        # a few columns of a trained residual stream are far larger than the rest
        loud = 1 + 20 * (torch.rand(k, generator=g, device="cuda") < 0.01)
        return {"x": normal(m, k).to(kind), "weight": (1 + 0.2 * normal(k)).to(kind),
                "residual": (3 * normal(m, k) * loud).to(kind) if case["residual"] else None}
    if case["op"] == "logits":
        n, k = case["tokens"], case["dim"]
        kb = -(-k // BLOCK)
        x = torch.zeros(m, kb * BLOCK, device="cuda")
        x[:, :k] = normal(m, k)
        t = x.view(m, kb, BLOCK)
        xs = (t.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
        wide = -(-k // 16) * 16  # rows of activations start on 16 bytes, as head_norm lays them out
        x8 = torch.zeros(m, wide, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
        x8.view(torch.uint8)[:, :k] = (t / xs[..., None]).reshape(m, -1)[:, :k].to(torch.float8_e4m3fn).view(torch.uint8)
        rows = torch.exp(0.3 * normal(n, 1)) / math.sqrt(k)  # rare tokens have smaller rows
        w8, ws = _blocks_of_rows(normal(n, k).mul_(rows))
        return {"x8": x8[:, :k], "xs": xs.t().contiguous().t(), "w8": w8, "ws": ws}
    n = case["tokens"]
    spread = 1.2 if case["shape"] == "flat" else 2.5
    logits = spread * normal(m, n)
    if case["shape"] == "peaked":  # a few tokens that the context makes likely
        at = (torch.randint(0, n, (m, 1), generator=g, device="cuda") + torch.arange(40, device="cuda") * (n // 41)) % n
        logits.scatter_(1, at, 8 + 3 * normal(m, 40))
    rand = torch.rand(m, 5, generator=g, device="cuda")
    f = case["filters"]
    return {"logits": logits.to(kind), "u": rand[:, 0].contiguous(),
            "temperature": 0.6 + 0.6 * rand[:, 1],
            "top_k": (20 + 180 * rand[:, 2]).to(torch.int32) if f in ("top_k", "all") else None,
            "top_p": 0.8 + 0.18 * rand[:, 3] if f in ("top_p", "all") else None,
            "min_p": 0.02 + 0.08 * rand[:, 4] if f in ("min_p", "all") else None}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"], s["type"] = case["op"], case["type"]
    m = case["rows"]
    # the buffers that a serving loop keeps for the results
    if case["op"] == "norm":
        k = case["dim"]
        s["y8"] = torch.zeros(m, -(-k // 16) * 16, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :k]
        s["scales"] = torch.empty(-(-k // BLOCK), m, device="cuda").t()
        s["stream"] = torch.empty_like(s["x"]) if case["residual"] else None
    elif case["op"] == "logits":
        s["out"] = torch.empty(m, case["tokens"], device="cuda", dtype=TYPES[case["type"]])
    else:
        s["ids"] = torch.empty(m, device="cuda", dtype=torch.int32)
        s["logprob"] = torch.empty(m, device="cuda")
    return s


# -------------------------------------------------------------- the plain ---

def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    m, k = x.shape
    y = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + 1e-6) * s["weight"].float()
    kb = -(-k // BLOCK)
    full = torch.zeros(m, kb * BLOCK, device=x.device)
    full[:, :k] = y
    t = full.view(m, kb, BLOCK)
    scale = (t.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
    q = (t / scale[..., None]).reshape(m, kb * BLOCK)[:, :k].to(torch.float8_e4m3fn)
    return [q, scale] + ([x.to(s["x"].dtype)] if s["residual"] is not None else [])


def _plain_logits(s):
    m, k = s["x8"].shape
    n = s["w8"].shape[0]
    x = s["x8"].float() * s["xs"][:, torch.arange(k, device="cuda") // BLOCK]
    i = torch.arange(n, device="cuda") // BLOCK
    w = s["w8"].float() * s["ws"][i][:, torch.arange(k, device="cuda") // BLOCK]
    return (x @ w.t()).to(TYPES[s["type"]])


def _weights(s):
    """(logits, z, integer weights of the draw) of every row."""
    v = s["logits"].float()
    v = torch.where(torch.isnan(v), float("-inf"), v)
    top = v.amax(dim=1, keepdim=True)
    z = torch.where(v == top, 0.0, (v - top) * (1.0 / s["temperature"])[:, None])
    return v, z, (torch.exp(z) * ONE).to(torch.int64)


def _plain_sample(s):
    v, z, w = _weights(s)
    m, n = v.shape
    order = torch.sort(v, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    keep = torch.ones(m, n, dtype=torch.bool, device="cuda")
    if s["top_k"] is not None:
        keep &= torch.arange(n, device="cuda")[None] < s["top_k"][:, None]
    if s["top_p"] is not None:
        mass = torch.where(keep, ws, 0)
        before = torch.cumsum(mass, dim=1) - mass
        edge = (s["top_p"].double() * mass.sum(dim=1).double()).to(torch.int64)
        keep &= before < edge[:, None].clamp_min(1)
    if s["min_p"] is not None:
        keep &= ws >= (s["min_p"].clamp(max=1.0) * ONE).to(torch.int64)[:, None]
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    run_mass = torch.cumsum(torch.where(kept, w, 0), dim=1)
    total = run_mass[:, -1]
    t = torch.minimum((s["u"].double() * total.double()).to(torch.int64), total - 1)
    ids = (run_mass <= t[:, None]).sum(dim=1)
    logprob = z.gather(1, ids[:, None])[:, 0] - torch.log(total.float() * 2.0 ** -40)
    return [ids.to(torch.int32), logprob]


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
        return {"norm": _plain_norm, "logits": _plain_logits, "sample": _plain_sample}[s["op"]](s)
    ctx = _own()
    if s["op"] == "norm":
        q, scale, stream = ctx.head_norm(s["x"], s["weight"], s["residual"], eps=1e-6, out=s["y8"], scales=s["scales"],
                                         residual_out=s["stream"])
        return [q, scale] + ([stream] if s["residual"] is not None else [])
    if s["op"] == "logits":
        return ctx.head_logits(s["x8"], s["xs"], s["w8"], s["ws"], out=s["out"])
    ids, logprob = ctx.head_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                   top_p=s["top_p"], min_p=s["min_p"], ids=s["ids"], logprob=s["logprob"])
    return [ids, logprob]


# -------------------------------------------------------------- in 64 bits ---

def _exact_norm(s):
    x = s["x"].double()
    if s["residual"] is not None:
        x = x + s["residual"].double()
    m, k = x.shape
    y = x / (x.square().sum(1, keepdim=True) / k + 1e-6).sqrt() * s["weight"].double()
    scale = torch.stack([b.abs().amax(1) for b in y.split(BLOCK, dim=1)], dim=1) / E4M3_MAX
    scale = scale.clamp_min(TINY)
    # the values that the 8 bits stand for, before they are rounded
    q = torch.cat([b / scale[:, i:i + 1] for i, b in enumerate(y.split(BLOCK, dim=1))], dim=1)
    return [q, scale] + ([x] if s["residual"] is not None else [])


def _exact_logits(s):
    """Sums without rounding: an e4m3 value is hi + lo / 512 with |hi| <= 448 and |lo| <= 256 whole numbers, so that 32-bit
    products over 64 columns are whole numbers below 2^24; the blocks are then scaled and added in 64 bits."""
    m, k = s["x8"].shape
    n = s["w8"].shape[0]
    x, w = s["x8"].float(), s["w8"].float()
    xh, wh = x.round(), w.round()
    xl, wl = (x - xh) * 512, (w - wh) * 512
    out = torch.zeros(m, n, device="cuda", dtype=torch.float64)
    for c in range(0, k, 64):
        e = min(k, c + 64)
        a, b, p, q = xh[:, c:e], xl[:, c:e], wh[:, c:e].t(), wl[:, c:e].t()
        left = s["xs"][:, c // BLOCK].double()[:, None]
        right = s["ws"][:, c // BLOCK].double().repeat_interleave(BLOCK)[:n]
        part = (a @ q).double().add_(b @ p)
        part.mul_(2.0 ** -9).add_(a @ p)
        part.add_(b @ q, alpha=2.0 ** -18)
        out.addcmul_(part.mul_(left), right[None])
    return out


def _exact_sample(s):
    """The draw is over whole numbers that come from 32-bit exponentials by definition; the log-probability of the drawn id
    is in 64 bits.  Row by row, on lists of (value, index)."""
    v = s["logits"].float()
    inverse = torch.ones_like(s["temperature"]) / s["temperature"]
    ids, logprob = [], []
    for r in range(v.shape[0]):
        mass = torch.ldexp(torch.exp((v[r] - v[r].max()) * inverse[r]), torch.tensor(40, device="cuda")).long()
        at = torch.nonzero(mass)[:, 0]  # what has no weight is never drawn
        at = at[torch.argsort(v[r][at], descending=True, stable=True)]
        mass = mass[at]
        if s["top_k"] is not None:
            mass = mass[:int(s["top_k"][r])]
        if s["top_p"] is not None:
            edge = int(float(s["top_p"][r]) * float(int(mass.sum())))
            mass = mass[:max(1, int((mass.cumsum(0) - mass < edge).sum()))]
        if s["min_p"] is not None:
            mass = mass[mass >= int(float(s["min_p"][r]) * ONE)]
        at, back = at[:mass.numel()].sort()
        run_mass = mass[back].cumsum(0)
        total = int(run_mass[-1])
        t = min(int(float(s["u"][r]) * float(total)), total - 1)
        one = at[int(torch.searchsorted(run_mass, t, right=True))]
        x = (v[r].double() - v[r].double().amax()) / s["temperature"][r].double()
        ids.append(one)
        logprob.append(x[one] - torch.logsumexp(x[at], 0))
    return [torch.stack(ids).to(torch.int32), torch.stack(logprob)]


def exact(case, seed):
    s = _inputs(case, seed)
    return {"norm": _exact_norm, "logits": _exact_logits, "sample": _exact_sample}[case["op"]](s)
