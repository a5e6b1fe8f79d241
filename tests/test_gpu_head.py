"""The output head on the GPU against plain implementations in 64 bits.

Tolerances come from the number formats: a 32-bit operation is off by 2^-24 of
its result, a sum of n terms by n times that of the sum of magnitudes; the
tensor cores' additions are taken as off by 2^-23 each.  An e4m3 value is half
a step (2^-4 of itself, 2^-10 below 2^-6) from what it stands for.  Ids have no
tolerance.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -126
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def ctx():
    import bpe_trie_encode_gb300 as bt
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    c = bt.Context(0)
    yield c
    c.close()


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def blocks_of(dim):
    return [(b, slice(b, min(b + 128, dim))) for b in range(0, dim, 128)]


# ------------------------------------------------------------------- norm ---

def norm_reference(x, weight, residual, eps):
    s = x.double() + (residual.double() if residual is not None else 0.0)
    y = s / (s.square().mean(1, keepdim=True) + eps).sqrt() * weight.double()
    scale = torch.stack([y[:, c].abs().amax(1) for _, c in blocks_of(x.shape[1])], 1) / 448
    return y, scale.clamp_min(TINY)


def check_norm(y8, scales, x, weight, residual, eps):
    y, scale = norm_reference(x.cpu(), weight.cpu(), residual.cpu() if residual is not None else None, eps)
    dim = x.shape[1]
    # the sum of squares in any order (dim steps), halved by the root; the root, three products, the scale's division
    rel = (dim / 2 + 10) * 2.0 ** -24
    got = scales.cpu().double()
    assert got.shape == scale.shape
    assert ((got - scale).abs() <= rel * scale).all()
    q = y8.cpu().float().double()
    for i, (_, c) in enumerate(blocks_of(dim)):
        want = y[:, c] / scale[:, i:i + 1]
        step = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
        assert ((q[:, c] - want).abs() <= step * (1 + 2 * rel) + 3 * rel * want.abs()).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 2), (1, 127), (2, 128), (5, 129), (4, 1000), (1, 4096), (7, 4104),
                                      (160, 512), (3, 8191), (2, 32768)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(ctx, dtype, rows, dim, with_residual):
    x = randn(rows, dim, seed=1).to(dtype).cuda()
    w = (1 + 0.3 * randn(dim, seed=2)).to(dtype).cuda()
    r = (4 * randn(rows, dim, seed=3)).to(dtype).cuda() if with_residual else None
    y8, scales, total = ctx.head_norm(x, w, r, eps=1e-5)
    assert y8.dtype == E4M3 and y8.shape == (rows, dim) and y8.stride(0) % 16 == 0
    check_norm(y8, scales, x, w, r, 1e-5)
    if with_residual:
        assert torch.equal(total, (x.float() + r.float()).to(dtype))
    else:
        assert total is None


def test_norm_strides_types_and_place(ctx):
    """Odd strides, unaligned rows, a 32-bit weight, the sum written over the residual."""
    for rows, dim, pad in [(5, 256, 3), (3, 640, 8), (4, 77, 1)]:
        big = randn(rows, dim + pad, seed=4).to(BF16).cuda()
        x = big[:, pad:]
        r = (2 * randn(rows, dim + pad, seed=5)).to(BF16).cuda()[:, :dim]
        w = (1 + 0.1 * randn(dim, seed=6)).float().cuda()
        keep = r.clone()
        out = torch.zeros(rows, dim + 5, device="cuda").to(E4M3)[:, 5:]
        scales = torch.full((rows, 2 * -(-dim // 128)), -1.0, device="cuda")[:, ::2]
        y8, sc, total = ctx.head_norm(x, w, r, eps=1e-6, out=out, scales=scales, residual_out=r)
        assert y8.data_ptr() == out.data_ptr() and total.data_ptr() == r.data_ptr()
        check_norm(y8, sc, x, w, keep, 1e-6)
        assert torch.equal(r, (x.float() + keep.float()).to(BF16))
        x2 = x.clone()
        y8b, _, total = ctx.head_norm(x2, w, keep, eps=1e-6, residual_out=x2)
        assert torch.equal(y8b.float(), y8.float()) and torch.equal(x2, r)
        # columns apart, rows broadcast: inputs are copied
        t = randn(dim, rows, seed=7).to(BF16).cuda().t()
        y8, sc, _ = ctx.head_norm(t, w)
        check_norm(y8, sc, t, w, None, 1e-6)
        one = t[:1].expand(rows, dim)
        y8, sc, _ = ctx.head_norm(one, w)
        check_norm(y8, sc, one, w, None, 1e-6)
        # the sum without a residual is x itself
        assert torch.equal(ctx.head_norm(x, w, residual_out=torch.empty_like(x2))[2], x)


def test_norm_zeros_infinities_and_nan(ctx):
    x = torch.zeros(5, 300, device="cuda")
    x[1] = 1.0
    x[1, 200] = NAN          # the mean is NaN: every block
    x[2, 5] = INF            # the mean is inf, 1/rms 0: 0 elsewhere, NaN at the infinity
    x[3] = 1e-30             # far below eps
    x[4] = 1e20              # squares overflow 32 bits: 1/rms 0
    w = torch.ones(300, device="cuda")
    y8, scales, _ = ctx.head_norm(x, w, eps=1e-6)
    y, s = y8.float().cpu(), scales.cpu()
    assert (y[0] == 0).all() and (s[0] == TINY).all()
    assert s[1].isnan().all() and y[1].isnan().all()
    assert s[2, 0].isnan() and y[2, :128].isnan().all() and (y[2, 128:] == 0).all() and (s[2, 1:] == TINY).all()
    check_norm(y8[3:4], scales[3:4], x[3:4], w, None, 1e-6)
    assert (y[4] == 0).all()
    w[7] = INF               # an infinity in one block only
    y8, scales, _ = ctx.head_norm(torch.ones(1, 300, device="cuda"), w, eps=0.0)
    s = scales.cpu()
    assert s[0, 0] == INF and torch.isfinite(s[0, 1:]).all()
    assert y8.float()[0, 7].isnan() and torch.isfinite(y8.float()[0, 128:]).all()


def test_norm_no_rows(ctx):
    y8, scales, total = ctx.head_norm(torch.empty(0, 256, device="cuda"), torch.ones(256, device="cuda"),
                                      torch.empty(0, 256, device="cuda"))
    assert y8.shape == (0, 256) and scales.shape == (0, 2) and total.shape == (0, 256)


# --------------------------------------------------------------- quantize ---

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,dim", [(1, 1), (128, 128), (129, 127), (300, 1000), (512, 64)])
def test_quantize(ctx, dtype, n, dim):
    w = randn(n, dim + 3, seed=8).to(dtype).cuda()[:, 3:]
    w8, ws = ctx.head_quantize(w)
    assert ws.shape == (-(-n // 128), -(-dim // 128))
    v, q, s = w.cpu().double(), w8.cpu().float().double(), ws.cpu().double()
    for i, (_, r) in enumerate(blocks_of(n)):
        for j, (_, c) in enumerate(blocks_of(dim)):
            want = v[r, c].abs().max().item() / 448
            assert abs(s[i, j].item() - want) <= 2.0 ** -23 * want
            t = v[r, c] / s[i, j]
            step = torch.maximum(t.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
            assert ((q[r, c] - t).abs() <= step * (1 + 2.0 ** -20)).all()


def test_quantize_zeros_and_nan(ctx):
    w = torch.zeros(256, 256, device="cuda")
    w[200, 5] = NAN
    w8, ws = ctx.head_quantize(w)
    assert ws[0, 0] == TINY and ws[1, 1] == TINY and ws[1, 0].isnan()
    assert (w8.float()[:128] == 0).all()


# ----------------------------------------------------------------- logits ---

def logits_inputs(rows, n, dim, seed, x_pad=0, w_pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, dim + x_pad, generator=g).mul_(60).clamp_(-448, 448).to(E4M3).cuda()[:, x_pad:]
    w = torch.randn(n, dim + w_pad, generator=g).mul_(90).clamp_(-448, 448).to(E4M3).cuda()[:, w_pad:]
    kb = -(-dim // 128)
    xs = (torch.rand(rows, kb, generator=g) + 0.01).cuda()
    ws = (torch.rand(-(-n // 128), kb, generator=g) * 0.02 + 1e-4).cuda()
    return x, xs, w, ws


def check_logits(out, x, xs, w, ws):
    rows, dim = x.shape
    n = w.shape[0]
    want = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    X, W = x.float().double(), w.float().double()
    for i, (_, c) in enumerate(blocks_of(dim)):
        s = xs[:, i].double()[:, None] * ws[:, i].double().repeat_interleave(128)[:n][None]
        want += s * (X[:, c] @ W[:, c].t())
        size += s * (X[:, c].abs() @ W[:, c].abs().t())
    tol = (min(dim, 128) + -(-dim // 128) + 4) * 2.0 ** -23 * size
    # the 32-bit sum is within tol, and rounding to the output's type keeps order
    lo, hi = (want - tol).float().to(out.dtype).double(), (want + tol).float().to(out.dtype).double()
    if out.dtype == F32:
        lo, hi = want - tol, want + tol
    assert out.shape == want.shape
    bad = ~((out.double() >= lo) & (out.double() <= hi))
    assert not bad.any(), (bad.nonzero()[:4], out[bad][:4], want[bad][:4])


SIZES = [(1, 1, 1), (1, 512, 128), (1, 4352, 4096), (2, 129, 160), (15, 300, 1040), (16, 512, 512), (17, 4352, 256),
         (31, 1000, 144), (33, 640, 2048), (64, 512, 4096), (65, 300, 512), (127, 257, 128), (128, 256, 384),
         (129, 4352, 1024), (200, 1, 256), (300, 700, 1008), (640, 2048, 512), (1, 32256, 512), (5, 40000, 128)]


@pytest.mark.parametrize("rows,n,dim", SIZES)
def test_logits(ctx, rows, n, dim):
    x, xs, w, ws = logits_inputs(rows, n, dim, seed=rows + n + dim)
    check_logits(ctx.head_logits(x, xs, w, ws), x, xs, w, ws)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows", [3, 20, 50, 140])
def test_logits_types(ctx, dtype, rows):
    x, xs, w, ws = logits_inputs(rows, 777, 640, seed=rows)
    out = ctx.head_logits(x, xs, w, ws.mul_(0.05), dtype=dtype)
    assert out.dtype == dtype
    check_logits(out, x, xs, w, ws)


@pytest.mark.parametrize("rows", [1, 9, 150])
@pytest.mark.parametrize("dim,x_pad,w_pad", [(1000, 0, 0), (129, 1, 3), (127, 0, 1), (256, 16, 32), (512, 1, 0), (77, 3, 0)])
def test_logits_strides(ctx, rows, dim, x_pad, w_pad):
    """Rows that start anywhere, scales in either order, an output inside a wider one."""
    n = 403
    x, xs, w, ws = logits_inputs(rows, n, dim, seed=dim + rows, x_pad=x_pad, w_pad=w_pad)
    xs, ws = xs.t().contiguous().t(), ws.t().contiguous().t()
    wide = torch.full((rows, n + 13), 7.0, device="cuda")
    got = ctx.head_logits(x, xs, w, ws, out=wide[:, 5:5 + n])
    assert got.data_ptr() == wide[:, 5:].data_ptr()
    check_logits(got, x, xs, w, ws)
    assert (wide[:, :5] == 7).all() and (wide[:, 5 + n:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows", [70, 200])
@pytest.mark.parametrize("n", [1, 6, 64, 259, 520])
def test_logits_output_place(ctx, dtype, rows, n):
    """An output whose rows start at any element gets the same values, and nothing around them is written."""
    x, xs, w, ws = logits_inputs(rows, n, 256, seed=rows + n)
    plain = torch.empty(rows, -(-n // 8) * 8, dtype=dtype, device="cuda")[:, :n]
    want = ctx.head_logits(x, xs, w, ws.mul_(0.05), out=plain)
    for before in range(9):
        wide = torch.full((rows, n + 11 + before % 2), 7.0, dtype=dtype, device="cuda")
        ctx.head_logits(x, xs, w, ws, out=wide[:, before:before + n])
        assert torch.equal(wide[:, before:before + n], want)
        assert (wide[:, :before] == 7).all() and (wide[:, before + n:] == 7).all()


def test_logits_copies_on_two_streams_and_in_a_graph(ctx):
    """Rows that have to be copied first: each stream and each captured graph has its own copy."""
    sets = [logits_inputs(5, 4000, 1001, seed=40 + i) for i in range(2)]
    want = [ctx.head_logits(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(ctx.head_logits(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want[0])
    with torch.cuda.graph(graph):
        ctx.head_logits(*sets[0], out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want[0])


def test_logits_nan_stays_in_its_row(ctx):
    for rows in (4, 140):
        x, xs, w, ws = logits_inputs(rows, 300, 512, seed=11)
        clean = ctx.head_logits(x, xs, w, ws)
        xs[1, 2] = NAN
        xs[3, 0] = INF
        out = ctx.head_logits(x, xs, w, ws)
        keep = [r for r in range(rows) if r not in (1, 3)]
        assert out[1].isnan().all() and not torch.isfinite(out[3]).any()
        assert torch.equal(out[keep], clean[keep])


def test_logits_same_bits_every_time(ctx):
    for rows, n, dim in [(1, 512, 4096), (7, 4352, 2048), (300, 1000, 1024)]:
        x, xs, w, ws = logits_inputs(rows, n, dim, seed=12)
        first = ctx.head_logits(x, xs, w, ws)
        for _ in range(5):
            assert torch.equal(ctx.head_logits(x, xs, w, ws), first)


def test_logits_no_rows(ctx):
    x, xs, w, ws = logits_inputs(2, 300, 256, seed=13)
    assert ctx.head_logits(x[:0], xs[:0], w, ws).shape == (0, 300)


def test_logits_offsets_past_32_bits(ctx):
    """An output of more than 2^32 bytes: the last rows land where they belong."""
    rows, n, dim = 4200, 262144, 128
    x, xs, w, ws = logits_inputs(rows, n, dim, seed=14)
    out = torch.empty(rows, n, dtype=F32, device="cuda")
    ctx.head_logits(x, xs, w, ws, out=out)
    for part in (slice(0, 2), slice(2100, 2102), slice(rows - 3, rows)):
        check_logits(out[part], x[part], xs[part], w, ws)


# ----------------------------------------------------------------- sample ---

def per_row(v, rows, kind):
    if v is None:
        return [None] * rows
    return [kind(a) for a in v.cpu().tolist()] if isinstance(v, torch.Tensor) else [kind(v)] * rows


def sample_reference(logits, u, temperature=1.0, top_k=None, top_p=None, min_p=None):
    """Row by row, sorted, in whole numbers; exp is torch's 32-bit one on the GPU."""
    rows, n = logits.shape
    f = np.float32
    temps = per_row(temperature, rows, f)
    ks, ps, qs = per_row(top_k, rows, int), per_row(top_p, rows, f), per_row(min_p, rows, f)
    ids, lps = [], []
    for r in range(rows):
        v = logits[r].float()
        v = torch.where(v.isnan(), -INF, v)
        top = v.max()
        if top == -INF:
            ids.append(-1)
            lps.append(-INF)
            continue
        if not temps[r] >= f(TINY):
            ids.append(int((v == top).nonzero()[0, 0]))
            lps.append(0.0)
            continue
        inv = torch.tensor(f(1.0) / temps[r], device="cuda")
        z = torch.where(v == top, torch.zeros_like(v), (v - top) * inv)
        w = (torch.exp(z).double() * 2.0 ** 40).to(torch.int64).cpu().numpy()
        order = np.argsort(-v.double().cpu().numpy(), kind="stable")
        if ks[r] is not None and 1 <= ks[r] < n:
            order = order[:ks[r]]
        if ps[r] is not None and ps[r] < 1:
            mass = w[order]
            edge = max(1, int(float(ps[r]) * float(mass.sum())))
            order = order[np.cumsum(mass) - mass < edge]
        if qs[r] is not None and qs[r] > 0:
            order = order[w[order] >= int(float(min(qs[r], f(1.0))) * 2.0 ** 40)]
        order = np.sort(order)
        run = np.cumsum(w[order])
        total = int(run[-1])
        at = float(f(u[r].item())) * float(total)
        i = int(order[np.searchsorted(run, min(int(at) if at > 0 else 0, total - 1), side="right")])
        ids.append(i)
        zd = z[i].double().item()
        lps.append(zd - math.log(total * 2.0 ** -40))
    return ids, lps


def check_sample(ctx, logits, u, **kw):
    ids, lp = ctx.head_sample(logits, u, **kw)
    want_ids, want_lp = sample_reference(logits, u, **kw)
    assert ids.cpu().tolist() == want_ids
    for a, b in zip(lp.cpu().tolist(), want_lp):
        # one rounding of a difference of numbers of either size, and the mass's 32-bit weights
        assert a == b if not math.isfinite(b) else abs(a - b) <= 2.0 ** -22 * (2 + abs(b))
    return ids


def uniforms(rows, seed):
    return torch.rand(rows, generator=torch.Generator().manual_seed(seed)).cuda()


def some_logits(rows, n, dtype, seed, spread=3.0):
    return (spread * randn(rows, n, seed=seed)).to(dtype).cuda()


FILTERS = [{}, {"top_k": 1}, {"top_k": 5}, {"top_k": 40}, {"top_p": 0.9}, {"top_p": 0.3}, {"min_p": 0.05},
           {"top_k": 50, "top_p": 0.8}, {"top_k": 20, "top_p": 0.95, "min_p": 0.1}, {"top_p": 0.99, "min_p": 0.001}]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 512, 1023, 4352, 8195])
def test_sample(ctx, dtype, n):
    for i, kw in enumerate(FILTERS):
        check_sample(ctx, some_logits(6, n, dtype, seed=n + i), uniforms(6, i), temperature=0.5 + 0.2 * i, **kw)


@pytest.mark.parametrize("dtype,n,rows", [(F32, 32256, 3), (BF16, 65536, 2), (F32, 250000, 2), (F16, 100001, 2), (BF16, 32256, 5),
                                          (F32, 400001, 1), (BF16, 800003, 1)])
@pytest.mark.parametrize("spread", [0.01, 0.7, 4.0])
def test_sample_large_vocabularies(ctx, dtype, n, rows, spread):
    """Flat rows, whose nuclei hold most of the vocabulary and whose 16-bit values tie, and peaked ones."""
    for i, kw in enumerate([{}, {"top_p": 0.95}, {"top_k": 1000}, {"top_k": n // 2, "top_p": 0.5, "min_p": 0.01}]):
        check_sample(ctx, some_logits(rows, n, dtype, seed=i, spread=spread), uniforms(rows, 50 + i), **kw)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,pad", [(1000, 0), (999, 2), (5120, 0), (5121, 7), (20000, 0)])
def test_sample_more_rows_than_multiprocessors(ctx, dtype, n, pad):
    """CTAs that take several rows in turn; rows with every kind of filter, masks and infinities among them."""
    rows = 2500 if n <= 1000 else 400
    x = some_logits(rows, n + pad, dtype, seed=n)[:, :n]
    x[5::97] = -INF
    x[7::101, n // 2] = INF
    x[11::103, 1:] = NAN
    g = torch.Generator().manual_seed(n)
    kw = {"temperature": torch.rand(rows, generator=g).cuda() + 0.1,
          "top_k": torch.randint(-20, 300, (rows,), generator=g, dtype=torch.int32).cuda(),
          "top_p": (torch.rand(rows, generator=g) * 1.3).cuda(), "min_p": (torch.rand(rows, generator=g) * 0.1 - 0.03).cuda()}
    kw["temperature"][::50] = 0.0
    u = uniforms(rows, n + 1)
    some = torch.arange(0, rows, 7)   # the reference goes row by row
    ids, lp = ctx.head_sample(x, u, **kw)
    want, want_lp = sample_reference(x[some], u[some], **{a: v[some] for a, v in kw.items()})
    assert ids[some].cpu().tolist() == want
    for a, b in zip(lp[some].cpu().tolist(), want_lp):
        assert a == b if not math.isfinite(b) else abs(a - b) <= 2.0 ** -22 * (2 + abs(b))
    plain = {"temperature": 0.7}
    ids, _ = ctx.head_sample(x, u, **plain)
    assert ids[some].cpu().tolist() == sample_reference(x[some], u[some], **plain)[0]


def test_sample_settings_of_each_row(ctx):
    rows, n = 12, 4352
    g = torch.Generator().manual_seed(3)
    t = torch.rand(rows, generator=g) * 1.5
    t[0], t[1], t[2] = 0.0, -1.0, NAN
    k = torch.randint(-1, 60, (rows,), generator=g, dtype=torch.int32)
    p = torch.rand(rows, generator=g) * 1.2
    q = torch.rand(rows, generator=g) * 0.2
    kw = {"temperature": t.cuda(), "top_k": k.cuda(), "top_p": p.cuda(), "min_p": q.cuda()}
    for dtype in (F32, BF16, F16):
        check_sample(ctx, some_logits(rows, n, dtype, seed=4), uniforms(rows, 5), **kw)
    # settings that lie apart, every second value of a longer vector
    apart = {a: torch.stack([v, v], 1).reshape(-1)[::2] for a, v in kw.items()}
    assert not apart["top_p"].is_contiguous()
    logits, u = some_logits(rows, n, F32, seed=4), uniforms(rows, 5)
    assert torch.equal(ctx.head_sample(logits, u, **apart)[0], ctx.head_sample(logits, u, **kw)[0])


def test_sample_masks(ctx):
    """Rows whose mask leaves nothing, one token, or the lowest finite value; infinities and NaN."""
    n = 5000
    x = some_logits(9, n, F32, seed=6)
    x[0] = -INF
    x[1] = NAN
    x[2] = -INF
    x[2, 4321] = -3.0
    x[3] = torch.finfo(F32).min
    x[4, 100:] = torch.finfo(F32).min
    x[5, ::2] = NAN
    x[6, 17] = INF
    x[7, 40] = INF
    x[7, 4000] = INF
    x[8, 50:] = -INF
    for i, kw in enumerate(FILTERS):
        check_sample(ctx, x, uniforms(9, 60 + i), **kw)
        check_sample(ctx, x.to(BF16), uniforms(9, 60 + i), **kw)
    ids = check_sample(ctx, x, uniforms(9, 70), temperature=0.0)
    assert ids[:4].tolist() == [-1, -1, 4321, 0] and ids[6] == 17 and ids[7] == 40


def test_sample_ties_zeros_and_ends(ctx):
    """Equal logits go to the lowest ids; -0 equals 0; u at both ends and outside."""
    x = torch.zeros(4, 700, device="cuda")
    x[1, ::2] = -0.0
    x[2, 300:] = -1.0
    x[3] = torch.arange(700, device="cuda") % 7
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 0.5, 0.999], device="cuda")
    for kw in FILTERS + [{"top_k": 700}, {"top_k": 701}, {"top_p": 0.0}, {"top_p": 1.0}, {"top_p": -1.0}, {"top_p": 1e-30},
                         {"min_p": 1.0}, {"min_p": 2.0}, {"min_p": -1.0}, {"top_k": -3}, {"top_p": NAN}, {"min_p": NAN}]:
        for shift in range(4):
            check_sample(ctx, x, u.roll(shift), **kw)
    ids = ctx.head_sample(x[:1].expand(4, 700), u, top_k=3)[0].tolist()
    assert ids == [0, 2, 1, 2]
    odd = torch.tensor([-1.0, 1.0, 5.0, NAN], device="cuda")
    assert ctx.head_sample(x[:1].expand(4, 700), odd, top_k=3)[0].tolist() == [0, 2, 2, 0]


@pytest.mark.parametrize("temperature", [1e-37, 1e-6, 1e-3, 30.0, 1e30, INF])
def test_sample_temperatures(ctx, temperature):
    for kw in ({}, {"top_p": 0.9}, {"top_k": 9, "min_p": 0.5}):
        check_sample(ctx, some_logits(5, 3001, F32, seed=9), uniforms(5, 10), temperature=temperature, **kw)


def test_sample_strides_and_outputs(ctx):
    n = 1001
    wide = some_logits(6, n + 24, BF16, seed=11)
    for off in (0, 1, 3, 8):
        check_sample(ctx, wide[:, off:off + n], uniforms(6, 12), top_p=0.9)
        check_sample(ctx, wide[::2, off:off + n], uniforms(3, 13), top_k=30)
    check_sample(ctx, some_logits(n, 4, F32, seed=12).t(), uniforms(4, 14), top_p=0.7)
    ids = torch.full((6,), -5, dtype=torch.int32, device="cuda")
    lp = torch.empty(6, device="cuda")
    got = ctx.head_sample(wide[:, :n], uniforms(6, 12), top_p=0.9, ids=ids, logprob=lp)
    assert got[0].data_ptr() == ids.data_ptr() and got[1].data_ptr() == lp.data_ptr() and (ids >= 0).all()
    assert ctx.head_sample(wide[:0], uniforms(0, 1))[0].numel() == 0


def test_sample_follows_the_distribution(ctx):
    """Evenly spaced random numbers: each id comes up by its probability, to within one draw at either end."""
    n, draws = 40, 4096
    x = randn(1, n, seed=15).float().cuda() * 2
    u = (torch.arange(draws, device="cuda") + 0.5) / draws
    for kw in ({}, {"top_k": 7}, {"top_p": 0.8}, {"min_p": 0.1}):
        ids, lp = ctx.head_sample(x.expand(draws, n), u, temperature=0.9, **kw)
        count = torch.bincount(ids.long().cpu(), minlength=n)
        p = torch.softmax(x[0].double().cpu() / 0.9, 0)
        s, order = p.sort(descending=True)
        keep = torch.ones(n, dtype=torch.bool)
        if "top_k" in kw:
            keep[7:] = False
        if "top_p" in kw:
            keep &= s.cumsum(0) - s < 0.8
        if "min_p" in kw:
            keep &= s >= 0.1 * s[0]
        q = torch.zeros(n, dtype=torch.float64)
        q[order[keep]] = s[keep] / s[keep].sum()
        assert ((count - q * draws).abs() <= 1 + 1e-3).all()
        assert (lp.cpu().double() - q[ids.long().cpu()].log()).abs().max() < 1e-5


def test_sample_same_answer_every_time(ctx):
    x, u = some_logits(40, 32256, BF16, seed=16), uniforms(40, 17)
    first = ctx.head_sample(x, u, top_p=0.95)
    for _ in range(5):
        again = ctx.head_sample(x, u, top_p=0.95)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_sample_many_rows_and_offsets_past_32_bits(ctx):
    """Rows that start more than 2^32 elements into the tensor."""
    n = 1 << 21
    x = torch.zeros(2100, n, dtype=BF16, device="cuda")
    x[2099, 77777] = 60.0
    x[2048, 5] = 60.0
    ids = ctx.head_sample(x, uniforms(2100, 18), top_p=0.9)[0]
    assert ids[2099] == 77777 and ids[2048] == 5
    ids = ctx.head_sample(some_logits(1, 1000, F32, seed=19).expand(70000, 1000), uniforms(70000, 20), temperature=0.0)[0]
    assert (ids == ids[0]).all()


# --------------------------------------------------------------- together ---

def test_other_streams_and_graphs(ctx):
    """The step on a side stream, and captured once and replayed on new inputs."""
    rows, dim, n = 6, 640, 4352
    w8, ws = ctx.head_quantize((0.05 * randn(n, dim, seed=21)).to(BF16).cuda())
    g = torch.ones(dim, dtype=BF16, device="cuda")
    h = [randn(rows, dim, seed=22 + i).to(BF16).cuda() for i in range(3)]
    u = uniforms(rows, 25)

    def step(x):
        x8, xs, _ = ctx.head_norm(x, g)
        return ctx.head_sample(ctx.head_logits(x8, xs, w8, ws), u, top_p=0.9)

    want = [step(x) for x in h]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(h[0])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    x = h[0].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(x)
    for i in (1, 2, 0):
        x.copy_(h[i])
        graph.replay()
        assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])


def test_example_generates_the_same_text_again(ctx):
    """examples/generate.py: train, encode, norm, logits, draw and decode in one run; each id had its chance."""
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "generate.py")
    spec = importlib.util.spec_from_file_location("generate", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    out, logprob, texts, merges = example.main(["--rows", "3", "--tokens", "20", "--merges", "64"])
    again = example.main(["--rows", "3", "--tokens", "20", "--merges", "64"])
    assert torch.equal(out, again[0]) and torch.equal(logprob, again[1]) and texts == again[2]
    assert out.shape == (3, 20) and (out >= 0).all() and (out < 256 + len(merges)).all()
    assert (logprob <= 0).all() and torch.isfinite(logprob).all()
    assert all(len(t) >= 20 for t in texts)


def test_refusals(ctx):
    import bpe_trie_encode_gb300 as bt
    x, w = torch.zeros(2, 256, device="cuda"), torch.ones(256, device="cuda")
    cases = [
        (TypeError, lambda: ctx.head_norm(x.cpu(), w)),
        (TypeError, lambda: ctx.head_norm(x.double(), w)),
        (ValueError, lambda: ctx.head_norm(x[0], w)),
        (ValueError, lambda: ctx.head_norm(x, w[:255])),
        (TypeError, lambda: ctx.head_norm(x, w.int())),
        (TypeError, lambda: ctx.head_norm(x, w, x.to(BF16))),
        (ValueError, lambda: ctx.head_norm(x, w, x[:1])),
        (ValueError, lambda: ctx.head_norm(x, w, out=torch.zeros(256, 2, device="cuda").to(E4M3).t())),
        (ValueError, lambda: ctx.head_norm(x, w, scales=torch.zeros(2, 3, device="cuda"))),
        (ValueError, lambda: ctx.head_norm(x, w, scales=torch.zeros(1, 2, device="cuda").expand(2, 2))),
        (bt.BpeError, lambda: ctx.head_norm(x, w, eps=-1.0)),
        (bt.BpeError, lambda: ctx.head_norm(torch.zeros(1, 32769, device="cuda"), torch.ones(32769, device="cuda"))),
        (bt.BpeError, lambda: ctx.head_norm(torch.zeros(1, 0, device="cuda"), torch.ones(0, device="cuda"))),
        (TypeError, lambda: ctx.head_quantize(x.to(E4M3))),
        (bt.BpeError, lambda: ctx.head_quantize(torch.zeros(0, 128, device="cuda"))),
    ]
    x8, xs, w8, ws = logits_inputs(2, 300, 256, seed=30)
    cases += [
        (TypeError, lambda: ctx.head_logits(x8.float(), xs, w8, ws)),
        (TypeError, lambda: ctx.head_logits(x8, xs.double(), w8, ws)),
        (ValueError, lambda: ctx.head_logits(x8, xs[:, :1], w8, ws)),
        (ValueError, lambda: ctx.head_logits(x8, xs, w8[:, :255], ws)),
        (ValueError, lambda: ctx.head_logits(x8, xs, w8, ws[:2])),
        (ValueError, lambda: ctx.head_logits(x8, xs, w8, ws, out=torch.zeros(2, 299, device="cuda"))),
        (ValueError, lambda: ctx.head_logits(x8, xs, w8, ws, out=torch.zeros(300, 2, device="cuda").t())),
        (TypeError, lambda: ctx.head_logits(x8, xs, w8, ws, dtype=torch.float64)),
        (bt.BpeError, lambda: ctx.head_logits(x8, xs, w8[:0], ws[:0])),
    ]
    u = torch.zeros(2, device="cuda")
    cases += [
        (TypeError, lambda: ctx.head_sample(x.double(), u)),
        (TypeError, lambda: ctx.head_sample(x, u.double())),
        (ValueError, lambda: ctx.head_sample(x, u[:1])),
        (TypeError, lambda: ctx.head_sample(x, u, top_k=torch.ones(2, device="cuda"))),
        (ValueError, lambda: ctx.head_sample(x, u, top_p=torch.ones(3, device="cuda"))),
        (TypeError, lambda: ctx.head_sample(x, u, temperature=torch.ones(2))),
        (TypeError, lambda: ctx.head_sample(x, u, ids=torch.zeros(2, device="cuda"))),
        (ValueError, lambda: ctx.head_sample(x, u, ids=torch.zeros(4, dtype=torch.int32, device="cuda")[::2])),
        (bt.BpeError, lambda: ctx.head_sample(torch.zeros(1, 0, device="cuda"), u[:1])),
        (bt.BpeError, lambda: ctx.head_sample(torch.zeros(1, (1 << 22) + 1, dtype=BF16, device="cuda"), u[:1])),
    ]
    for i, (kind, call) in enumerate(cases):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {i} was taken")
    with pytest.raises(bt.BpeError, match="eps"):
        ctx.head_norm(x, w, eps=NAN)
    # the context stays usable
    check_sample(ctx, x, u)
