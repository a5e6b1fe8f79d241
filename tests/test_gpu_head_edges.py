"""The output head on the GPU at its edges: exact roundings, sizes between launch limits, waits that give up, captures."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")
C448 = np.float32(1) / np.float32(448)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ctx():
    import bpe_trie_encode_gb300 as bt
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    c = bt.Context(0)
    yield c
    c.close()


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


# ------------------------------------------------------- exact roundings ---

def blocks_exactly(v):
    """Scales and 8-bit values of the rows of v [rows, dim] (f32), each step one 32-bit operation rounded to nearest even."""
    rows, dim = v.shape
    q, scales = torch.empty(rows, dim), []
    for c in range(0, dim, 128):
        part = v[:, c:c + 128].numpy()
        scale = np.maximum(np.abs(part).max(1) * C448, np.float32(2.0 ** -126))
        q[:, c:c + 128] = torch.from_numpy(part / scale[:, None]).clamp(-448, 448).to(E4M3).float()
        scales.append(torch.from_numpy(scale))
    return q, torch.stack(scales, 1)


@pytest.mark.parametrize("dim,off", [(4096, 0), (1024, 3), (128, 0)])
def test_norm_scales_and_values_are_the_formulas(ctx, dim, off):
    """A state of +-1 has the root mean square 1, so that y is the weight: scales and e4m3(y / scale) bit for bit."""
    sign = randn(64, dim, seed=1).sign()
    for seed in range(8):
        w = randn(dim, seed=10 + seed) * 10.0 ** (seed - 4)
        x = torch.empty(64, dim + off)
        x[:, off:] = sign
        y8, scales, _ = ctx.head_norm(x.cuda()[:, off:], w.cuda(), eps=0.0)
        q, want = blocks_exactly(sign * w)
        assert torch.equal(scales.cpu(), want)
        assert torch.equal(y8.cpu().float(), q)


def test_quantize_scales_and_values_are_the_formulas(ctx):
    for seed in range(4):
        w = randn(128 * 40, 128, seed=20 + seed)
        w8, ws = ctx.head_quantize(w.cuda())
        part = w.view(40, -1).numpy()
        scale = np.abs(part).max(1) * C448
        assert np.array_equal(ws.cpu().numpy()[:, 0], scale)
        assert torch.equal(w8.cpu().float().view(40, -1), torch.from_numpy(part / scale[:, None]).to(E4M3).float())


# --------------------------------------------------- waits that give up ---

def logits_inputs(rows, n, dim, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, dim, generator=g).mul_(60).clamp_(-448, 448).to(E4M3).cuda()
    w = torch.randn(n, dim, generator=g).mul_(90).clamp_(-448, 448).to(E4M3).cuda()
    kb = -(-dim // 128)
    xs = (torch.rand(rows, kb, generator=g) + 0.01).cuda()
    ws = (torch.rand(-(-n // 128), kb, generator=g) * 0.001 + 1e-5).cuda()
    return x, xs, w, ws


# few rows; single CTAs with an output that TMA and that threads write; pairs of CTAs with both
STALLS = [(5, 4096, 256), (50, 4096, 256), (140, 1024, 384), (140, 1023, 384), (512, 60000, 256), (512, 60001, 256)]


@pytest.mark.parametrize("rows,n,dim", STALLS)
def test_logits_wait_that_runs_out(ctx, rows, n, dim):
    """A CTA whose tiles never arrive gives up its waits, all its warps together; the others finish, the failure is
    reported once, and the context stays usable."""
    import bpe_trie_encode_gb300 as bt
    from bpe_trie_encode_gb300 import _capi
    args = logits_inputs(rows, n, dim, seed=rows)
    want = ctx.head_logits(*args)
    out = torch.full_like(want, 5.0)
    ctx.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, 2)
    try:
        ctx.head_logits(*args, out=out)
        torch.cuda.synchronize()
    finally:
        ctx.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, -1)
    done = out == want
    assert not done.all() and done.float().mean() > 0.7
    with pytest.raises(bt.BpeError) as e:
        ctx.head_logits(*args)
    assert e.value.name == "TIMEOUT"
    assert torch.equal(ctx.head_logits(*args), want)


@pytest.mark.parametrize("rows,n,dim,dtype", [s + (F32,) for s in STALLS] + [s + (t,) for s in STALLS[2:4] for t in (BF16, F16)])
def test_logits_that_were_given_up_are_nan(ctx, rows, n, dim, dtype):
    """Nothing of an earlier step is left where a wait gave up."""
    import bpe_trie_encode_gb300 as bt
    from bpe_trie_encode_gb300 import _capi
    args = logits_inputs(rows, n, dim, seed=rows + 1)
    want = ctx.head_logits(*args, dtype=dtype)
    out = torch.full_like(want, 5.0)
    ctx.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, 2)
    try:
        ctx.head_logits(*args, out=out)
        torch.cuda.synchronize()
    finally:
        ctx.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, -1)
    done = out == want
    assert not done.all() and out[~done].isnan().all()
    with pytest.raises(bt.BpeError):
        ctx.head_logits(*args)


def test_draw_from_logits_that_were_given_up(ctx):
    """The draw that is already queued behind them has no token to draw."""
    import bpe_trie_encode_gb300 as bt
    from bpe_trie_encode_gb300 import _capi
    args = logits_inputs(3, 16, 128, seed=1)
    u, out = torch.full((3,), 0.5, device="cuda"), torch.ones(3, 16, device="cuda")
    want = ctx.head_sample(ctx.head_logits(*args), u)   # what a first call sets up is set up
    torch.cuda.synchronize()
    ctx.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, 0)
    try:
        ids, logprob = ctx.head_sample(ctx.head_logits(*args, out=out), u)
        torch.cuda.synchronize()
    finally:
        ctx.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, -1)
    assert (ids == -1).all() and (logprob == -INF).all()
    with pytest.raises(bt.BpeError):
        ctx.head_logits(*args)
    assert torch.equal(ctx.head_sample(ctx.head_logits(*args), u)[0], want[0])


def test_given_up_waits_are_reported(ctx):
    """By a check after a replayed graph, and by the next draw; once each."""
    import bpe_trie_encode_gb300 as bt
    from bpe_trie_encode_gb300 import _capi
    args = logits_inputs(3, 16, 128, seed=2)
    u, out = torch.full((3,), 0.5, device="cuda"), torch.empty(3, 16, device="cuda")
    want = ctx.head_sample(ctx.head_logits(*args, out=out), u)
    torch.cuda.synchronize()
    ctx.head_check()
    graph = torch.cuda.CUDAGraph()
    ctx.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, 0)
    try:
        with torch.cuda.graph(graph):
            ctx.head_logits(*args, out=out)
    finally:
        ctx.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, -1)
    for report in (ctx.head_check, lambda: ctx.head_sample(out, u), lambda: ctx.head_logits(*args)):
        graph.replay()
        torch.cuda.synchronize()
        with pytest.raises(bt.BpeError) as e:
            report()
        assert e.value.name == "TIMEOUT"
        ctx.head_check()
        assert torch.equal(ctx.head_sample(ctx.head_logits(*args), u)[0], want[0])


# ------------------------------------------------- launches of odd widths ---

# f32 rows of 12,281 to 12,288 take less than 48 KB by themselves, but not with the kernel's static arrays
@pytest.mark.parametrize("dim,off", [(8191, 0), (12280, 1), (12281, 0), (12287, 0), (12288, 1), (12289, 0), (32767, 0), (32768, 1)])
def test_norm_widths_in_a_fresh_process(dim, off):
    """The first call of a process, so that no wider one has raised the kernel's limits."""
    code = f"""
import torch, bpe_trie_encode_gb300 as bt
ctx = bt.Context(0)
x = torch.randn(3, {dim} + {off}, device="cuda")[:, {off}:]
w = torch.ones({dim}, device="cuda", dtype=torch.bfloat16)
y8, scales, _ = ctx.head_norm(x, w)
y = x.double() / (x.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
got = y8.double() * scales.double().repeat_interleave(128, 1)[:, :{dim}]
assert ((got - y).abs() <= y.abs() / 15 + 1e-3).all()   # half a step of e4m3 is 2^-4 of the value, 2^-10 of a scale below
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_norm_widths_from_two_threads(ctx):
    """Two contexts of one device: a narrower row's call never takes room from a wider one's."""
    import threading

    import bpe_trie_encode_gb300 as bt
    failed = []

    def run(dim):
        try:
            c = bt.Context(0)
            x, w = torch.randn(2, dim, device="cuda"), torch.ones(dim, device="cuda")
            first = c.head_norm(x, w)[0]
            for _ in range(300):
                assert torch.equal(c.head_norm(x, w)[0].float(), first.float())
        except Exception as e:
            failed.append(repr(e))

    threads = [threading.Thread(target=run, args=(dim,)) for dim in (13001, 32767)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed


# ------------------------------------------------------------------ sizes ---

def test_sizes_and_top_k_beyond_32_bits(ctx):
    one = torch.zeros(1, 1, device="cuda")
    rows = 2 ** 32 + 5
    u = torch.zeros(1, device="cuda").expand(rows)
    with pytest.raises(ValueError, match="above"):
        ctx.head_sample(one.expand(rows, 1), u)
    with pytest.raises(ValueError, match="above"):
        ctx.head_norm(one.expand(rows, 1), torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="above"):
        ctx.head_logits(one.to(E4M3).expand(rows, 1), one.expand(rows, 1), one.to(E4M3), one)
    with pytest.raises(ValueError, match="above"):
        ctx.head_quantize(one.expand(rows, 1))
    x = randn(64, 500, seed=3).cuda()
    u = torch.rand(64, generator=torch.Generator().manual_seed(4)).cuda()
    off = ctx.head_sample(x, u)[0]
    assert torch.equal(ctx.head_sample(x, u, top_k=2 ** 32 + 1)[0], off)
    assert torch.equal(ctx.head_sample(x, u, top_k=-2 ** 33 + 1)[0], off)
    assert not torch.equal(ctx.head_sample(x, u, top_k=1)[0], off)


# --------------------------------------------------------------- captures ---

@pytest.mark.parametrize("rows,off", [(3, 0), (3, 1), (200, 0), (200, 1)])
def test_first_calls_of_a_process_are_captured(rows, off):
    """Nothing has been called before the capture; with off the weights' rows have to be copied to scratch."""
    code = f"""
import torch, bpe_trie_encode_gb300 as bt
rows, dim, n = {rows}, 640, 1000
ctx = bt.Context(0)
g = torch.Generator().manual_seed(1)
h, w = torch.randn(rows, dim, generator=g).cuda(), torch.randn(n, dim, generator=g).cuda()
gain, u = torch.ones(dim, device="cuda"), torch.rand(rows, generator=g).cuda()
w8 = torch.randn(n, dim + {off}, generator=g).mul_(90).clamp_(-448, 448).to(torch.float8_e4m3fn).cuda()[:, {off}:]
torch.cuda.synchronize()

def step():
    x8, xs, _ = ctx.head_norm(h, gain)
    _, ws = ctx.head_quantize(w)
    logits = ctx.head_logits(x8, xs, w8, ws)
    return logits, *ctx.head_sample(logits, u, temperature=30.0, top_p=0.9)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ----------------------------------------------------- infinite distances ---

@pytest.mark.parametrize("dtype,n", [(F32, 1000), (BF16, 4352), (F32, 65536), (F32, 250000), (F32, 400001), (BF16, 800003)])
@pytest.mark.parametrize("temperature", [INF, 3e38])
def test_infinite_distances(ctx, dtype, n, temperature):
    """A distance of infinity leaves nothing at any temperature: neither below an infinite logit nor across the type's range.
    The last two vocabularies are beyond a cluster's shared memory."""
    big = torch.finfo(dtype).max
    x = torch.zeros(4, n, dtype=dtype, device="cuda")
    x[0, 7] = x[0, n - 2] = INF
    x[1] = -big
    x[1, 5] = x[1, 900] = big
    x[2, 100:] = -INF
    x[2, :100] = NAN
    x[2, 40] = -big
    u = torch.tensor([0.25, 0.75, 0.5, 0.999], device="cuda")
    for kw in ({}, {"top_k": 3}, {"top_p": 0.999}, {"top_k": 400, "top_p": 0.99, "min_p": 0.5}):
        ids, logprob = ctx.head_sample(x, u, temperature=temperature, **kw)
        assert ids[:3].tolist() == [7, 900, 40], kw
        half = torch.tensor(0.5).log()
        assert (logprob[:2].cpu() - half).abs().max() < 1e-6 and logprob[2] == 0
        assert ids[3] >= 0 and torch.isfinite(logprob[3])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [8, 72, 128, 136, 1000, 4104])
def test_norm_of_a_state_whose_squares_vanish(ctx, dtype, dim):
    """Without eps 1 / rms is infinite: a block holds infinities, not NaN, also where the row ends inside it; the same by
    either kernel (rows one element off take the general one)."""
    x = torch.full((3, dim + 1), 1e-30, dtype=dtype, device="cuda")
    w = torch.ones(dim, dtype=dtype, device="cuda")
    for rows in (x[:, 1:], x[:, 1:].contiguous()):
        y8, scales, _ = ctx.head_norm(rows, w, eps=0.0)
        assert (scales == INF).all()
        zero = ctx.head_norm(torch.zeros_like(rows), w, eps=0.0)   # 0 * infinity
        assert zero[1].isnan().all()


# ------------------------------------------- several tiles a CTA or a pair ---

def logits_bounds(x, xs, w, ws):
    """The product in 64 bits, and how far 32-bit sums may be from it (2^-23 of the magnitudes for each addition)."""
    rows, dim = x.shape
    n = w.shape[0]
    want = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    X, W = x.float().double(), w.float().double()
    for i, c in enumerate(range(0, dim, 128)):
        s = xs[:, i].double()[:, None] * ws[:, i].double().repeat_interleave(128)[:n][None]
        want += s * (X[:, c:c + 128] @ W[:, c:c + 128].t())
        size += s * (X[:, c:c + 128].abs() @ W[:, c:c + 128].abs().t())
    return want, (min(dim, 128) + -(-dim // 128) + 4) * 2.0 ** -23 * size


def check_bounds(out, want, tol):
    lo, hi = want - tol, want + tol
    if out.dtype != F32:   # rounding to the output's type keeps order
        lo, hi = lo.float().to(out.dtype).double(), hi.float().to(out.dtype).double()
    bad = ~((out.double() >= lo) & (out.double() <= hi))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


# on 152 SMs: pairs of CTAs with 6 to 7 tiles each of 5, 4, 1 and 9 blocks, then single CTAs with 4 to 5 of 9, 4 and 3
@pytest.mark.parametrize("rows,n,dim", [(512, 60000, 640), (512, 60001, 512), (500, 60004, 100), (400, 60004, 1040),
                                        (300, 60000, 1040), (300, 60001, 512), (290, 60004, 384)])
def test_logits_of_many_tiles(ctx, rows, n, dim):
    """Stages, sums and scales carried from tile to tile, with outputs that TMA writes whole, up to the last 16 bytes of a
    row, or not at all."""
    x, xs, w, ws = logits_inputs(rows, n, dim, seed=dim)
    want, tol = logits_bounds(x, xs, w, ws)
    for dtype in (F32, BF16, F16):
        check_bounds(ctx.head_logits(x, xs, w, ws, dtype=dtype), want, tol)
        for before, wide in ((0, -(-n // 8) * 8), (1, n + 3)):
            out = torch.full((rows, wide), 7.0, dtype=dtype, device="cuda")
            ctx.head_logits(x, xs, w, ws, out=out[:, before:before + n])
            check_bounds(out[:, before:before + n], want, tol)
            assert (out[:, :before] == 7).all() and (out[:, before + n:] == 7).all()


# ------------------------------------------------------ what pads the rows ---

@pytest.mark.parametrize("dim", [127, 1000, 1039])
@pytest.mark.parametrize("rows", [1, 2, 40, 150, 600])
def test_logits_do_not_read_past_a_row(ctx, dim, rows):
    """Rows that start on 16 bytes and end inside them go to TMA as they are: whatever pads them, NaN included."""
    n = 300
    x, xs, w, ws = logits_inputs(rows, n, dim, seed=dim + rows)
    got = []
    for pad in (0x00, 0x70, 0x7F):   # 0, 256, NaN
        def padded(t):
            full = torch.full((t.shape[0], -(-dim // 16) * 16), pad, dtype=torch.uint8, device="cuda")
            full[:, :dim] = t.view(torch.uint8)
            return full.view(E4M3)[:, :dim]
        got.append(ctx.head_logits(padded(x), xs, padded(w), ws))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    check_bounds(got[0], *logits_bounds(x, xs, w, ws))


@pytest.mark.parametrize("off", [0, 1])
def test_graph_that_outlives_its_context(off):
    """Nothing that a captured product uses ends with the context, the word that a given-up wait sets included."""
    import bpe_trie_encode_gb300 as bt
    from bpe_trie_encode_gb300 import _capi
    x, xs, w, ws = logits_inputs(4, 4096, 256, seed=5)
    w = torch.cat([w[:, :off].view(torch.uint8), w.view(torch.uint8)], 1).view(E4M3)[:, off:]
    graphs, outs = [], []
    c = bt.Context(0)
    want = c.head_logits(x, xs, w, ws)
    torch.cuda.synchronize()
    for stall in (-1, 2):
        outs.append(torch.zeros_like(want))
        graphs.append(torch.cuda.CUDAGraph())
        c.set_option(_capi.BPE_OPT_TEST_STALL_HEAD, stall)
        with torch.cuda.graph(graphs[-1]):
            c.head_logits(x, xs, w, ws, out=outs[-1])
    c.close()
    for _ in range(2):
        outs[0].zero_()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert outs[1].isnan().any()
    other = bt.Context(0)   # has the word now, and begins without a report
    assert torch.equal(other.head_logits(x, xs, w, ws), want)
    torch.cuda.synchronize()
    other.head_check()
    other.close()


def test_quantize_scales_over_the_whole_range(ctx):
    """A column of weights has a scale per 128: magnitudes from the smallest scale's to near the type's largest."""
    blocks = 16384
    g = torch.Generator().manual_seed(30)
    size = 2.0 ** torch.randint(-117, 127, (blocks, 1), generator=g).float()
    w = (torch.rand(blocks, 128, generator=g) * 2 - 1) * size
    w8, ws = ctx.head_quantize(w.view(-1, 1).cuda())
    part = w.numpy()
    scale = np.maximum(np.abs(part).max(1) * C448, np.float32(2.0 ** -126))
    assert np.array_equal(ws.cpu().numpy()[:, 0], scale)
    assert torch.equal(w8.cpu().float().view(blocks, 128), torch.from_numpy(part / scale[:, None]).to(E4M3).float())
