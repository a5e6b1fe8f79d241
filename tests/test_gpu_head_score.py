"""Scoring and distillation of the output head on the GPU against plain implementations in 64 bits.

With U = 2^-24, the half step of 32 bits: z = (v - m) c is off by some roundings of |z|, an exponential of it by that and
two steps, a sum of n terms by the depth of its additions (n / 256 of a thread at most, and some twenty more), each U of
the sum of magnitudes.  `room` adds these up, eight roundings of |z| for its four (difference, 1 / T, log2 e, product) and
their spread over the row.  Results of 16 bits add half a step of their own.  Ids have no tolerance.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")
U = 2.0 ** -24
TINY = 2.0 ** -126
LEAST = {F32: 2.0 ** -126, BF16: 2.0 ** -126, F16: 2.0 ** -25}   # numbers below may be lost: half the smallest, or flushed


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


def inverse(t, rows):
    """1 / temperature in 32 bits, infinity for the limit: float64 [rows, 1]."""
    t = np.asarray(t.cpu() if isinstance(t, torch.Tensor) else [t] * rows, dtype=np.float32)
    with np.errstate(all="ignore"):
        c = np.where(t >= np.float32(2.0 ** -126), np.float32(1.0) / t, np.float32(INF))
    return torch.from_numpy(c.astype(np.float64))[:, None]


def softmax64(logits, t=1.0):
    """m, z, p, log s of the definition, in 64 bits; rows without a logit above -infinity have p = 0."""
    v = logits.detach().cpu().double()
    v = torch.where(torch.isnan(v), -INF, v)
    m = v.amax(1, keepdim=True)
    d = torch.where(v == m, 0.0, v - m)
    d = torch.where(d < -torch.finfo(F32).max * (1 + U), -INF, d)   # -infinity where the difference in 32 bits is
    c = inverse(t, v.shape[0])
    z = torch.where(d == 0, 0.0, torch.where(d == -INF, -INF, d * c))
    z = torch.where((v == m) & (m > -INF), 0.0, z)
    z = torch.where(m > -INF, z, torch.full_like(z, -INF))
    e = torch.exp(z)
    s = e.sum(1, keepdim=True)
    return m[:, 0], z, torch.where(s > 0, e / s, 0.0), torch.where(s > 0, torch.log(s), 0.0)[:, 0], c


def mean_of(p, x):
    return torch.where(p > 0, p * x, 0.0).sum(1)


def room(z, p, log_s):
    """What log s may be off by, in units of U."""
    n = z.shape[1]
    return 8 * mean_of(p, z.abs()) + 2 * log_s.abs() + n / 256 + 40


def near(got, want, tol):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    want = torch.where(want.abs() > torch.finfo(F32).max, INF * want.sign(), want)
    same = got == want   # infinities
    off = torch.where(same, 0.0, (got - want).abs())
    bad = ~(off <= tol)
    assert not bad.any(), (got[bad][:4], want[bad][:4], (tol + 0 * off)[bad][:4], bad.nonzero()[:4])


def check_logprobs(ctx, logits, ids, t=1.0, top=0):
    out = ctx.head_logprobs(logits, ids, temperature=t, top=top)
    rows, n = logits.shape
    m, z, p, log_s, c = softmax64(logits, t)
    lp, entropy, top_ids, top_lp, norm = out
    r = room(z, p, log_s)
    near(norm[:, 0], m, torch.zeros(rows))
    near(norm[:, 1], log_s, U * r)
    ez = mean_of(p, z.abs())
    # log s - sum p z: the second has the roundings of its terms, and the sum's
    near(entropy, log_s - mean_of(p, z), U * (r * (1 + ez) + 8 * mean_of(p, z * z) + 8 * ez))
    if ids is not None:
        i = ids.cpu().long()
        ok = (i >= 0) & (i < n)
        zi = z.gather(1, i.clamp(0, n - 1)[:, None])[:, 0]
        want = torch.where(ok, zi - log_s, 0.0)
        near(lp, want, torch.where(zi == -INF, 0.0, U * (r + 8 * zi.abs() + 2 * want.abs())))
    else:
        assert lp is None
    if not top:
        assert top_ids is None and top_lp is None
        return out
    v = logits.cpu().double()
    v = torch.where(torch.isnan(v), -INF, v)
    order = torch.sort(-v, dim=1, stable=True).indices[:, :top]
    if order.shape[1] < top:
        order = torch.cat([order, torch.zeros(rows, top - order.shape[1], dtype=torch.long)], 1)
    some = (v > -INF).sum(1, keepdim=True)
    there = torch.arange(top)[None] < some
    assert torch.equal(top_ids.cpu().long(), torch.where(there, order, -1))
    zt = z.gather(1, order)
    want = torch.where(there, zt - log_s[:, None], -INF)
    near(top_lp, want, torch.where(want == -INF, 0.0, U * (r[:, None] + 8 * zt.abs() + 2 * want.abs())))
    return out


def grad64(logits, ids, a, b, t=1.0):
    """The gradient of a logprob + b entropy, and what it may be off by before its rounding."""
    m, z, p, log_s, c = softmax64(logits, t)
    rows, n = z.shape
    lp = z - log_s[:, None]
    h = (log_s - mean_of(p, z))[:, None]
    i = ids.cpu().long()
    ok = (i >= 0) & (i < n)
    a = torch.where(ok, a.cpu().double(), 0.0)[:, None]
    b = b.cpu().double()[:, None] if b is not None else torch.zeros(rows, 1, dtype=torch.float64)
    hot = torch.zeros_like(p).scatter_(1, i.clamp(0, n - 1)[:, None], ok.double()[:, None])
    lp0 = torch.where(p > 0, lp, 0.0)
    dead = (m == -INF)[:, None] | torch.isinf(c)
    c0 = torch.where(dead, 0.0, c)
    d = torch.where(dead, 0.0, c0 * (a * (hot - p) - b * p * (lp0 + h)))
    r = room(z, p, log_s)[:, None]
    rel = U * (8 * torch.where(p > 0, z.abs(), 0.0) + r + 16)
    ez = mean_of(p, z.abs())[:, None]
    off = c0 * (p * rel * (a.abs() + b.abs() * (lp0.abs() + h)) + b.abs() * p * U * (r * (2 + ez) + 16 * (lp0.abs() + h) + 8 * ez)
                + 4 * U * a.abs() * hot)
    # exponentials relative to the largest are flushed below 2^-126: what they are multiplied by is lost that often
    off = off + c0 * TINY * (a.abs() + b.abs() * (lp0.abs() + h))
    return d, torch.where(dead, 0.0, off)


def rounded(got, want, off, dtype, scale=1.0):
    """Off by `off`, and by half a step of the type; what is smaller than its smallest number is lost."""
    half = torch.finfo(dtype).eps / 2 if dtype != F32 else 4 * U
    near(got.float(), want, off * (1 + 2 * half) + half * want.abs() + LEAST[dtype] * (1 + scale))


SIZES = [(1, 1), (3, 2), (2, 7), (5, 130), (4, 1000), (300, 263), (3, 4351), (2, 32256), (1, 65537), (1, 250000), (160, 2049)]


def some_logits(rows, n, dtype, seed=0):
    v = 2 * randn(rows, n, seed=seed)
    k = min(n, 30)
    v.scatter_(1, torch.randint(0, n, (rows, k), generator=torch.Generator().manual_seed(seed + 1)), 8 + 3 * randn(rows, k, seed=seed + 2))
    return v.to(dtype).cuda()


def some_ids(rows, n, seed=0):
    ids = torch.randint(0, n, (rows,), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    if rows > 2:
        ids[1], ids[2] = -1, n
    return ids.cuda()


# --------------------------------------------------------- log-probabilities ---

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("top", [0, 1, 20, 128])
def test_logprobs(ctx, dtype, rows, n, top):
    check_logprobs(ctx, some_logits(rows, n, dtype), some_ids(rows, n), t=1.0, top=top)


def hard_rows(n, dtype):
    """Rows at which a softmax goes wrong: masks of every kind, infinities, equal and sorted logits, far spreads."""
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    v = 2 * randn(18, n, seed=5)
    v[0] = -INF
    v[1] = NAN
    v[2] = low
    v[3] = -INF
    v[3, n // 2] = 1.5
    v[4] = low
    v[4, n - 1] = -3.0
    v[4, 0] = 0.25
    v[5, n // 3] = INF
    v[6, n // 3] = INF
    v[6, n - 1] = INF
    v[7] = 0.0
    v[8] = torch.linspace(-20, 20, n, dtype=torch.float64)
    v[9] = torch.linspace(20, -20, n, dtype=torch.float64)
    v[10, ::2] = NAN
    v[11, ::3] = -INF
    v[12] = high
    v[13] = low
    v[13, 0] = high
    v[14] = -INF
    v[14, : min(n, 5)] = low
    v[15] = torch.where(randn(n, seed=6) > 0, 0.0, -0.0)
    v[16] = torch.round(v[16])           # many equal ones
    v[17] = -1e4 + v[17] if dtype != BF16 else -1e30
    return v.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [1, 5, 300, 5000, 40001])
@pytest.mark.parametrize("top", [0, 3, 60, 128])
def test_logprobs_of_hard_rows(ctx, dtype, n, top):
    logits = hard_rows(n, dtype)
    for j in (0, n // 3, n - 1):
        check_logprobs(ctx, logits, torch.full((len(logits),), j, dtype=torch.int32).cuda(), top=top)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(7, 50), (7, 5000), (7, 300_000), (900, 2000)])
def test_alternatives_of_masked_rows(ctx, dtype, rows, n):
    """Fewer tokens than alternatives, the others at -infinity, at the type's lowest value, or at several low values."""
    low = torch.finfo(dtype).min
    x = 2 * randn(rows, n, seed=91)
    keep = torch.zeros(rows, n, dtype=torch.bool)
    keep.scatter_(1, torch.randint(0, n, (rows, 6), generator=torch.Generator().manual_seed(4)), True)
    x[0::7] = torch.where(keep, x, -INF)[0::7]
    x[1::7] = torch.where(keep, x, low)[1::7]
    x[2::7] = torch.where(keep, x, NAN)[2::7]
    x[3::7] = torch.where(keep, x, -INF)[3::7]
    x[3::7, n - 3:] = low                          # three masked ones at the end, and nothing else
    x[4::7] = torch.where(keep, x, low)[4::7]
    x[4::7, n // 2:n // 2 + 2] = low / 2           # two values below every other
    x[5::7] = torch.where(keep, x, low / 2)[5::7]
    x[5::7, n // 3] = low
    x = x.to(dtype).cuda()
    some = torch.arange(min(rows, 14))
    for top in (1, 5, 6, 7, 20, 128):
        for t in (1.0, 0.7):
            out = ctx.head_logprobs(x, None, temperature=t, top=top)

            class Some:
                @staticmethod
                def head_logprobs(*_, **__):
                    return tuple(o if o is None else o[:len(some)] for o in out)

            check_logprobs(Some, x[:len(some)], None, t=t, top=top)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [40, 4351])
def test_logprobs_at_any_temperature(ctx, dtype, n):
    ts = [1.0, 0.01, 100.0, 0.0, -1.0, NAN, INF, 2.0 ** -126, 2.0 ** -127, 1e-30, 1e30, 3e38, 1e-4, 1e5]
    t = torch.tensor(ts).cuda()
    logits = some_logits(len(ts), n, dtype, seed=3)
    logits[:, 7] = logits.amax(1)            # two largest ones
    logits[:, 9] = -INF
    check_logprobs(ctx, logits, some_ids(len(ts), n), t=t, top=20)
    for one in (0.7, 0.0, INF):
        check_logprobs(ctx, logits, some_ids(len(ts), n), t=one, top=2)
    hard = hard_rows(n, dtype)
    for one in (0.25, 3.0, 0.0, INF, 1e20, 1e-20):
        check_logprobs(ctx, hard, some_ids(len(hard), n), t=one, top=5)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_logprobs_of_views(ctx, dtype):
    """Rows that start anywhere, wide strides, broadcast rows, columns apart; only what was asked for is written."""
    for rows, n, pad in [(3, 1000, 1), (5, 333, 3), (2, 4096, 8), (4, 4096, 5), (2, 30001, 7)]:
        big = some_logits(rows, n + pad, dtype, seed=n)
        ids = some_ids(rows, n)
        check_logprobs(ctx, big[:, pad:], ids, t=0.9, top=20)
        check_logprobs(ctx, big[:, :n], ids, t=0.9, top=20)
        check_logprobs(ctx, big[:1, pad:].expand(rows, n), ids, top=7)
        check_logprobs(ctx, big.t().contiguous().t()[:, :n], ids, top=7)
    logits, ids = some_logits(4, 900, dtype), some_ids(4, 900)
    buf = torch.full((64, 5), -7.0, device="cuda")
    top = ctx.head_logprobs(logits, ids, top=5, top_logprob=buf[3:7], logprob=buf[20, :4], entropy=buf.view(-1)[151:155],
                            norm=buf.view(-1)[201:209].view(4, 2))
    assert top[3].data_ptr() == buf[3:7].data_ptr() and top[4].data_ptr() == buf.view(-1)[201:].data_ptr()
    mark = torch.zeros_like(buf, dtype=torch.bool)
    mark[3:7], mark[20, :4] = True, True
    mark.view(-1)[151:155], mark.view(-1)[201:209] = True, True
    assert (buf[~mark] == -7).all() and (buf[mark] != -7).all()
    again = ctx.head_logprobs(logits, ids, top=5)
    for a, b in zip(top, again):
        assert torch.equal(a, b)


def test_logprobs_agree_with_the_draw(ctx):
    """The log-probability that a draw returns is that of the same id here."""
    logits = some_logits(64, 4352, BF16)
    ids, lp = ctx.head_sample(logits, torch.rand(64, generator=torch.Generator().manual_seed(0)).cuda(), temperature=0.8)
    mine = check_logprobs(ctx, logits, ids, t=0.8)[0]
    # the draw's weights are whole numbers of 2^-40
    near(lp, mine.cpu(), 1e-5 + 4352 * 2.0 ** -40)


# ------------------------------------------------------------ its gradient ---

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("with_entropy", [False, True])
def test_backward(ctx, dtype, rows, n, with_entropy):
    logits, ids = some_logits(rows, n, dtype, seed=11), some_ids(rows, n)
    t = (0.5 + torch.rand(rows, generator=torch.Generator().manual_seed(1))).cuda()
    _, h, _, _, norm = ctx.head_logprobs(logits, ids, temperature=t)
    a = randn(rows, seed=12).float().cuda()
    b = randn(rows, seed=13).float().cuda() if with_entropy else None
    d = ctx.head_logprobs_backward(logits, ids, norm, a, h if with_entropy else None, b, temperature=t)
    assert d.dtype == dtype
    want, off = grad64(logits, ids, a, b, t)
    rounded(d, want, off, dtype)
    if with_entropy:
        d = ctx.head_logprobs_backward(logits, None, norm, None, h, b, temperature=t)
        want, off = grad64(logits, ids, torch.zeros(rows), b, t)
        rounded(d, want, off, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [1, 5, 300, 5000])
def test_backward_of_hard_rows(ctx, dtype, n):
    logits = hard_rows(n, dtype)
    rows = len(logits)
    for t in (1.0, 0.0, INF, 0.25, 1e-20):
        for j in (0, n // 3):
            ids = torch.full((rows,), j, dtype=torch.int32).cuda()
            _, h, _, _, norm = ctx.head_logprobs(logits, ids, temperature=t)
            a, b = randn(rows, seed=12).float().cuda(), randn(rows, seed=13).float().cuda()
            d = ctx.head_logprobs_backward(logits, ids, norm, a, h, b, temperature=t)
            want, off = grad64(logits, ids, a, b, t)
            big = want.abs() > torch.finfo(dtype).max
            assert torch.isfinite(d.cpu()[~big]).all()
            rounded(torch.where(big.cuda(), 0, d), torch.where(big, 0.0, want), torch.where(big, 0.0, off), dtype)


def test_backward_against_differences(ctx):
    n, rows = 37, 4
    logits, ids = some_logits(rows, n, F32, seed=21), torch.tensor([3, -1, 0, 36], dtype=torch.int32).cuda()
    a, b = randn(rows, seed=22).float().cuda(), randn(rows, seed=23).float().cuda()
    t = 0.8
    _, h, _, _, norm = ctx.head_logprobs(logits, ids, temperature=t)
    d = ctx.head_logprobs_backward(logits, ids, norm, a, h, b, temperature=t).cpu().double()

    def value(v):   # 64 bits
        y = v / float(np.float32(t))
        lp = torch.log_softmax(y, 1)
        i = ids.cpu().long()
        given = torch.where(i >= 0, lp.gather(1, i.clamp_min(0)[:, None])[:, 0], 0.0)
        return a.cpu().double() * given - b.cpu().double() * (lp.exp() * lp).sum(1)

    v, step = logits.cpu().double(), 1e-4
    for j in range(n):
        e = torch.zeros(rows, n, dtype=torch.float64)
        e[:, j] = step
        # the third derivative is below 30 (|a| + |b|) / t^3, times step^2 / 6; the gradient's own error below 500 U of 3
        near(d[:, j], (value(v + e) - value(v - e)) / (2 * step), 1e-4 + 30 * 3 * step ** 2)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_backward_of_views_and_in_place(ctx, dtype):
    for rows, n, pad in [(3, 1000, 1), (5, 333, 3), (2, 4096, 8), (4, 4096, 5), (2, 30001, 7)]:
        big = some_logits(rows, n + pad, dtype, seed=n)
        ids, a = some_ids(rows, n), randn(rows, seed=3).float().cuda()
        for x in (big[:, pad:], big[:, :n]):
            norm = ctx.head_logprobs(x, ids)[4]
            want, off = grad64(x, ids, a, None)
            plain = ctx.head_logprobs_backward(x, ids, norm, a)
            rounded(plain, want, off, dtype)
            for shift in (0, 1, 3):   # an output that starts elsewhere
                frame = torch.full((rows, n + 9), -7.0, dtype=dtype, device="cuda")
                d = ctx.head_logprobs_backward(x, ids, norm, a, out=frame[:, shift:shift + n])
                assert torch.equal(d, plain)
                assert (frame[:, :shift] == -7).all() and (frame[:, shift + n:] == -7).all()
            both = big.clone()
            y = both[:, pad:] if x.data_ptr() != big.data_ptr() else both[:, :n]
            assert ctx.head_logprobs_backward(y, ids, norm, a, out=y).data_ptr() == y.data_ptr()
            assert torch.equal(y, plain)
            edge, kept = (both[:, :pad], big[:, :pad]) if x.data_ptr() != big.data_ptr() else (both[:, n:], big[:, n:])
            assert torch.equal(edge, kept)
        # logits and gradient side by side in one buffer
        wide = torch.full((rows, 2 * n), -7.0, dtype=dtype, device="cuda")
        wide[:, :n] = big[:, :n]
        norm = ctx.head_logprobs(wide[:, :n], ids)[4]
        ctx.head_logprobs_backward(wide[:, :n], ids, norm, a, out=wide[:, n:])
        assert torch.equal(wide[:, :n], big[:, :n])
        rounded(wide[:, n:], *grad64(big[:, :n], ids, a, None), dtype)


# ------------------------------------------------------------- distillation ---

def distill64(logits, ids, values, t, rest, g=None):
    """loss, what it may be off by, the gradient and what it may be off by before its rounding; entry by entry."""
    m, z, p, log_s, c = softmax64(logits, t)
    rows, n = z.shape
    ids, values = ids.cpu().long(), values.detach().cpu().double()
    k = ids.shape[1]
    loss, off = torch.zeros(rows, dtype=torch.float64), torch.zeros(rows, dtype=torch.float64)
    d, doff = torch.zeros_like(z), torch.zeros_like(z)
    r_all = room(z, p, log_s)
    for r in range(rows):
        ok = (ids[r] >= 0) & (ids[r] < n) & (values[r] > -INF)
        i, x = ids[r][ok], values[r][ok]
        if rest:
            lq, e_lq = x, x.abs() * 2
        else:
            top = x.max() if len(x) else torch.tensor(0.0)
            zq = torch.where(x == top, 0.0, x - top)
            lq = zq - torch.logsumexp(zq, 0) if len(x) else x
            e_lq = 4 * zq.abs() + 4 * lq.abs() + 24
        q = lq.exp()
        e_q = q * (e_lq + 6)                       # of a q, in U
        total = q.sum()
        e_total = e_q.sum() + 24 * total
        q_rest = torch.clamp(1 - total, min=0.0) if rest else torch.tensor(0.0, dtype=torch.float64)
        e_rest = e_total + 4 if rest else 0.0
        listed = torch.zeros(n, dtype=torch.bool)
        listed[i] = True
        above = logits[r].cpu() > -INF   # a NaN is not
        if not above[~listed].any():
            q_rest = 0.0 * q_rest
        Q = total + q_rest
        if m[r] == -INF:
            loss[r] = INF if Q > 0 else 0.0
            continue
        lp = z[r] - log_s[r]
        has = q > 0
        loss[r] = (q[has] * (lq[has] - lp[i][has])).sum()
        rr = r_all[r]
        fin = has & (lp[i] > -INF)
        off[r] = (e_q[fin] * (lq[fin].abs() + lp[i][fin].abs() + 1) + q[fin] * (e_lq[fin] + 8 * z[r][i][fin].abs() + 2 * lp[i][fin].abs() + rr)).sum() + 24 * (
            q[fin] * (lq[fin].abs() + lp[i][fin].abs())).sum()
        ratio, e_ratio = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
        if rest and above[~listed].any():
            # 1 - sum of q, exact once the sum is (both are near 1), is off by what the sum is, U * e_rest, on either side of 0
            # too: x log x is off by that times the logarithm of the larger of the two, and each share by that
            least = torch.maximum(q_rest, U * e_rest)
            lpr = torch.logsumexp(lp[~listed], 0)
            if lpr == -INF:
                loss[r] = INF if q_rest > 0 else loss[r]
            # the share of each among them, relative to their largest
            zu = softmax64(logits[r:r + 1].masked_fill(listed.to(logits.device), -INF), t[r:r + 1] if isinstance(t, torch.Tensor) else t)
            share, zz = zu[2][0], torch.where(zu[2][0] > 0, zu[1][0].abs(), 0.0)
            ez = (share * zz).sum()
            if lpr > -INF:
                e_lpr = rr + 8 * (lpr - log_s[r]).abs() + 8 * ez + 10 * lpr.abs() + n / 256 + 40
                loss[r] += q_rest * (q_rest.log() - lpr) if q_rest > 0 else 0.0
                off[r] += e_rest * (least.log().abs() + lpr.abs() + 1) + q_rest * e_lpr
            ratio = q_rest * share
            e_ratio = share * e_rest + ratio * (8 * zz + 8 * ez + n / 256 + 60)
        qj = torch.zeros(n, dtype=torch.float64).index_add_(0, i, q)
        e_qj = torch.zeros(n, dtype=torch.float64).index_add_(0, i, e_q + 4 * q)
        if not torch.isinf(c[r]):
            w = float(c[r]) * (float(g[r]) if g is not None else 1.0)
            d[r] = w * (Q * p[r] - qj - ratio)
            zz = torch.where(p[r] > 0, z[r].abs(), 0.0)
            doff[r] = abs(w) * U * (Q * p[r] * (8 * zz + rr + 30) + p[r] * (e_total + e_rest) + e_qj + 4 * qj + e_ratio)
            doff[r] += abs(w) * TINY * (Q + q_rest)   # flushed exponentials, as above
    return loss, U * off, d, doff


def check_distill(ctx, logits, ids, values, t=1.0, rest=False, g=None):
    rows = len(logits)
    loss, none = ctx.head_distill(logits, ids, values, temperature=t, rest=rest)
    assert none is None
    if g is None:
        g = (0.5 + torch.rand(rows, generator=torch.Generator().manual_seed(9))).cuda()
    loss2, d = ctx.head_distill(logits, ids, values, temperature=t, rest=rest, grad=g)
    assert d.dtype == logits.dtype
    want, off, dwant, doff = distill64(logits, ids, values, t, rest, g)
    near(loss, want, off)
    near(loss2, want, off)
    big = dwant.abs() > torch.finfo(logits.dtype).max
    assert torch.isfinite(d.cpu()[~big]).all()
    rounded(torch.where(big.cuda(), 0, d), torch.where(big, 0.0, dwant), torch.where(big, 0.0, doff), logits.dtype)
    return loss2, d


def some_teacher(logits, k, seed=0, noise=1.0):
    t = logits.cpu().double() + noise * randn(*logits.shape, seed=seed)
    lp = torch.log_softmax(t, 1)
    top = lp.topk(min(k, logits.shape[1]), dim=1)
    ids, values = top.indices.to(torch.int32), top.values.float()
    if ids.shape[1] < k:
        pad = k - ids.shape[1]
        ids = torch.cat([ids, torch.full((len(ids), pad), -1, dtype=torch.int32)], 1)
        values = torch.cat([values, torch.zeros(len(ids), pad)], 1)
    return ids.cuda(), values.cuda()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("k", [1, 8, 65, 128])
@pytest.mark.parametrize("rest", [False, True])
def test_distill(ctx, dtype, rows, n, k, rest):
    logits = some_logits(rows, n, dtype, seed=31)
    ids, values = some_teacher(logits, k)
    t = (0.5 + torch.rand(rows, generator=torch.Generator().manual_seed(1))).cuda()
    check_distill(ctx, logits, ids, values, t=t, rest=rest)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("value_type", [F32, BF16, F16])
def test_distill_of_odd_lists(ctx, rest, value_type):
    """Ids twice, ids of nothing, values of -infinity and NaN, empty lists, a list of every token."""
    n = 900
    logits = some_logits(8, n, F32, seed=41)
    ids = torch.randint(0, n, (8, 20), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    values = torch.log_softmax(randn(8, 25, seed=42), 1)[:, :20].clone()
    ids[0, 5] = ids[0, 3]
    ids[0, 19] = ids[0, 3]
    ids[1, :] = ids[1, 0]
    ids[2, 4:] = -1
    ids[3, ::2] = n
    ids[3, 1] = 2 ** 31 - 1
    ids[3, 3] = -2 ** 31
    values[4, ::3] = -INF
    values[4, 1] = NAN
    ids[5, :] = -1
    values[6, :] = -INF
    values[7, 3:] = -200.0   # a q of 0: listed all the same
    check_distill(ctx, logits, ids.cuda(), values.to(value_type).cuda(), rest=rest)
    few = some_logits(3, 20, F32, seed=43)
    every = torch.arange(20, dtype=torch.int32).expand(3, 20).contiguous().cuda()
    values = torch.log_softmax(randn(3, 20, seed=44), 1)
    check_distill(ctx, few, every, values.to(value_type).cuda(), rest=rest)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("n", [1, 5, 300, 5000])
def test_distill_of_hard_rows(ctx, dtype, rest, n):
    logits = hard_rows(n, dtype)
    rows = len(logits)
    k = min(n, 6)
    at = torch.tensor([0, n // 3, n // 2, n - 1, 1 % n, 2 % n][:k])
    ids = at.to(torch.int32).expand(rows, k).contiguous().cuda()
    values = torch.log_softmax(randn(rows, 8, seed=4), 1)[:, :k].float().cuda()
    for t in (1.0, 0.0, INF, 0.25, 1e-20):
        check_distill(ctx, logits, ids, values, t=t, rest=rest)


def test_distill_of_far_masses(ctx):
    """A row of which the listed tokens hold all but e^-200: the unlisted ones' share among themselves stays."""
    n = 700
    logits = randn(4, n, seed=51)
    ids = torch.tensor([[5, 9]] * 4, dtype=torch.int32).cuda()
    logits[:, 5], logits[:, 9] = 200.0, 199.0
    values = torch.tensor([[0.5, 0.25]] * 4).log().cuda()
    for dtype in (F32, BF16):
        check_distill(ctx, logits.to(dtype).cuda(), ids, values, rest=True)


@pytest.mark.parametrize("n,k", [(300, 1), (5000, 3), (70000, 40)])
def test_a_small_divergence_keeps_its_digits(ctx, n, k):
    """Teacher and student that differ by a hundredth: the divergence is some 10^-5, far less than its terms."""
    logits = some_logits(40, n, F32, seed=55)
    t = logits.cpu().double() + 0.01 * randn(40, n, seed=56)
    top = torch.log_softmax(t, 1).topk(k, dim=1)
    ids, values = top.indices, top.values.float()
    loss, _ = ctx.head_distill(logits, ids.to(torch.int32).cuda(), values.cuda(), rest=True)
    _, z, p, log_s, _ = softmax64(logits)
    lp, lq = (z - log_s[:, None]).gather(1, ids), values.double()
    q, pk = lq.exp(), lp.exp()
    q_rest, left = 1 - q.sum(1), torch.ones(40, n, dtype=torch.bool).scatter_(1, ids, False)
    p_rest = torch.where(left, p, 0.0).sum(1)

    def term(q, p):
        return q * (q / p).log() - q + p

    want = term(q, pk).sum(1) + term(q_rest, p_rest)
    # q h(d) changes by (p - q) for a change of d, of which the roundings of log p are room's and a few of its own; q_rest is off
    # by the roundings of the q and their sum, and h by a few of its own
    e = U * (room(z, p, log_s) + 8 * z.gather(1, ids).abs().amax(1) + 4 * p_rest.log().abs() + 4 * lq.abs().amax(1) + n / 256 + 60)
    off = ((pk - q).abs().sum(1) + (p_rest - q_rest).abs()) * e + U * (2 * lq.abs().amax(1) + 30) * (p_rest / q_rest - 1).abs() + 32 * U * want + e * e
    near(loss, want, off)
    assert ((off < 0.1 * want).float().mean() > 0.8).item(), (off / want).quantile(0.8)   # the bound says something


@pytest.mark.parametrize("rest", [False, True])
def test_distill_against_differences(ctx, rest):
    n, rows, k = 31, 3, 4
    logits = some_logits(rows, n, F32, seed=61)
    ids, values = some_teacher(logits, k, seed=62)
    _, d = ctx.head_distill(logits, ids, values, temperature=0.7, rest=rest, grad=2.0)
    q = values.cpu().double().exp() if rest else torch.softmax(values.cpu().double(), 1)
    i = ids.cpu().long()

    def value(v):   # 64 bits
        lp = torch.log_softmax(v / float(np.float32(0.7)), 1)
        loss = (q * (q.log() - lp.gather(1, i))).sum(1)
        if rest:
            left = torch.ones(rows, n, dtype=torch.bool).scatter_(1, i, False)
            qr = 1 - q.sum(1)
            loss = loss + qr * (qr.log() - torch.logsumexp(torch.where(left, lp, -INF), 1))
        return 2.0 * loss

    v, step = logits.cpu().double(), 1e-4
    for j in range(n):
        e = torch.zeros(rows, n, dtype=torch.float64)
        e[:, j] = step
        near(d.cpu().double()[:, j], (value(v + e) - value(v - e)) / (2 * step), 1e-4 + 30 * 3 * step ** 2)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rest", [False, True])
def test_distill_of_views_and_in_place(ctx, dtype, rest):
    for rows, n, pad in [(3, 1000, 1), (5, 333, 3), (2, 4096, 8), (4, 4096, 5), (2, 30001, 7)]:
        big = some_logits(rows, n + pad, dtype, seed=n)
        for x in (big[:, pad:], big[:, :n]):
            ids, values = some_teacher(x, 9)
            loss, plain = check_distill(ctx, x, ids, values, rest=rest, g=torch.full((rows,), 0.25).cuda())
            assert torch.equal(ctx.head_distill(x, ids, values, rest=rest, grad=0.25)[1], plain)
            for shift in (0, 1, 3):
                frame = torch.full((rows, n + 9), -7.0, dtype=dtype, device="cuda")
                d = ctx.head_distill(x, ids, values, rest=rest, grad=0.25, out=frame[:, shift:shift + n])[1]
                assert torch.equal(d, plain)
                assert (frame[:, :shift] == -7).all() and (frame[:, shift + n:] == -7).all()
            both = big.clone()
            y = both[:, pad:] if x.data_ptr() != big.data_ptr() else both[:, :n]
            l2, d2 = ctx.head_distill(y, ids, values, rest=rest, grad=0.25, out=y)
            assert torch.equal(y, plain) and torch.equal(l2, loss) and d2.data_ptr() == y.data_ptr()
            edge, kept = (both[:, :pad], big[:, :pad]) if x.data_ptr() != big.data_ptr() else (both[:, n:], big[:, n:])
            assert torch.equal(edge, kept)
            # lists that are columns of wider ones are copied
            wide = torch.cat([ids, ids], 1)[:, :9]
            assert torch.equal(ctx.head_distill(x, wide, values, rest=rest)[0], loss)


@pytest.mark.parametrize("n", [600_011, 1 << 22])
def test_the_largest_vocabularies(ctx, n):
    logits = some_logits(2, n, F16, seed=71)
    ids, a = some_ids(2, n), randn(2, seed=72).float().cuda()
    norm = check_logprobs(ctx, logits, ids, top=128)[4]
    rounded(ctx.head_logprobs_backward(logits, ids, norm, a), *grad64(logits, ids, a, None), F16)
    tids, values = some_teacher(logits, 100)
    for rest in (False, True):
        check_distill(ctx, logits, tids, values, rest=rest)


# ------------------------------------------------------- every kind of launch ---
# A row has a warp, 64 to 512 threads or a cluster, and a gradient's row stays in shared memory or is read again, by numbers
# of rows and sizes: a few rows of each are checked, and all of them by a second call on the rows in another order, which no
# row's result may depend on (where rows start anywhere, in the same order: a row's sums go by its first byte's place).

LAUNCHES = [(1300, 7), (1300, 264), (1300, 1001), (1301, 4352), (800, 9000), (2500, 9001), (400, 17000), (1100, 33000), (100, 70001),
            (310, 66000), (160, 131080), (20, 250000)]


def another_order(rows, n):
    return (torch.randperm(rows, generator=torch.Generator().manual_seed(0)) if n % 8 == 0 else torch.arange(rows)).cuda()


def launch_logits(rows, n, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + n)
    x = 2 * torch.randn(rows, n, generator=g, device="cuda")
    at = torch.randint(0, n, (rows, 25), generator=g, device="cuda")
    x.scatter_(1, at, 8 + 3 * torch.randn(rows, 25, generator=g, device="cuda"))
    x[3] = -INF                       # rows for the general forms among the others
    x[5, : n // 2] = torch.finfo(dtype).min
    x[6] = 0.5
    x[7, 0] = INF
    x[8, 1:] = NAN
    return x.to(dtype), torch.tensor(sorted({0, 1, 3, 5, 6, 7, 8, rows // 2, rows - 2, rows - 1}))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", LAUNCHES)
def test_logprobs_of_every_launch(ctx, dtype, rows, n):
    x, some = launch_logits(rows, n, dtype)
    ids = some_ids(rows, n)
    a, order = randn(rows, seed=1).float().cuda(), another_order(rows, n)
    for top in (0, 5, 21, 40, 64, 128):
        out = ctx.head_logprobs(x, ids, temperature=0.8, top=top)

        class Some:   # the rows to be checked, as check_logprobs asks for them
            @staticmethod
            def head_logprobs(*_, **__):
                return tuple(o if o is None else o[some.cuda()] for o in out)

        check_logprobs(Some, x[some.cuda()], ids[some.cuda()], t=0.8, top=top)
        again = ctx.head_logprobs(x[order], ids[order], temperature=0.8, top=top)
        for one, two in zip(out, again):
            assert (one is None and two is None) or torch.equal(one[order], two)
    _, h, _, _, norm = out
    for b in (None, a):
        d = ctx.head_logprobs_backward(x, ids, norm, a, h if b is not None else None, b, temperature=0.8)
        at = some.cuda()
        want, off = grad64(x[at], ids[at], a[at], a[at] if b is not None else None, 0.8)
        rounded(d[at], want, off, dtype)
        args = (norm[order], a[order], h[order] if b is not None else None, b[order] if b is not None else None)
        assert torch.equal(d[order], ctx.head_logprobs_backward(x[order], ids[order], *args, temperature=0.8))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", LAUNCHES)
@pytest.mark.parametrize("rest", [False, True])
def test_distill_of_every_launch(ctx, dtype, rows, n, rest):
    x, some = launch_logits(rows, n, dtype)
    k = min(n, 50)
    t = x.float().nan_to_num(-1e4, 1e4, -1e4) + torch.randn(rows, n, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    top = torch.log_softmax(t.clamp_min(-1e4), 1).topk(k, dim=1)
    ids, values = top.indices.to(torch.int32), top.values
    ids[0, : k // 2] = -1
    if k > 2:
        ids[rows - 1, 2] = ids[rows - 1, 0]
    g, order = (0.5 + torch.rand(rows, generator=torch.Generator().manual_seed(3))).cuda(), another_order(rows, n)
    at = some.cuda()
    loss, _ = ctx.head_distill(x, ids, values, temperature=0.8, rest=rest)
    loss2, d = ctx.head_distill(x, ids, values, temperature=0.8, rest=rest, grad=g)
    want, off, dwant, doff = distill64(x[at], ids[at], values[at], 0.8, rest, g[at])
    near(loss[at], want, off)
    near(loss2[at], want, off)
    rounded(d[at], dwant, doff, dtype)
    again, e = ctx.head_distill(x[order], ids[order], values[order], temperature=0.8, rest=rest, grad=g[order])
    assert torch.equal(loss2[order], again) and torch.equal(d[order], e)
    assert torch.equal(loss[order], ctx.head_distill(x[order], ids[order], values[order], temperature=0.8, rest=rest)[0])
    assert torch.equal(ctx.head_distill(x, ids, values, temperature=0.8, rest=rest, grad=g, out=x)[1], d) and torch.equal(x, d)


# ------------------------------------------------------- streams and graphs ---

def test_other_streams_and_captured_graphs(ctx):
    """Two graphs that hold every call, replayed on new inputs from two streams at once, and eager calls between them."""
    rows, n = 64, 5001
    g = torch.Generator(device="cuda").manual_seed(0)

    def build(seed):
        x = some_logits(rows, n, BF16, seed=seed)
        ids = some_ids(rows, n, seed)
        tids, values = some_teacher(x, 16, seed)
        a = randn(rows, seed=seed).float().cuda()

        def step():
            lp, h, ti, tl, norm = ctx.head_logprobs(x, ids, top=12, temperature=0.9)
            d = ctx.head_logprobs_backward(x, ids, norm, a, h, a, temperature=0.9)
            loss, e = ctx.head_distill(x, tids, values, rest=True, grad=a)
            return lp, h, ti, tl, norm, d, loss, e

        return x, step

    made = [build(s) for s in (1, 2)]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, step in made:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for turn in range(3):
        for x, _ in made:
            x.copy_((2 * torch.randn(rows, n, device="cuda", generator=g)).to(BF16))
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (x, step), out, s in zip(made, outs, streams):
            with torch.cuda.stream(s):
                again = step()
            s.synchronize()
            for one, two in zip(out, again):
                assert torch.equal(one, two)


def test_equal_calls_give_equal_results(ctx):
    logits = some_logits(33, 40000, BF16)
    ids = some_ids(33, 40000)
    tids, values = some_teacher(logits, 50)
    first = [*ctx.head_logprobs(logits, ids, top=64), *ctx.head_distill(logits, tids, values, rest=True, grad=1.0)]
    for _ in range(5):
        again = [*ctx.head_logprobs(logits, ids, top=64), *ctx.head_distill(logits, tids, values, rest=True, grad=1.0)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------ refusals ---

def test_refusals(ctx):
    from bpe_trie_encode_gb300 import BpeError
    x, ids = some_logits(4, 100, F32), some_ids(4, 100)
    tids, values = some_teacher(x, 5)
    norm = ctx.head_logprobs(x, ids)[4]
    a = torch.ones(4, device="cuda")
    lp, bad = ctx.head_logprobs, pytest.raises
    with bad(TypeError):
        lp(x.double(), ids)
    with bad(TypeError):
        lp(x, ids.long())
    with bad(TypeError):
        lp(x.cpu(), ids)
    with bad(ValueError):
        lp(x, ids[:3])
    for top in (-1, 129):
        with bad(ValueError):
            lp(x, ids, top=top)
    with bad(ValueError):
        lp(x, logprob=a)
    with bad(ValueError):
        lp(x, ids, top_ids=tids)
    with bad(ValueError):
        lp(x, ids, top=4, top_ids=tids)
    with bad(ValueError):
        lp(x, ids, norm=norm.t().contiguous().t())
    with bad(BpeError, match="tokens"):
        lp(x[:, :0], ids)
    back = ctx.head_logprobs_backward
    with bad(ValueError):
        back(x, None, norm, a)
    with bad(ValueError):
        back(x, ids, norm, a, None, a)
    with bad(ValueError):
        back(x, ids, norm[:3], a)
    with bad(TypeError):
        back(x, ids, norm, a, out=x.half())
    with bad(ValueError):
        back(x, ids, norm, a, out=x.t().contiguous().t())
    with bad(BpeError, match="overlaps"):
        back(x[:, :50], ids, norm, a, out=x[:, 49:99])
    with bad(BpeError, match="overlaps"):
        back(x.view(-1)[:300].view(4, 75), ids, norm, a, out=x.view(-1)[100:].view(4, 75))
    dist = ctx.head_distill
    with bad(ValueError):
        dist(x, tids, values[:, :4])
    with bad(TypeError):
        dist(x, tids.long(), values)
    with bad(TypeError):
        dist(x, tids, values.double())
    with bad(ValueError):
        dist(x, tids[:, :0], values[:, :0])
    with bad(ValueError):
        dist(x, tids.repeat(1, 26), values.repeat(1, 26))
    with bad(ValueError):
        dist(x, tids, values, out=x)
    with bad(ValueError):
        dist(x, tids, values, grad=a[:2])
    with bad(BpeError, match="overlaps"):
        dist(x[:, :50], tids, values, grad=1.0, out=x[:, 10:60])
    # nothing to do
    assert lp(x[:0], ids[:0])[1].shape == (0,)
    assert back(x[:0], ids[:0], norm[:0], a[:0]).shape == (0, 100)
    assert dist(x[:0], tids[:0], values[:0], grad=1.0)[1].shape == (0, 100)


# ----------------------------------------------------------- one after another ---

def test_a_step_of_distillation(ctx):
    """A teacher's logits by the 8-bit product, its alternatives, a student's loss and gradient, and the weights' gradient."""
    rows, dim, n, k = 96, 256, 1111, 40
    hidden, teacher = randn(rows, dim, seed=81).float().cuda(), randn(n, dim, seed=82).float().cuda() / 4
    x8, xs, _ = ctx.head_norm(hidden, torch.ones(dim, device="cuda"))
    logits = ctx.head_logits(x8, xs, *ctx.head_quantize(teacher))
    _, _, tids, values, _ = ctx.head_logprobs(logits, top=k)
    student = (randn(n, dim, seed=83).float().cuda() / 16).requires_grad_()
    out = hidden @ student.t()
    loss, d = ctx.head_distill(out.detach(), tids, values, rest=True, grad=1.0 / rows)
    out.backward(d)
    # the formula in 64 bits, through autograd, from the same 32-bit logits
    v = out.detach().cpu().double().requires_grad_()
    lp = torch.log_softmax(v, 1)
    q, i = values.cpu().double().exp(), tids.cpu().long()
    left = torch.ones(rows, n, dtype=torch.bool).scatter_(1, i, False)
    q_rest = 1 - q.sum(1)
    want = (q * (q.log() - lp.gather(1, i))).sum(1) + q_rest * (q_rest.log() - torch.logsumexp(lp.masked_fill(~left, -INF), 1))
    (want.sum() / rows).backward()
    near(loss, want.detach(), 1e-4)
    near(d, v.grad, 1e-5 / rows)
    weight = v.grad.t() @ hidden.cpu().double()
    near(student.grad, weight, 1e-4 / rows * math.sqrt(rows) * 10)
    # the same entry points score the student's own tokens
    lp2, h, _, _, norm = ctx.head_logprobs(out.detach(), tids[:, 0].contiguous())
    near(lp2, lp.detach().gather(1, i[:, :1])[:, 0], 1e-5)
    d = ctx.head_logprobs_backward(out.detach(), tids[:, 0].contiguous(), norm, torch.full((rows,), -1.0, device="cuda"))
    one, e = ctx.head_distill(out.detach(), tids[:, :1], values[:, :1], grad=1.0)   # cross entropy of the first
    near(one, -lp2.cpu(), 1e-5)
    near(d, e.cpu(), 1e-6)
