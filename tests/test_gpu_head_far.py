"""Logits far from 0 and far temperatures in the scoring and training kernels, against 64 bits.

Rows are summed in powers of two relative to R, the largest logit's m c log2 e rounded once: from 2^24 of m c on R's rounding
alone is more than a step of the exponent, so that tiles, warps and CTAs of masked logits, and whole rows, must not go by it.
Bounds are those of test_gpu_head_score, with the depth of a warp's sums: a lane adds 1 / 64 of a row's terms to each half of a
pair.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_head_score as base                                                                              # noqa: E402
from test_gpu_head_score import BF16, F16, F32, INF, check_distill, check_logprobs, ctx, grad64, randn, rounded  # noqa: E402, F401


@pytest.fixture(autouse=True)
def room_of_warps(monkeypatch):
    """`room` with n / 64, and what distill64 adds of its own (n / 256 twice) made up for."""
    monkeypatch.setattr(base, "room", lambda z, p, log_s: 8 * base.mean_of(p, z.abs()) + 2 * log_s.abs() + z.shape[1] / 32 + 40)


def some_ids(logits):
    """The largest logit of some rows, any token of others, none of every seventh."""
    rows, n = logits.shape
    ids = torch.where(torch.arange(rows) % 2 == 0, logits.cpu().double().nan_to_num(-INF).argmax(1), torch.arange(rows) * 37 % n)
    ids[6::7] = -1
    return ids.to(torch.int32).cuda()


def check_all(ctx, logits, t, tops=(0, 5, 40), listed=6, teacher=None, check=None):
    """Every call on these rows; weights of gradients are in proportion to the temperature.  `check`: the rows to be compared."""
    rows, n = logits.shape
    at = torch.arange(rows) if check is None else check
    some = at.cuda()
    x, ids, t_some = logits[some], some_ids(logits), t[some]

    def part(o):
        return o if o is None else o[some]

    class Rows:   # the whole batch is computed, some of its rows are compared
        @staticmethod
        def head_logprobs(*_, top, **__):
            return tuple(part(o) for o in ctx.head_logprobs(logits, ids, temperature=t, top=top))

        @staticmethod
        def head_distill(*_, rest, grad=None, **__):
            return tuple(part(o) for o in ctx.head_distill(logits, tids, values, temperature=t, rest=rest, grad=None if grad is None else g))

    for top in tops:
        check_logprobs(Rows, x, ids[some], t=t_some, top=top)
    _, h, _, _, norm = ctx.head_logprobs(logits, ids, temperature=t)
    a, b = (randn(rows, seed=3).float().cuda() * t).contiguous(), (randn(rows, seed=4).float().cuda() * t).contiguous()
    for e in (None, b):
        d = ctx.head_logprobs_backward(logits, ids, norm, a, None if e is None else h, e, temperature=t)
        want, off = grad64(x, ids[some], a[some], part(e), t_some)
        rounded(d[some], want, off, logits.dtype)
    k = min(listed, n)
    if teacher is None:
        order = torch.sort(logits.float().nan_to_num(-INF), dim=1, descending=True, stable=True).indices[:, :k]
    else:
        order = teacher
    tids = order.to(torch.int32).contiguous()
    values = torch.log_softmax(randn(rows, k + 1, seed=5), 1)[:, :k].float().contiguous().cuda()
    g = ((0.5 + torch.rand(rows, generator=torch.Generator().manual_seed(9))).cuda() * t).contiguous()
    for rest in (False, True):
        check_distill(Rows, x, tids[some], values[some], t=t_some, rest=rest, g=g[some])


# ------------------------------------------------ masked parts of ordinary rows ---

def masked_parts(rows, n, value, dtype):
    """Ordinary rows with `value` in a part: the first half, the last, all but twelve, stretches in turn, nothing."""
    x = 2 * randn(rows, n, seed=n)
    x.scatter_(1, torch.randint(0, n, (rows, min(n, 9)), generator=torch.Generator().manual_seed(1)), 9 + 3 * randn(rows, min(n, 9), seed=2))
    j = torch.arange(n)
    masks = [j < n // 2, j >= n // 2, (j * 31 + 7) % n >= 12, j // min(1024, n // 5) % 2 == 0, j // min(2048, n // 3) % 2 == 1, j > n, j < n - 12]
    for r in range(rows):
        x[r] = torch.where(masks[r % len(masks)], value, x[r])
    return x.to(dtype).cuda()


FAR = [-1e9, -1e10, -3e11, -1e12, -1e15, -2.0 ** 59, -1e19, -INF]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,n", [(7, 300), (7, 5000), (14, 70001)])
@pytest.mark.parametrize("value", FAR)
def test_rows_with_parts_masked_far(ctx, dtype, rows, n, value):
    logits = masked_parts(rows, n, value, dtype)
    for t in (1.0, 0.1, 0.003):
        check_all(ctx, logits, torch.full((rows,), t).cuda())


@pytest.mark.parametrize("rows,n", [(7, 300), (7, 5000), (14, 70001)])
@pytest.mark.parametrize("value", [-1e4, -65504.0, -INF])
def test_half_rows_with_parts_masked_at_low_temperatures(ctx, rows, n, value):
    """In 16-bit floats -infinity counts as their lowest number in the sums: at far temperatures that is far too."""
    logits = masked_parts(rows, n, value, F16)
    for t in (0.1, 1e-4, 1e-5, 2e-6):
        check_all(ctx, logits, torch.full((rows,), t).cuda())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(1300, 1001), (1300, 2304), (800, 9000), (400, 17000)])
def test_many_rows_with_parts_masked_far(ctx, dtype, rows, n):
    """Rows of a warp, and of 64 and 128 threads; each row with its own mask value and temperature."""
    x = masked_parts(rows, n, -1.0, F32)
    kept = masked_parts(rows, n, INF, F32)
    far = torch.tensor(FAR[:5] if dtype != F16 else [-1e4, -65504.0, -3e4, -INF, -6e4])
    x = torch.where(kept == INF, far[torch.arange(rows) % 5][:, None].cuda(), x).to(dtype)
    t = torch.tensor([1.0, 0.1, 0.01] if dtype != F16 else [1.0, 1e-5, 2e-6])[torch.arange(rows) // 35 % 3].cuda()
    check_all(ctx, x, t, tops=(0, 5, 21, 64), check=torch.arange(0, rows, 1)[:105])


# ------------------------------------------------------------ rows that are far ---

def far_rows(n, dtype):
    """Rows of which all logits are far from 0, or all but one or two."""
    v = [-1e9, -1e10, -3e11, -1e12, -1e15, 1e10, 1e12, 2.0 ** 49, -2.0 ** 49] if dtype != F16 else [-16000.0, -65504.0, 65504.0, 3e4]
    x = torch.empty(2 * len(v) + 4, n, dtype=torch.float64)
    for i, one in enumerate(v):
        x[2 * i] = one
        x[2 * i + 1] = one * (1 + 2.0 ** -6 * randn(n, seed=i).abs())   # far apart, all but some
    x[-4] = 1.0
    x[-4, 0] = v[5] if dtype != F16 else 65504.0
    x[-3] = v[1]
    x[-3, n - 1] = 0.5
    x[-2] = v[3]
    x[-2, : n // 2] = v[1]
    x[-1] = 2 * randn(n, seed=99)
    big = torch.finfo(dtype).max
    return x.clamp(-big, big).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [2, 300, 5000, 70001])
@pytest.mark.parametrize("t", [1.0, 0.1, 1e-5, 2e-6])
def test_rows_far_from_0(ctx, dtype, n, t):
    logits = far_rows(n, dtype)
    check_all(ctx, logits, torch.full((len(logits),), t).cuda())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,n", [(20, 400), (20, 40000), (1300, 900)])
def test_unlisted_tokens_far_below_the_listed(ctx, dtype, rows, n):
    """Listed tokens as usual and the unlisted ones masked: the far ones among themselves decide the rest's shares."""
    value = torch.tensor([-1e9, -1e10, -1e12, -1e15])[torch.arange(rows) % 4][:, None].double()
    x = value * (1 + 2.0 ** -20 * randn(rows, n, seed=7).abs() * (torch.arange(rows) % 2)[:, None])
    listed = (torch.arange(6) * 31 + 5)[None].expand(rows, 6) % n
    x = x.scatter(1, listed, 3 * randn(rows, 6, seed=8)).to(dtype).cuda()
    t = torch.tensor([1.0, 0.5])[torch.arange(rows) // 8 % 2].cuda()
    check_all(ctx, x, t, tops=(0, 5), teacher=listed.cuda(), check=torch.arange(min(rows, 40)))


# On both sides of each number that decides between the usual form and the general one: the inverse of the temperature, the largest
# logit, and their product.
def limits(dtype):
    """(what lies at 0, how far logits spread, temperature)"""
    for e in (1 - 2.0 ** -9, 1 + 2.0 ** -9):
        yield 0.0, 2.0 ** -19, 2.0 ** -20 * e
        yield 4.0, 2.0 ** -19, 2.0 ** -20 * e
        for s in (1.0, -1.0):
            yield s * 2.0 ** 24 * e * 2.0 ** -12, 2.0 ** -4, 2.0 ** -12
            yield s * 2.0 ** 24 * e * 2.0 ** -20, 2.0 ** -18, 2.0 ** -20
            yield s * 2.0 ** 14 * e, 4.0, 1.0
        if dtype == F16:
            yield 0.0, 100.0, 64.0 * e
            yield -16384.0 * e, 30.0, 10.0
            yield 65000.0 * min(e, 1), 30.0, 60.0
        else:
            yield 0.0, 2.0 ** 41, 2.0 ** 40 * e
            for s in (1.0, -1.0):
                yield s * 2.0 ** 24 * e, 4.0, 1.0
                yield s * 2.0 ** 25 * e, 4.0, 1.0
                yield s * 2.0 ** 50 * e, 2.0 ** 33, 2.0 ** 32
                yield s * 2.0 ** 50 * e, 2.0 ** 28, 2.0 ** 26
                yield s * 2.0 ** 60 * e, 2.0 ** 41, 2.0 ** 39


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [9, 1000, 20000])
def test_both_sides_of_the_usual_form(ctx, dtype, n):
    every = list(limits(dtype))
    rows = 2 * len(every)
    x, t = torch.empty(rows, n, dtype=torch.float64), torch.empty(rows)
    for i, (at, spread, temperature) in enumerate(every):
        x[2 * i:2 * i + 2], t[2 * i:2 * i + 2] = at + spread * randn(2, n, seed=i), temperature
        if n > 4:   # half of the second one masked at the type's lowest number
            x[2 * i + 1, n // 2:] = torch.finfo(dtype).min
    check_all(ctx, x.to(dtype).cuda(), t.cuda(), tops=(0, 3))


# ------------------------------------------------------- gradients of any size ---

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(6, 300), (6, 6000), (400, 900)])
def test_masked_logits_have_no_gradient_however_large_its_weight(ctx, dtype, rows, n):
    """What is multiplied by a probability of 0 may be beyond 32 bits: the product is 0."""
    x = masked_parts(rows, n, -INF, dtype)
    x[:, 1] = torch.finfo(dtype).min
    x[:, 5] = 1.0
    gone = torch.isinf(x)
    gone[:, 1] = True
    if dtype == F16:
        gone = x < -60000
    ids = some_ids(x)
    for t, weights in ((1.0, (1.0, 2.0 ** 66, 2.0 ** 70, 2.0 ** 120, -3e38)), (2.0 ** -19, (1e-6, 2.0 ** 28, 2.0 ** 31, 2.0 ** 60, -3e38))):
        _, h, _, _, norm = ctx.head_logprobs(x, ids, temperature=t)
        for w in weights:
            w = torch.full((rows,), w).cuda()
            for a, b in ((w, None), (None, w), (w, w)):
                d = ctx.head_logprobs_backward(x, ids if a is not None else None, norm, a, None if b is None else h, b, temperature=t)
                listed = torch.zeros_like(gone).scatter_(1, ids.long().clamp_min(0)[:, None], a is not None and (ids >= 0)[:, None])
                assert (d[gone & ~listed] == 0).all(), (t, w[0])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(6, 300), (6, 6000), (400, 900)])
@pytest.mark.parametrize("rest", [False, True])
def test_masked_logits_have_no_distilled_gradient_however_large_its_weight(ctx, dtype, rows, n, rest):
    x = masked_parts(rows, n, -INF, dtype)
    x[:, 5] = 1.0
    x[:, 7] = -INF
    gone = torch.isinf(x)
    tids = torch.tensor([[5, 7, 9]], dtype=torch.int32).expand(rows, 3).contiguous().cuda()
    values = torch.tensor([[-0.5, -300.0, -2.0]]).expand(rows, 3).contiguous().cuda()   # no q is left of the masked one
    listed = torch.zeros_like(gone).scatter_(1, tids[:, ::2].long(), True)
    for t in (1.0, 2.0 ** -19, 1e-30):
        for w in (1.0, 2.0 ** 100, 2.0 ** 120, -3e38):
            d = ctx.head_distill(x, tids, values, temperature=t, rest=rest, grad=w)[1]
            assert (d[gone & ~listed] == 0).all(), (t, w)
