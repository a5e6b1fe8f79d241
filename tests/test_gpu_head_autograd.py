"""Gradients that overwrite logits which autograd may have kept."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import bpe_trie_encode_gb300 as bt
    c = bt.Context(0)
    yield c
    c.close()


def calls(ctx, rows):
    ids, one = torch.arange(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, 1, device="cuda")

    def scored(x, out):
        norm = ctx.head_logprobs(x, ids)[4]
        return ctx.head_logprobs_backward(x, ids, norm, torch.full((rows,), -1.0, device="cuda"), out=out)

    return scored, lambda x, out: ctx.head_distill(x, ids[:, None].contiguous(), one, grad=1.0, out=out)[1]


@pytest.mark.parametrize("which", [0, 1])
def test_kept_logits_that_are_overwritten_are_an_error(ctx, which):
    """log_softmax keeps what it returns: its backward pass on a gradient in that place would be wrong without a word."""
    rows, n = 4, 300
    call = calls(ctx, rows)[which]
    w = torch.randn(rows, n, generator=torch.Generator().manual_seed(0)).cuda().requires_grad_()
    logits = torch.log_softmax(w, 1)
    d = call(logits.detach(), None)
    logits.backward(d)
    plain = w.grad.clone()
    assert (plain - (torch.softmax(w, 1) - torch.eye(rows, n, device="cuda")).detach()).abs().max() < 1e-5
    logits = torch.log_softmax(w, 1)
    d = call(logits.detach(), logits.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        logits.backward(d)


@pytest.mark.parametrize("which", [0, 1])
def test_logits_that_nothing_keeps_may_be_overwritten(ctx, which):
    rows, n, dim = 4, 300, 16
    call = calls(ctx, rows)[which]
    g = torch.Generator().manual_seed(1)
    hidden, weight = torch.randn(rows, dim, generator=g).cuda(), torch.randn(n, dim, generator=g).cuda().requires_grad_()
    grads = []
    for in_place in (False, True):
        logits = hidden @ weight.t()
        d = call(logits.detach(), logits.detach() if in_place else None)
        logits.backward(d)
        grads.append(weight.grad)
        weight.grad = None
    assert torch.equal(*grads)
    with torch.inference_mode():
        logits = hidden @ weight.t()
        assert call(logits, logits).data_ptr() == logits.data_ptr()
    graph = torch.cuda.CUDAGraph()
    kept = (hidden @ weight.t()).detach()
    logits = kept.clone()
    call(logits, logits)   # once before the capture
    want = logits.clone()
    logits.copy_(kept)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(logits, logits)
    graph.replay()
    assert torch.equal(logits, want)
