"""Threads that share a context, each on a stream of its own."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_threads_share_a_context():
    """Each call reads what its own stream has just written, behind work that takes longer than the call's way to the device."""
    import bpe_trie_encode_gb300 as bt
    ctx, rows, n, wrong = bt.Context(0), 16, 4096, []

    def work(seed):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            g = torch.Generator(device="cuda").manual_seed(seed)
            ids = torch.arange(rows, dtype=torch.int32, device="cuda") * 200 + seed
            big = torch.ones(4 << 20, device="cuda")
            for _ in range(60):
                x = torch.randn(rows, n, generator=g, device="cuda")
                for _ in range(4):
                    big.mul_(1.0)
                x += 0 * big[0]
                x.mul_(2.0)
                lp, _, top, _, norm = ctx.head_logprobs(x, ids, top=3)
                d = ctx.head_logprobs_backward(x, ids, norm, torch.ones(rows, device="cuda"))
                want = torch.log_softmax(x.double(), 1)
                grad = torch.nn.functional.one_hot(ids.long(), n) - want.exp()
                ok = ((lp - want.gather(1, ids.long()[:, None])[:, 0]).abs() < 1e-4).all() & ((d - grad).abs() < 1e-5).all() \
                    & (top[:, 0] == x.argmax(1)).all()
                stream.synchronize()
                if not ok.item():
                    wrong.append(seed)

    threads = [threading.Thread(target=work, args=(s,)) for s in range(1, 4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    ctx.close()
