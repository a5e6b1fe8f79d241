"""How a Context hands its stream to the library, with a library that only notes what it is told: no GPU."""
import ctypes
import sys
import threading
import time

import pytest

torch = pytest.importorskip("torch")

import bpe_trie_encode_gb300 as bt  # noqa: E402

HERE = threading.local()   # the current stream of a thread


class Library:
    """The stream that the library has, and for every call the caller's and the one that it ran on."""

    def __init__(self):
        self.word, self.ran = ctypes.c_size_t(0), []

    @property
    def stream(self):
        return self.word.value

    def bpe_ctx_stream(self, handle):
        return ctypes.addressof(self.word)

    def bpe_ctx_set_stream(self, handle, stream):
        time.sleep(1e-5)   # other threads run, as while ctypes is in a call
        self.word.value = int(getattr(stream, "value", stream) or 0)
        time.sleep(1e-5)
        return 0

    def __getattr__(self, name):
        if not name.startswith("head_"):
            raise AttributeError(name)

        def call(*_):
            time.sleep(1e-5)
            self.ran.append((name, HERE.stream, self.stream))
            return 0

        return call


@pytest.fixture
def ctx(monkeypatch):
    monkeypatch.setattr(bt, "_raw_stream", lambda index: HERE.stream)
    monkeypatch.setattr(bt.torch.cuda, "is_available", lambda: True)
    made = Library()
    made.bpe_ctx_create = lambda *_: 0
    made.bpe_ctx_destroy = lambda *_: None
    monkeypatch.setattr(bt._capi, "load", lambda: made)
    HERE.stream = 5
    ctx = bt.Context(0)
    ctx.device = torch.device("cpu")
    made.word.value = 5
    return ctx


def every_call(ctx):
    x, ids, one = torch.zeros(2, 16), torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    norm = ctx.head_logprobs(x, ids)[4]
    ctx.head_logprobs_backward(x, ids, norm, one)
    ctx.head_distill(x, ids[:, None], one[:, None], grad=1.0)
    ctx.head_sample(x, one)


def test_a_stream_set_on_the_handle_does_not_last(ctx):
    every_call(ctx)
    ctx.lib.bpe_ctx_set_stream(ctx._h, 9)   # by other means than the binding's
    every_call(ctx)
    HERE.stream = 6
    every_call(ctx)
    assert len(ctx.lib.ran) == 12 and all(mine == its for _, mine, its in ctx.lib.ran), ctx.lib.ran


def test_threads_run_on_their_own_streams(ctx):
    def work(stream):
        HERE.stream = stream
        for _ in range(40):
            every_call(ctx)

    often, threads = sys.getswitchinterval(), [threading.Thread(target=work, args=(s,)) for s in (11, 12, 13, 14)]
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(often)
    wrong = [r for r in ctx.lib.ran if r[1] != r[2]]
    assert len(ctx.lib.ran) == 4 * 40 * 4 and not wrong, (len(wrong), wrong[:3])


def test_an_error_leaves_the_context_usable(ctx):
    ctx.lib.head_sample = lambda *_: -1
    ctx.lib.bpe_last_error = lambda *_: b"refused"
    with pytest.raises(bt.BpeError, match="refused"):
        ctx.head_sample(torch.zeros(2, 16), torch.zeros(2))
    ctx.head_logprobs(torch.zeros(2, 16))
    assert ctx.lib.ran == [("head_logprobs", 5, 5)]


def test_where_the_stream_is_kept():
    lib = bt._capi.load()
    assert lib.bpe_ctx_stream(None) is None


def test_a_call_within_a_call_of_the_same_thread(ctx):
    """As a signal handler makes one."""
    def handled(handle, stream):
        ctx.lib.word.value = stream
        del ctx.lib.bpe_ctx_set_stream
        ctx.head_sample(torch.zeros(2, 16), torch.zeros(2))
        return 0

    ctx.lib.bpe_ctx_set_stream = handled
    HERE.stream = 8
    done = []

    def work():
        HERE.stream = 8
        ctx.head_logprobs(torch.zeros(2, 16))
        done.append(ctx.lib.ran)

    t = threading.Thread(target=work, daemon=True)
    t.start()
    t.join(10)
    assert done == [[("head_sample", 8, 8), ("head_logprobs", 8, 8)]]
