"""The output head's scoring and distillation without a GPU: refusals at the C ABI and the binding's checks."""
import os

import pytest

from bpe_trie_encode_gb300 import _capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_null_context_is_refused():
    lib = _capi.load()
    assert lib.head_logprobs(None, None, 0, 0, 1, 1, None, 1.0, None, 0, None, None, None, None, None) == -1
    assert lib.head_logprobs_backward(None, None, 0, 0, 1, 1, None, 1.0, None, None, None, None, None, None, 0) == -1
    assert lib.head_distill(None, None, 0, 0, 1, 1, None, None, 0, 1, 0, 1.0, None, None, 0.0, None, None, 0) == -1


def test_binding_repeats_the_header():
    txt = open(os.path.join(ROOT, "include", "bpetrie.h")).read()
    assert f"BPE_HEAD_MAX_TOP {_capi.BPE_HEAD_MAX_TOP}u" in txt


def test_tables():
    torch = pytest.importorskip("torch")
    import bpe_trie_encode_gb300 as bt
    cpu = torch.device("cpu")
    t = torch.zeros(4, 6)
    assert bt._head_table(t, "x", cpu, (torch.float32,), 4) is t
    assert bt._head_table(t[:, :3], "x", cpu, (torch.float32,), 4, 3).is_contiguous()
    with pytest.raises(ValueError, match="contiguous"):
        bt._head_table(t[:, :3], "x", cpu, (torch.float32,), 4, 3, out=True)
    for rows, columns in ((3, None), (4, 5)):
        with pytest.raises(ValueError, match="must be"):
            bt._head_table(t, "x", cpu, (torch.float32,), rows, columns)
    with pytest.raises(TypeError):
        bt._head_table(t, "x", cpu, (torch.int32,), 4)
    with pytest.raises(TypeError):
        bt._head_table([1], "x", cpu, (torch.int32,), 1)


def test_numbers():
    torch = pytest.importorskip("torch")
    import bpe_trie_encode_gb300 as bt
    cpu = torch.device("cpu")
    assert bt._head_number(0.5, "t", cpu, 3) == (0.5, None, None)
    some = torch.ones(6)[::2]
    number, kept, at = bt._head_number(some, "t", cpu, 3)
    assert number == 1.0 and kept.is_contiguous() and at == kept.data_ptr()
    with pytest.raises(ValueError):
        bt._head_number(some, "t", cpu, 4)
