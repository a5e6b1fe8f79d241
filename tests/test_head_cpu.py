"""The output head's entry points without a GPU: refusals at the C ABI, and the header's limits."""
import os
import re

from bpe_trie_encode_gb300 import _capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_null_context_is_refused():
    lib = _capi.load()
    assert lib.head_norm(None, None, 0, 0, None, 0, None, 0, 1, 128, 1e-6, None, 0, None, 0, None, 0, 0) == -1
    assert lib.head_quantize(None, None, 0, 0, 1, 128, None, 0, None, 0) == -1
    assert lib.head_logits(None, None, 0, None, 0, 0, None, 0, None, 0, 0, 1, 1, 128, None, 0, 0) == -1
    assert lib.head_sample(None, None, 0, 0, 1, 1, None, None, None, None) == -1


def test_binding_repeats_the_header():
    txt = open(os.path.join(ROOT, "include", "bpetrie.h")).read()
    assert f"BPE_HEAD_BLOCK {_capi.BPE_HEAD_BLOCK}u" in txt
    assert f"BPE_HEAD_MAX_DIM {_capi.BPE_HEAD_MAX_DIM}u" in txt
    assert _capi.BPE_HEAD_MAX_TOKENS == 1 << 22 and "BPE_HEAD_MAX_TOKENS (1u << 22)" in txt
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} head_filters;", txt).group(1)
    fields = re.findall(r"(\w+);", body)
    assert fields == [f[0] for f in _capi.head_filters._fields_]
