"""The output head's checks that need no GPU: refusals at the C ABI and the binding's limits."""
from bpe_trie_encode_gb300 import _capi


def test_check_of_a_null_context_is_refused():
    assert _capi.load().head_check(None) == -1
