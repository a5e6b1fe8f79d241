"""The output head's checks that need no GPU: refusals at the C ABI and the binding's limits."""
import pytest

from bpe_trie_encode_gb300 import _capi


def test_check_of_a_null_context_is_refused():
    assert _capi.load().head_check(None) == -1


@pytest.mark.parametrize("size", [(2 ** 31, 1), (2 ** 32 + 5, 1), (1, 2 ** 31), (3, 2 ** 32 + 128)])
def test_sizes_beyond_the_librarys_are_refused(size):
    """They would be cut to 32 bits: 5 rows of 2^32 + 5 written and the rest left as it was."""
    torch = pytest.importorskip("torch")
    import bpe_trie_encode_gb300 as bt
    cpu = torch.device("cpu")
    many = torch.zeros(1, 1).expand(*size)   # takes no memory
    for out in (False, True):
        with pytest.raises(ValueError, match="above"):
            bt._head_matrix(many, "x", cpu, (torch.float32,), out=out)
    some = torch.zeros(3, 4)
    assert bt._head_matrix(some, "x", cpu, (torch.float32,)) == (some, 4)


def test_top_k_keeps_its_meaning_in_32_bits():
    import bpe_trie_encode_gb300 as bt
    for k, want in ((5, 5), (0, 0), (-1, -1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 1, 2 ** 31 - 1),
                    (-2 ** 32 + 7, -1), (True, 1)):
        k32 = _capi.head_filters(1.0, bt._head_count(k), 1.0, 0.0, None, None, None, None).top_k
        assert k32 == want
