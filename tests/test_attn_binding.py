"""The exact-attention calls' binding, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import sparse_exact_kv_gb300 as lib
    return lib


def test_selftest_blocks_outside_the_range_are_refused(L):
    assert L._lib.lola_selftest_attn_wait(-2, None) == L.LOLA_ERR_INVALID_ARG
    with pytest.raises(L.LolaError):
        L.lola_selftest_attn_wait(-2, stream=0)
