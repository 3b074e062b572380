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


def test_copies_of_a_layer_hold_their_own_description(L):
    """A layer copied, or pickled for another process, points at the description that it holds."""
    import copy
    import ctypes
    import pickle
    import torch
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for lay in (L.ExactAttention(4, 2, 64, scale=0.3), L.ExactAttention(4, 2, 64, torch.bfloat16, pool, pool.clone())):
        for other in (copy.copy(lay), copy.deepcopy(lay), pickle.loads(pickle.dumps(lay))):
            assert other._plan == (ctypes.addressof(other.cfg), lay._ws)
            assert bytes(other.cfg) == bytes(lay.cfg) and (other.Hq, other.Hkv, other.d, other.dtype) == (4, 2, 64, lay.dtype)
            assert (other.k_pool is None) == (lay.k_pool is None)
            if lay.k_pool is not None:
                assert torch.equal(other.k_pool, lay.k_pool) and other.v_pool.shape == lay.v_pool.shape
        assert copy.copy(lay).k_pool is lay.k_pool             # a shallow copy shares the cache


def test_a_scale_of_zero_is_refused(L):
    """It stands for 1 / sqrt(d) in the C structure; from Python that is None, and 0 would be taken for it."""
    import torch
    for make in (lambda s: L.make_attn_config(4, 2, 64, "bf16", s), lambda s: L.ExactAttention(4, 2, 64, scale=s),
                 lambda s: L.ExactAttention.allocate(4, 2, 64, 3, device="cpu", scale=s)):
        for zero in (0.0, 0, -0.0, 1e-50):
            with pytest.raises(ValueError):
                make(zero)
        make(None), make(0.25)
    assert L.make_attn_config(4, 2, 64, torch.bfloat16).scale == 0.0
