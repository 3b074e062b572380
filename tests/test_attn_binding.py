"""The exact-attention calls' binding, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import sparse_exact_kv_gb300 as lib
    return lib


def test_selftest_blocks_outside_the_range_are_refused(L):
    assert L._lib.lola_selftest_attn_wait(-2) == L.LOLA_ERR_INVALID_ARG
    with pytest.raises(L.LolaError):
        L.lola_selftest_attn_wait(-2)


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


def test_pools_that_do_not_fit_the_layer_are_refused(L, monkeypatch):
    """Pools put in place of a layer's own are looked at in every call."""
    import torch
    bf = torch.bfloat16
    monkeypatch.setattr(L, "_index_of", lambda dev: 0)
    lay = L.ExactAttention(4, 2, 64, bf, torch.zeros(4, 2, 16, 64, dtype=bf), torch.zeros(4, 2, 16, 64, dtype=bf))
    lens, table = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    pool = torch.zeros(6, 2, 16, 64, dtype=bf)
    lay.k_pool, lay.v_pool = pool, pool.clone()               # another cache of the same layer: taken
    assert lay._cache(lens, table)[0].n_pages == 6
    bad = [torch.zeros(4, 2, 16, 64, dtype=bf), torch.zeros(6, 1, 16, 64, dtype=bf), torch.zeros(6, 2, 16, 128, dtype=bf),
           torch.zeros(6, 2, 32, 64, dtype=bf), torch.zeros(6, 2, 16, 64), torch.zeros(6, 16, 2, 64, dtype=bf).transpose(1, 2),
           torch.zeros(12, 16, 64, dtype=bf), None]
    for other in bad:
        for k, v in ((pool, other), (other, pool)):
            lay.k_pool, lay.v_pool = k, v
            with pytest.raises(ValueError):
                lay._cache(lens, table)
    for other in bad[1:3] + bad[4:7]:
        lay.k_pool = lay.v_pool = other
        with pytest.raises(ValueError):
            lay._cache(lens, table)


def test_calls_decline_without_the_marshalling_module(L, tmp_path):
    """A module that is not there, or does not load, leaves the Python form of every call."""
    broken = tmp_path / "_lola_py-broken.so"
    broken.write_bytes(b"no module")
    for path in (str(tmp_path / "none.so"), str(broken)):
        fast = L._marshalling(path)
        for call in (fast.prefill, fast.prefill_paged, fast.decode, fast.append):
            assert call(1, None, "anything") is NotImplemented
    assert L._marshalling(L._PYMOD).decode() is NotImplemented         # the real one: wrong arguments, declined
    assert type(L._fast).__name__ == "module"


def test_the_package_does_not_need_the_marshalling_module(L):
    """Under another torch than the module was compiled against the package loads, and says so where it matters."""
    import subprocess
    import sys
    code = """
import warnings, torch
torch.__version__ = "0.0.0+other"
import sparse_exact_kv_gb300 as L
assert L.lola_check_config(L.make_config(1, 1, 64, 64, 64, 16, 16, 64, "bf16")) == 0
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    L.ExactAttention(4, 2, 64)
assert any("marshalling" in str(x.message) for x in w), w
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=_root())
    assert r.returncode == 0, r.stderr


def test_another_torch_makes_the_build_stale(L, monkeypatch):
    import __graft_entry__
    import torch
    build = __graft_entry__._build_module()
    assert not build._stale()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert build._stale()


def _root():
    import os
    return os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
