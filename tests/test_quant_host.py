"""The quantised cache and shared prefixes without a GPU: refusals return before anything is enqueued, layers check
what they are given, and the plain form's rounding is the one that is promised."""
import copy
import ctypes
import math
import pickle

import pytest
import torch

from quant_parity import decode, encode

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import sparse_exact_kv_gb300 as lib
    return lib


def cfg(L, **kw):
    a = dict(Hq=8, Hkv=2, d=128, dtype="bf16", scale=None)
    a.update(kw)
    return L.make_attn_config(**a)


def rows(L, data=256, row=1024, head=128):
    return ctypes.byref(L.lola_rows(data, row, head))


def paged(L, **kw):
    a = dict(K=256, V=256, n_pages=10, page=64, n_seq=3, width=4, table_stride=4, table=256, kv_len=256)
    a.update(kw)
    return ctypes.byref(L.lola_paged_kv(*a.values()))


def scales(L, K=256, V=256):
    return ctypes.byref(L.lola_kv_scales(K, V))


def prefixes(L, **kw):
    a = dict(n=2, width=4, table_stride=4, table=256, len=256, cu=256)
    a.update(kw)
    return ctypes.byref(L.lola_prefixes(*a.values()))


def append(L, c=None, kv=None, sc=None, n=3, cu=None, k=None, v=None, q=None, qo=None, inv=256, rot=64, pairs=0):
    return L._lib.lola_quant_append(ctypes.byref(c or cfg(L)), kv or paged(L), scales(L) if sc is None else sc, n, P(cu), k or rows(L),
                                    v or rows(L), q, qo, P(inv), rot, pairs, None, None)


def read(L, c=None, kv=None, sc=None, total=10, k=None, v=None, cu=256):
    return L._lib.lola_quant_read(ctypes.byref(c or cfg(L)), kv or paged(L), scales(L) if sc is None else sc, total, k or rows(L),
                                  v or rows(L), P(cu), None)


def step(L, c=None, kv=None, sc=None, q=None, o=None, lse=None, ws=256, size=1 << 40):
    return L._lib.lola_quant_decode(ctypes.byref(c or cfg(L)), kv or paged(L), scales(L) if sc is None else sc, q or rows(L), o or rows(L),
                                    P(lse), P(ws), size, None)


def shared(L, c=None, kv=None, sc=None, px=None, q=None, o=None, lse=None, ws=256, size=1 << 40):
    return L._lib.lola_shared_decode(ctypes.byref(c or cfg(L)), kv or paged(L), sc, prefixes(L) if px is None else px, q or rows(L), o or rows(L), P(lse),
                                     P(ws), size, None)


BAD_KV = [dict(K=0), dict(V=0), dict(K=264), dict(n_pages=0), dict(n_seq=0), dict(width=0), dict(table_stride=3), dict(table=0),
          dict(kv_len=0), dict(table=258), dict(page=0)]
BAD_ROWS = [dict(data=0), dict(data=264), dict(row=0), dict(row=-1024), dict(head=0), dict(row=1028), dict(head=132), dict(row=1 << 41)]


def test_refusals(L):
    E, U = L.LOLA_ERR_INVALID_ARG, L.LOLA_ERR_UNSUPPORTED
    calls = (append, read, step, shared)
    for call in calls:
        for bad in BAD_KV:
            assert call(L, kv=paged(L, **bad)) == E, (call, bad)
        for bad in (dict(Hq=0), dict(Hq=7), dict(dtype=5), dict(scale=-1.0)):
            assert call(L, c=cfg(L, **bad)) == E, (call, bad)
        assert call(L, c=cfg(L, d=96)) == U
        for page in (1, 8, 24, 512):
            assert call(L, kv=paged(L, page=page)) == U, (call, page)
        for bad in (dict(K=0), dict(V=0), dict(K=264), dict(V=264)):
            assert call(L, sc=scales(L, **bad)) == E, (call, bad)
    for call in (append, read, step):
        assert call(L, sc=ctypes.POINTER(L.lola_kv_scales)()) == E
    for bad in BAD_ROWS:
        assert append(L, k=rows(L, **bad)) == append(L, v=rows(L, **bad)) == E, bad
        assert read(L, k=rows(L, **bad)) == read(L, v=rows(L, **bad)) == E, bad
        for call in (step, shared):
            assert call(L, q=rows(L, **bad)) == call(L, o=rows(L, **bad)) == E, (call, bad)
    assert read(L, k=rows(L, row=128)) == E                       # rows that overlap
    assert read(L, total=-1) == read(L, cu=0) == read(L, cu=258) == E
    assert append(L, n=-1) == append(L, n=4) == append(L, rot=0) == append(L, pairs=2) == append(L, q=rows(L)) == E
    assert append(L, rot=24) == U
    assert append(L, n=0, cu=256) == 0                            # nothing to do is no error
    for call in (step, shared):
        assert call(L, ws=0) == call(L, ws=264) == call(L, lse=258) == E
        assert call(L, size=100) == L.LOLA_ERR_WORKSPACE


def test_prefix_refusals(L):
    E, U = L.LOLA_ERR_INVALID_ARG, L.LOLA_ERR_UNSUPPORTED
    for bad in (dict(n=0), dict(n=-1), dict(width=0), dict(table_stride=3), dict(table=0), dict(table=258), dict(len=0), dict(len=258),
                dict(cu=258), dict(cu=0)):
        assert shared(L, px=prefixes(L, **bad)) == E, bad
    assert shared(L, px=ctypes.POINTER(L.lola_prefixes)()) == E
    assert shared(L, px=prefixes(L, width=1 << 26, table_stride=1 << 26)) == U
    one = L._lib.lola_shared_decode_workspace_bytes
    c = cfg(L)
    need = one(ctypes.byref(c), 3)
    assert need > L.lola_paged_decode_workspace_bytes(c)
    assert shared(L, size=need - 1) == L.LOLA_ERR_WORKSPACE
    assert one(ctypes.byref(c), 0) == one(ctypes.byref(c), -5) == E and one(ctypes.byref(cfg(L, Hq=1 << 20, Hkv=1)), 1 << 20) == U
    assert one(ctypes.byref(cfg(L, d=96)), 3) == U
    with pytest.raises(L.LolaError):
        L.lola_shared_decode_workspace_bytes(c, 0)


def test_layers_check_what_they_are_given(L, monkeypatch):
    monkeypatch.setattr(L, "_index_of", lambda dev: 0)
    lay = L.QuantizedAttention.allocate(4, 2, 64, 6, 16, device="cpu")
    lens, table = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    assert lay._cache(lens, table)[0].n_pages == 6
    good = lay.k_pool, lay.v_pool, lay.k_scale, lay.v_scale
    byte = torch.uint8
    z = lambda *s: torch.zeros(*s, dtype=byte)  # noqa: E731
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    for i, bad in ((0, None), (3, None), (0, z(6, 2, 16, 64)), (1, z(6, 2, 16, 32).view(e4)), (1, z(5, 2, 16, 64).view(e4)),
                   (2, z(6, 2, 16)), (2, z(6, 16, 2).view(e8)), (3, z(6, 2, 32).view(e8)), (0, z(6, 16, 2, 64).view(e4).transpose(1, 2)),
                   (0, z(6, 2, 16, 64).view(torch.float8_e5m2))):
        x = list(good)
        x[i] = bad
        with pytest.raises(ValueError):
            L.QuantizedAttention(4, 2, 64, torch.bfloat16, *x)
        lay.k_pool, lay.v_pool, lay.k_scale, lay.v_scale = x
        with pytest.raises(ValueError):
            lay.decode_step(q, lens, table)
        with pytest.raises(ValueError):
            lay.append(q[:, :2], q[:, :2], lens, table)
        with pytest.raises(ValueError):
            lay.decode_shared(q, lens, table, lens, table)
        with pytest.raises(ValueError):
            lay.read(lens, table, 1)
    lay.k_pool, lay.v_pool, lay.k_scale, lay.v_scale = good
    with pytest.raises(ValueError):
        lay.prefill_paged(q, torch.zeros(2, dtype=torch.int32), lens, table)          # total_k is needed
    for total in (-1, 1.5, None, 1 << 31):
        with pytest.raises((ValueError, TypeError)):
            lay.read(lens, table, total)
    for kw in (dict(prefix_len=lens.long()), dict(prefix_len=torch.ones(2, dtype=torch.int32)), dict(prefix_table=table.long()),
               dict(cu_prefix=lens), dict(prefix_len=torch.ones(2, dtype=torch.int32), prefix_table=torch.zeros(2, 1, dtype=torch.int32)),
               dict(prefix_table=torch.zeros(1, 4, dtype=torch.int32)[:, ::2])):
        a = dict(prefix_len=lens, prefix_table=table)
        a.update(kw)
        with pytest.raises(ValueError):
            lay.decode_shared(q, lens, table, **a)
    none = L.QuantizedAttention(4, 2, 64)
    for call in (lambda: none.decode_step(q, lens, table), lambda: none.read(lens, table, 1), lambda: none.decode_shared(q, lens, table, lens, table),
                 lambda: none.append(q[:, :2], q[:, :2], lens, table)):
        with pytest.raises(ValueError):
            call()


def test_copies_of_a_layer(L):
    lay = L.QuantizedAttention.allocate(4, 2, 64, 3, 16, device="cpu", scale=0.3)
    for other in (copy.copy(lay), copy.deepcopy(lay), pickle.loads(pickle.dumps(lay))):
        assert other._plan == (ctypes.addressof(other.cfg), lay._ws) and bytes(other.cfg) == bytes(lay.cfg)
        assert other.k_scale.shape == (3, 2, 16) and other.v_pool.dtype == torch.float8_e4m3fn
    assert copy.copy(lay).k_scale is lay.k_scale


def test_rounding_of_the_plain_form():
    """Half a step at most, the smallest power that fits, exact numbers kept."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(400, 64, generator=gen) * 2.0 ** torch.linspace(-60, 60, 400)[:, None]
    codes, power = encode(x)
    e = power.double() - 127
    top = x.double().abs().amax(-1)
    assert bool((top <= 448 * 2.0 ** e).all()) and bool((top > 448 * 2.0 ** (e - 1)).all())
    off = (decode(codes, power) - x.double()).abs()
    assert bool((off <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** (e - 10)[:, None])).all())
    again, p2 = encode(decode(codes, power).float())
    assert torch.equal(decode(again, p2), decode(codes, power))
    assert float(encode(torch.tensor([[math.nan, 448.0]]))[0][0, 1].float()) == 448.0
