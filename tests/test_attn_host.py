"""Exact attention over packed prompts and a paged cache, without a GPU: refusals return before
anything is enqueued, and the position arithmetic that the kernels share never leaves the pool."""
import ctypes
import random

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import sparse_exact_kv_gb300 as lib
    return lib


P = ctypes.c_void_p


def cfg(L, **kw):
    a = dict(Hq=8, Hkv=2, d=128, dtype="bf16", scale=None)
    a.update(kw)
    return L.make_attn_config(**a)


def rows(L, data=256, row=1024, head=128):
    return L.lola_rows(data, row, head)


def paged(L, **kw):
    a = dict(K=256, V=256, n_pages=10, page=64, n_seq=3, width=4, table_stride=4, table=256, kv_len=256)
    a.update(kw)
    return L.lola_paged_kv(*a.values())


BAD_CFG = [dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(d=0), dict(dtype=5), dict(scale=-1.0), dict(scale=float("nan")),
           dict(scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD_CFG)
def test_invalid_configs(L, bad):
    c = cfg(L, **bad)
    assert L._lib.lola_paged_decode_workspace_bytes(ctypes.byref(c)) == L.LOLA_ERR_INVALID_ARG
    assert prefill(L, c=c) == L.LOLA_ERR_INVALID_ARG
    with pytest.raises(L.LolaError):
        L.lola_paged_decode_workspace_bytes(c)


@pytest.mark.parametrize("bad", [dict(d=96), dict(d=256), dict(d=32)])
def test_unsupported_widths(L, bad):
    assert prefill(L, c=cfg(L, **bad)) == L.LOLA_ERR_UNSUPPORTED
    assert decode(L, c=cfg(L, **bad)) == L.LOLA_ERR_UNSUPPORTED
    assert append(L, c=cfg(L, **bad)) == L.LOLA_ERR_UNSUPPORTED


def prefill(L, c=None, n_seq=2, tq=10, tk=10, cu_q=256, cu_k=256, q=None, k=None, v=None, o=None, lse=None):
    r = lambda x: ctypes.byref(x if x is not None else rows(L))  # noqa: E731
    return L._lib.lola_attn_prefill(ctypes.byref(c or cfg(L)), n_seq, tq, tk, P(cu_q), P(cu_k), r(q), r(k), r(v), r(o),
                                    P(lse), None)


def decode(L, c=None, kv=None, q=None, o=None, lse=None, ws=256, size=1 << 30):
    r = lambda x: ctypes.byref(x if x is not None else rows(L))  # noqa: E731
    return L._lib.lola_paged_decode(ctypes.byref(c or cfg(L)), ctypes.byref(kv or paged(L)), r(q), r(o), P(lse), P(ws),
                                    size, None)


def append(L, c=None, kv=None, n=3, cu=None, k=None, v=None, q=None, qo=None, inv=256, rot=64, pairs=0, pos=None):
    r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return L._lib.lola_paged_append(ctypes.byref(c or cfg(L)), ctypes.byref(kv or paged(L)), n, P(cu),
                                    r(k or rows(L)), r(v or rows(L)), r(q), r(qo), P(inv), rot, pairs, P(pos), None)


def prefill_paged(L, c=None, kv=None, tq=10, tk=0, cu_q=256, q=None, o=None, lse=None):
    r = lambda x: ctypes.byref(x if x is not None else rows(L))  # noqa: E731
    return L._lib.lola_paged_prefill(ctypes.byref(c or cfg(L)), ctypes.byref(kv or paged(L)), tq, tk, P(cu_q), r(q), r(o),
                                     P(lse), None)


BAD_ROWS = [dict(data=0), dict(data=264), dict(row=0), dict(row=-1024), dict(head=0), dict(row=1028), dict(head=132),
            dict(row=1 << 41), dict(head=1 << 41)]


def test_prefill_refusals(L):
    E = L.LOLA_ERR_INVALID_ARG
    for bad in BAD_ROWS:
        for what in "qkvo":
            assert prefill(L, **{what: rows(L, **bad)}) == E, (bad, what)
    # overlapping output rows: both orders of the strides are fine when dense, nothing else
    assert prefill(L, o=rows(L, row=128, head=128)) == E
    assert prefill(L, o=rows(L, row=512, head=128)) == E            # 8 heads of 128 need 1024
    assert prefill(L, o=rows(L, row=128, head=512)) == E            # 10 rows of 128 need 1280
    for kw in (dict(n_seq=0), dict(tq=-1), dict(tk=-1), dict(cu_q=0), dict(cu_q=258), dict(cu_k=258), dict(lse=258),
               dict(cu_k=0, tk=11)):
        assert prefill(L, **kw) == E, kw
    assert prefill(L, c=cfg(L, Hq=1 << 20, Hkv=1), tq=1 << 30, tk=1 << 30, o=rows(L, row=1 << 27)) in \
        (L.LOLA_ERR_UNSUPPORTED, E)
    assert prefill(L, tk=0x7fffffff, k=rows(L, row=128), v=rows(L, row=128)) == L.LOLA_ERR_UNSUPPORTED
    # nothing to do is not an error, and touches nothing
    assert prefill(L, tq=0, tk=0, q=rows(L, data=0), o=rows(L, data=0)) == 0


def test_decode_refusals(L):
    E = L.LOLA_ERR_INVALID_ARG
    for bad in BAD_ROWS:
        assert decode(L, q=rows(L, **bad)) == E, bad
        assert decode(L, o=rows(L, **bad)) == E, bad
    for bad in (dict(K=0), dict(V=0), dict(K=264), dict(V=264), dict(n_pages=0), dict(n_seq=0), dict(width=0),
                dict(table_stride=3), dict(table=0), dict(kv_len=0), dict(table=258), dict(kv_len=258), dict(page=0),
                dict(page=-16)):
        assert decode(L, kv=paged(L, **bad)) == E, bad
        assert append(L, kv=paged(L, **bad)) == E, bad
    for page in (1, 8, 24, 48, 512):
        assert decode(L, kv=paged(L, page=page)) == L.LOLA_ERR_UNSUPPORTED, page
    assert decode(L, kv=paged(L, n_pages=1 << 30)) == L.LOLA_ERR_UNSUPPORTED
    assert decode(L, kv=paged(L, width=1 << 26, table_stride=1 << 26)) == L.LOLA_ERR_UNSUPPORTED
    assert decode(L, ws=0) == E
    assert decode(L, ws=264) == E
    assert decode(L, lse=258) == E
    need = L.lola_paged_decode_workspace_bytes(cfg(L))
    assert need > 0
    assert decode(L, size=need - 1) == L.LOLA_ERR_WORKSPACE


def test_paged_prefill_refusals(L):
    E = L.LOLA_ERR_INVALID_ARG
    for bad in BAD_ROWS:
        assert prefill_paged(L, q=rows(L, **bad)) == E, bad
        assert prefill_paged(L, o=rows(L, **bad)) == E, bad
    assert prefill_paged(L, o=rows(L, row=128, head=128)) == E
    for bad in (dict(K=0), dict(V=264), dict(n_pages=0), dict(n_seq=0), dict(width=0), dict(table_stride=3), dict(table=0),
                dict(kv_len=258), dict(page=0)):
        assert prefill_paged(L, kv=paged(L, **bad)) == E, bad
    for page in (8, 24, 512):
        assert prefill_paged(L, kv=paged(L, page=page)) == L.LOLA_ERR_UNSUPPORTED, page
    for kw in (dict(tq=-1), dict(tk=-1), dict(cu_q=0), dict(cu_q=258), dict(lse=258)):
        assert prefill_paged(L, **kw) == E, kw
    assert prefill_paged(L, kv=paged(L, width=0x7fffff, table_stride=1 << 24, page=256)) == L.LOLA_ERR_UNSUPPORTED
    assert prefill_paged(L, tq=0x7fffffff, q=rows(L, row=128), o=rows(L)) in (E, L.LOLA_ERR_UNSUPPORTED)
    assert prefill_paged(L, tq=0, q=rows(L, data=0), o=rows(L, data=0)) == 0


def test_append_refusals(L):
    E = L.LOLA_ERR_INVALID_ARG
    for bad in BAD_ROWS:
        assert append(L, k=rows(L, **bad)) == E, bad
        assert append(L, v=rows(L, **bad)) == E, bad
        assert append(L, q=rows(L, **bad), qo=rows(L, data=1 << 20)) == E, bad
        assert append(L, qo=rows(L, **bad), q=rows(L, data=1 << 20)) == E, bad
    assert append(L, q=rows(L)) == E                              # q without its output
    assert append(L, qo=rows(L)) == E
    assert append(L, q=rows(L), qo=rows(L), inv=0) == E           # q without a rotation
    assert append(L, q=rows(L, row=2048), qo=rows(L)) == E        # in place, other strides
    for kw in (dict(n=-1), dict(n=4), dict(rot=0), dict(rot=144), dict(pairs=2), dict(pairs=-1), dict(cu=258),
               dict(inv=258), dict(pos=258)):
        assert append(L, **kw) == E, kw
    assert append(L, rot=24) == L.LOLA_ERR_UNSUPPORTED
    assert append(L, n=0, cu=256) == 0


def test_positions_never_leave_the_pool(L):
    """lola_paged_slot is the kernels' own resolution: over tables of any content and lengths of any
    value, a slot is inside the pool or refused."""
    r = random.Random(3)
    for trial in range(300):
        page = r.choice([16, 32, 64, 128, 256])
        n_pages, width, n_seq, stride = r.randint(1, 9), r.randint(1, 5), r.randint(1, 4), r.randint(5, 8)
        Hkv, d = r.choice([1, 2, 3]), r.choice([64, 128])
        c = cfg(L, Hq=Hkv * 2, Hkv=Hkv, d=d)
        values = [r.choice([-1, -2 ** 31, 2 ** 31 - 1, n_pages, n_pages - 1, 0, r.randint(0, n_pages - 1)])
                  for _ in range(n_seq * stride)]
        lens = [r.choice([-5, 0, 1, page, page * width, page * width + 7, 2 ** 31 - 1]) for _ in range(n_seq)]
        table, kv_len = torch.tensor(values, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
        kv = paged(L, n_pages=n_pages, page=page, n_seq=n_seq, width=width, table_stride=stride, table=table.data_ptr(),
                   kv_len=kv_len.data_ptr())
        for _ in range(60):
            b, h = r.randint(-1, n_seq), r.randint(-1, Hkv)
            pos = r.choice([-1, 0, page - 1, page, page * width - 1, page * width, r.randint(0, page * width), 2 ** 40])
            got = L.lola_paged_slot(c, kv, b, h, pos)
            ok = 0 <= b < n_seq and 0 <= h < Hkv and 0 <= pos < min(max(lens[b], 0), page * width)
            e = values[b * stride + pos // page] if ok else -1
            want = ((e * Hkv + h) * page + pos % page) * d if ok and 0 <= e < n_pages else -1
            assert got == want
            assert got == -1 or 0 <= got <= n_pages * Hkv * page * d - d


def test_page_tables_whose_rows_overlap_are_refused(L, monkeypatch):
    """An expanded table's rows have a stride of 0: the library gets it as it is, and refuses it."""
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    row, lens = torch.zeros(1, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    wide = torch.zeros(3, 5, dtype=torch.int32)
    lay = L.ExactAttention(4, 2, 64, torch.bfloat16, pool, pool.clone())
    monkeypatch.setattr(L, "_index_of", lambda dev: 0)
    for table, stride in ((row.expand(2, 3), 0), (wide.as_strided((2, 3), (2, 1)), 2), (wide[:2, :3], 5)):
        for kv in (L._paged(pool, pool, lens, table), lay._cache(lens, table)[0]):
            assert kv.table_stride == stride
            assert (L.lola_paged_slot(lay.cfg, kv, 1, 0, 0) >= 0) == (stride >= 3)
    for table in (row, row.expand(1, 3), wide[:1, :3], wide.as_strided((1, 3), (1, 1))):      # one row: any stride
        assert L.lola_paged_slot(lay.cfg, lay._cache(lens[:1], table)[0], 0, 0, 0) == 0


def test_layer_refuses_other_tensors(L):
    """The class checks shapes, types and devices before the library is called."""
    bf, f32 = torch.bfloat16, torch.float32
    pool = torch.zeros(4, 2, 16, 64, dtype=bf)
    with pytest.raises(L.LolaError):
        L.ExactAttention(3, 2, 64)
    with pytest.raises(ValueError):
        L.ExactAttention(4, 2, 64, bf, pool)
    with pytest.raises(ValueError):
        L.ExactAttention(4, 2, 64, f32, pool, pool)
    with pytest.raises(ValueError):
        L.ExactAttention(4, 2, 64, bf, pool, torch.zeros(5, 2, 16, 64, dtype=bf))
    with pytest.raises(ValueError):
        L.ExactAttention(4, 2, 64, bf, pool.transpose(1, 2), pool.transpose(1, 2))
    lay = L.ExactAttention(4, 2, 64, bf, pool, pool.clone())
    q, k = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    lens, table = torch.tensor([3], dtype=torch.int32), torch.tensor([[0]], dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(k=k[:2]), dict(cu_q=cu.long()), dict(cu_k=torch.zeros(3, dtype=torch.int32)),
                dict(out=q[:2]), dict(lse=torch.zeros(3, 4))):
        with pytest.raises(ValueError):
            lay.prefill(**{**dict(q=q, k=k, v=k, cu_q=cu), **bad})
    with pytest.raises(ValueError):
        lay.prefill(q, k, k, cu)                        # not on a CUDA device
    with pytest.raises(ValueError):
        lay.decode_step(q[:1], lens, table)
    with pytest.raises(ValueError):
        lay.append(k, k, lens, table, cu_new=cu)
    with pytest.raises(ValueError):
        L.ExactAttention(4, 2, 64, bf).decode_step(q[:1], lens, table)
