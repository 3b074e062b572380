"""The quantised paged cache and shared prefixes on the GPU against plain float64 forms.  Bounds: tests/quant_parity.py."""
import math

import pytest
import torch

from attn_parity import Paged, check, ints, offsets, randn, rotated
from quant_parity import E4, E8, QPaged, check_attention, decode, encode

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_exact_kv_gb300 as lib
    return lib


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(23)


def quiet(L):
    st, bits = L.lola_attn_status()
    assert st == 0 and bits == 0, bits


def check_decode(q, c, out, lse=None, scale=None, hidden=None):
    for b, n in enumerate(c.lens):
        check_attention(q[b], [(c.k[b][:n], c.v[b][:n], hidden[b] if hidden else None)], out[b], None if lse is None else lse[b],
                        scale, f"sequence {b}")


# ---------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------

def written(c, b, pos):
    """Codes and powers in the cache of a sequence's tokens: {"k": (codes, bytes), ...}."""
    at = c.table[b].long()[pos // c.page], pos % c.page
    return {w: (getattr(c, w + "_pool").view(torch.uint8)[at[0], :, at[1]].view(E4),
                getattr(c, w + "_scale").view(torch.uint8)[at[0], :, at[1]]) for w in "kv"}


@pytest.mark.parametrize("dtype,d,rot", [(BF, 128, 128), (BF, 64, 64), (BF, 128, 48), (F32, 128, 128), (F32, 64, 16)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("new,before", [([1, 1, 1], [0, 15, 4000]), ([5, 0, 200], [11, 3, 0]), ([1], [0]), ([900], [7])])
def test_append(L, gen, dtype, d, rot, pairs, new, before):
    Hq, Hkv, page = 6, 2, 32
    total = [a + b for a, b in zip(new, before)]
    c = QPaged(gen, total, Hkv, d, page, dtype)
    pools = {w: (getattr(c, w + "_pool").view(torch.uint8).clone(), getattr(c, w + "_scale").view(torch.uint8).clone()) for w in "kv"}
    n = sum(new)
    q, k, v = (randn(gen, n, h, d, dtype=dtype) for h in (Hq, Hkv, Hkv))
    k *= torch.exp(2 * randn(gen, n, Hkv, 1, dtype=F32)).to(dtype)
    v *= torch.exp2(torch.randint(-30, 30, (n, Hkv, 1), generator=gen, device="cuda").float()).to(dtype)
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    freq = freq.float().cuda()
    qr = c.layer(L, Hq, Hkv, d, dtype).append(k, v, c.kv_len, c.table, cu_new=offsets(new), q=q, inv_freq=freq, pairs=pairs)
    quiet(L)
    r = 0
    for b, m in enumerate(new):
        pos = torch.arange(before[b], total[b], device="cuda")
        rows = slice(r, r + m)
        want, tol = rotated(q[rows], pos, freq, pairs)
        check(qr[rows], want, tol, f"q of sequence {b}")
        got = written(c, b, pos)
        codes, power = encode(v[rows])                        # values: bit for bit
        assert torch.equal(got["v"][0].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(got["v"][1], power)
        # keys: the power fits the largest magnitude, and no smaller one does; one rounding
        want, tol = rotated(k[rows], pos, freq, pairs)
        tol = tol - (2.0 ** -8 if dtype == BF else 2.0 ** -24) * want.abs()       # (not rounded to io)
        e = got["k"][1].double() - 127
        if m:
            top, slack = want.abs().amax(-1), tol.amax(-1)
            assert bool((top - slack <= 448 * 2.0 ** e).all()) and bool((top + slack > 448 * 2.0 ** (e - 1)).all())
        half = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** (e - 10)[..., None])
        check(decode(*got["k"]), want, half + tol * (1 + 2.0 ** -4), f"k of sequence {b}")
        r += m
    # nothing else is touched
    for w in "kv":
        for b, m in enumerate(new):
            pos = torch.arange(before[b], total[b], device="cuda")
            at = c.table[b].long()[pos // page], pos % page
            for old, now in zip(pools[w], (getattr(c, w + "_pool"), getattr(c, w + "_scale"))):
                old[at[0], :, at[1]] = now.view(torch.uint8)[at[0], :, at[1]]
        for old, now in zip(pools[w], (getattr(c, w + "_pool"), getattr(c, w + "_scale"))):
            assert torch.equal(old, now.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_every_magnitude_and_numbers_that_are_not_finite(L, gen, dtype):
    """Powers at both ends, rows of zeros, ties, and NaN and infinities beside finite numbers."""
    d, n = 128, 300
    c = QPaged(gen, [n], 1, d, 64, dtype)
    x = randn(gen, n, 1, d, dtype=F32) * 2.0 ** torch.linspace(-149, 126, n, device="cuda")[:, None, None]
    x[0] = 0.0
    x[1] = 448.0 * 2.0 ** torch.randint(-20, 20, (1, d), generator=gen, device="cuda").float()
    x[2], x[3] = 3.3e38, torch.where(torch.arange(d, device="cuda") % 2 == 0, 449.0, 1.0)
    x[4] = torch.arange(d, device="cuda").float() / 16        # ties between codes
    x[5:40, 0, 3], x[20:60, 0, 77], x[50:60, 0, 5] = math.nan, math.inf, -math.inf
    x[60] = math.inf
    x = x.to(dtype)
    c.layer(L, 1, 1, d, dtype).append(x, x.flip(-1).contiguous(), c.kv_len, c.table, cu_new=offsets([n]))
    quiet(L)
    got = written(c, 0, torch.arange(n, device="cuda"))
    for w, y in (("k", x), ("v", x.flip(-1))):
        codes, power = encode(y)
        assert torch.equal(got[w][1], power)
        nan = torch.isnan(codes.float())
        assert torch.equal(nan, torch.isnan(got[w][0].float()))
        assert torch.equal(codes.view(torch.uint8)[~nan], got[w][0].view(torch.uint8)[~nan])


def test_append_padded_batches_and_bad_pages(L, gen):
    """Rows outside cu_new and of empty sequences are skipped; a token without a slot is reported and its query written."""
    c = QPaged(gen, [40, 1, 33], 2, 64, 16, BF)
    lay = c.layer(L, 4, 2, 64, BF)
    q, k, v = (randn(gen, 9, h, 64, dtype=BF) for h in (4, 2, 2))
    freq = torch.rand(32, generator=gen, device="cuda")
    before = [x.view(torch.uint8).clone() for x in (c.k_pool, c.v_pool, c.k_scale, c.v_scale)]
    out = torch.full_like(q, 7.0)
    lay.append(k, v, ints([0, -3, 0]), c.table, cu_new=ints([2, 4, 4, 6]), q=q, inv_freq=freq, q_out=out)
    quiet(L)
    assert bool((out == 7).all())
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (c.k_pool, c.v_pool, c.k_scale, c.v_scale)))
    table = c.table.clone()
    table[0, 2], table[2, 2] = -1, c.n_pages
    lay.append(k[:3], v[:3], c.kv_len, table, q=q[:3], inv_freq=freq, q_out=out[:3])
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    want, tol = rotated(q[:3], ints([39, 0, 32]), freq, "halves")
    check(out[:3], want, tol, "q")
    got = written(c, 1, torch.zeros(1, dtype=torch.long, device="cuda"))
    codes, power = encode(v[1:2])
    assert torch.equal(got["v"][0].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(got["v"][1], power)
    before[1][c.table[1, 0].long(), :, 0] = codes.view(torch.uint8)[0]
    assert torch.equal(before[1], c.v_pool.view(torch.uint8))


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF, 128, 6, 3), (BF, 64, 12, 1), (F32, 128, 3, 3), (F32, 64, 9, 1)])
def test_append_many_rows_padded_bad_pages_and_numbers_that_are_not_finite(L, gen, dtype, d, Hq, Hkv):
    """As above, in calls of more tokens than a CTA each is given."""
    page, n, cu = 16, 1003, [2, 700, 700, 990]
    c = QPaged(gen, [750, 5, 290], Hkv, d, page, dtype)
    lay = c.layer(L, Hq, Hkv, d, dtype)
    q, k, v = (randn(gen, n, h, d, dtype=dtype) for h in (Hq, Hkv, Hkv))
    k *= torch.exp2(torch.randint(-90, 90, (n, Hkv, 1), generator=gen, device="cuda").float()).to(dtype)
    k[torch.rand(k.shape, generator=gen, device="cuda") < 0.01] = math.nan
    v[torch.rand(v.shape, generator=gen, device="cuda") < 0.01] = -math.inf
    table = c.table.clone()
    table[0, 30], table[2, 0] = c.n_pages, -5                # positions 480 .. 495 of sequence 0, 0 .. 15 of 2
    before = {w: (getattr(c, w + "_pool").view(torch.uint8).clone(), getattr(c, w + "_scale").view(torch.uint8).clone()) for w in "kv"}
    lay.append(k, v, c.kv_len, table, cu_new=ints(cu))
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    rows = [(b, cu[b] + i, len_ - (cu[b + 1] - cu[b]) + i) for b, len_ in enumerate(c.lens) for i in range(cu[b + 1] - cu[b])]
    rows = [r for r in rows if not (r[0] == 0 and 480 <= r[2] < 496) and not (r[0] == 2 and r[2] < 16)]
    b, r, pos = (torch.tensor(x, device="cuda") for x in zip(*rows))
    at = c.table.long()[b, pos // page], pos % page
    for w, x in (("k", k), ("v", v)):
        codes, power = encode(x[r])
        pool, scale = before[w]
        pool[at[0], :, at[1]], scale[at[0], :, at[1]] = codes.view(torch.uint8), power
        now = getattr(c, w + "_pool").view(torch.uint8)
        nan = (pool & 0x7f) == 0x7f                          # (NaN has two codes)
        assert torch.equal(nan, (now & 0x7f) == 0x7f) and torch.equal(pool[~nan], now[~nan])
        assert torch.equal(scale, getattr(c, w + "_scale").view(torch.uint8))
    # queries are written for tokens without a slot too, and for no row outside the sequences; positions of the caller's
    freq = torch.rand(d // 2, generator=gen, device="cuda")
    where = torch.randint(0, 1 << 24, (n,), generator=gen, device="cuda", dtype=torch.int64).int()
    out = torch.full_like(q, 7.0)
    lay.append(k, v, c.kv_len, table, cu_new=ints(cu), q=q, inv_freq=freq, q_out=out, positions=where, pairs="neighbours")
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    want, tol = rotated(q, where.long(), freq, "neighbours")
    inside = torch.zeros(n, dtype=torch.bool, device="cuda")
    inside[2:990] = True
    check(out[inside], want[inside], tol[inside], "q")
    assert bool((out[~inside] == 7).all())
    # in place, and in rows of one projection
    both = torch.cat([q, k, v], 1)
    lay.append(both[:, Hq:Hq + Hkv], both[:, Hq + Hkv:], c.kv_len, table, cu_new=ints(cu), q=both[:, :Hq], inv_freq=freq,
               q_out=both[:, :Hq], positions=where, pairs="neighbours")
    L.lola_attn_status()
    assert torch.equal(both[inside, :Hq], out[inside]) and torch.equal(both[~inside, :Hq], q[~inside])


# ---------------------------------------------------------------------------------------
# read
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d,Hkv", [(BF, 128, 2), (BF, 64, 3), (F32, 128, 1), (F32, 64, 4)])
@pytest.mark.parametrize("page,lens", [(16, [1]), (16, [15, 0, 17, 33]), (64, [127, 128, 129, 0]), (256, [1000, 3]), (32, [3] * 300)])
def test_read(L, gen, dtype, d, Hkv, page, lens):
    c = QPaged(gen, lens, Hkv, d, page, dtype)
    total = sum(lens)
    k, v, cu = c.layer(L, Hkv, Hkv, d, dtype).read(c.kv_len, c.table, total)
    quiet(L)
    assert torch.equal(cu, offsets(lens)) and k.shape == v.shape == (total, Hkv, d) and k.dtype == v.dtype == dtype
    assert torch.equal(k.double(), torch.cat(c.k)) and torch.equal(v.double(), torch.cat(c.v))


def test_read_rows_that_do_not_fit_and_bad_pages(L, gen):
    lens = [40, 20, 30]
    c = QPaged(gen, lens, 2, 64, 16, BF)
    lay = c.layer(L, 2, 2, 64, BF)
    want = torch.cat(c.k)
    kv, *_ = lay._cache(c.kv_len, c.table)
    k, v = (torch.full((95, 2, 64), 7.0, dtype=BF, device="cuda") for _ in range(2))
    cu = ints([9] * 4)
    L.lola_quant_read(lay.cfg, kv, *lay._scales(), k[:92], v[:92], cu)     # more rows than tokens
    quiet(L)
    assert torch.equal(k[:90].double(), want) and bool((k[90:] == 7).all()) and bool((v[90:] == 7).all())
    k.fill_(7.0), v.fill_(7.0)
    L.lola_quant_read(lay.cfg, kv, *lay._scales(), k[:50], v[:50], cu)     # fewer
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_OFFSETS
    assert torch.equal(k[:50].double(), want[:50]) and bool((k[50:] == 7).all()) and cu.tolist() == [0, 40, 50, 50]
    k, v, cu = lay.read(ints([0, -1, 0]), c.table, 0)                      # none
    quiet(L)
    assert k.shape[0] == 0 and cu.tolist() == [0, 0, 0, 0]
    table = c.table.clone()
    table[0, 1], table[1, 0] = -1, c.n_pages
    k, v, cu = lay.read(c.kv_len, table, 90)
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    want[16:32], want[40:56] = 0, 0
    assert torch.equal(k.double(), want)
    wide = c.table.shape[1] * 16
    k, v, cu = lay.read(ints([2 ** 31 - 1, 20, 0]), table.clamp(0, c.n_pages - 1), wide + 20)
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE and cu.tolist() == [0, wide, wide + 20, wide + 20]


# ---------------------------------------------------------------------------------------
# one token per sequence
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF, 128, 8, 2), (BF, 64, 6, 6), (BF, 128, 5, 1), (F32, 64, 4, 2), (F32, 128, 3, 3)])
@pytest.mark.parametrize("page,lens", [(16, [1]), (16, [15, 16, 17, 0, 33]), (32, [63, 64, 65, 1]), (64, [127, 128, 129]),
                                       (128, [1, 300, 0, 513]), (256, [1000, 255, 257]), (16, [2000, 5])])
def test_decode_lengths(L, gen, dtype, d, Hq, Hkv, page, lens):
    c = QPaged(gen, lens, Hkv, d, page, dtype)
    q = randn(gen, len(lens), Hq, d, dtype=dtype)
    lse = torch.empty(len(lens), Hq, dtype=F32, device="cuda")
    out = c.layer(L, Hq, Hkv, d, dtype).decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    check_decode(q, c, out, lse)
    assert torch.equal(out, c.layer(L, Hq, Hkv, d, dtype).decode_step(q, c.kv_len, c.table))


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF, 128, 16, 1), (BF, 64, 17, 1), (BF, 128, 40, 1), (BF, 64, 64, 2), (F32, 128, 16, 1),
                                            (F32, 64, 20, 1), (F32, 128, 20, 1)])
def test_decode_many_query_heads_per_key_head(L, gen, dtype, d, Hq, Hkv):
    c = QPaged(gen, [700, 64], Hkv, d, 64, dtype)
    q = randn(gen, 2, Hq, d, dtype=dtype)
    lse = torch.empty(2, Hq, dtype=F32, device="cuda")
    out = c.layer(L, Hq, Hkv, d, dtype).decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    check_decode(q, c, out, lse)


@pytest.mark.parametrize("dtype,d,n", [(BF, 128, 70001), (BF, 64, 30000), (F32, 64, 20001), (F32, 128, 9000)])
def test_decode_long(L, gen, dtype, d, n):
    c = QPaged(gen, [n, 17], 1, d, 128, dtype)
    q = randn(gen, 2, 4, d, dtype=dtype)
    lse = torch.empty(2, 4, dtype=F32, device="cuda")
    out = c.layer(L, 4, 1, d, dtype).decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    check_decode(q, c, out, lse)


def test_decode_many_sequences(L, gen):
    lens = [(37 * i) % 211 for i in range(700)]
    c = QPaged(gen, lens, 1, 64, 16, BF)
    q = randn(gen, 700, 2, 64, dtype=BF)
    out = c.layer(L, 2, 1, 64, BF).decode_step(q, c.kv_len, c.table)
    quiet(L)
    check_decode(q, c, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("up", [-60, -20, 15, 60])
def test_decode_powers_of_many_sizes(L, gen, dtype, up):
    """Values and keys of magnitudes far from one, and of many different ones in a sequence; queries that make up for it."""
    lens, d = [333, 90], 128
    c = QPaged(gen, lens, 1, d, 32, dtype)
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        f = 2.0 ** torch.randint(-6, 6, (n, 1, 1), generator=gen, device="cuda").double()
        c.k[b] = c.store("k", b, pos, (c.k[b] * 2.0 ** -up).float())
        c.v[b] = c.store("v", b, pos, (c.v[b] * f * 2.0 ** up).float())
    q = (randn(gen, 2, 3, d, dtype=F32) * 2.0 ** up).to(dtype)
    lse = torch.empty(2, 3, dtype=F32, device="cuda")
    out = c.layer(L, 3, 1, d, dtype).decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    check_decode(q, c, out, lse)


@pytest.mark.parametrize("dtype,scale", [(BF, 1.0), (BF, 0.01), (F32, 1.0)])
def test_decode_scales_and_queries_of_uneven_channels(L, gen, dtype, scale):
    """Sharp and flat softmaxes; channels of a query 2^20 times others, and whose keys are small."""
    lens, d = [500, 77], 64
    c = QPaged(gen, lens, 2, d, 64, dtype)
    q = randn(gen, 2, 4, d, dtype=F32)
    q[:, :, :5] *= 2.0 ** 14
    q[0, 1] = 0.0
    q = q.to(dtype)
    for b, n in enumerate(lens):
        x = c.k[b].clone()
        x[:, :, :5] *= 2.0 ** -14
        c.k[b] = c.store("k", b, torch.arange(n, device="cuda"), x.float())
    lse = torch.empty(2, 4, dtype=F32, device="cuda")
    out = c.layer(L, 4, 2, d, dtype, scale).decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    check_decode(q, c, out, lse, scale)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_codes_that_are_not_numbers(L, gen, d):
    """A NaN in a value reaches its channel of the sequence, one in a key the whole row; none reaches other sequences."""
    lens = [100, 90, 80]
    c = QPaged(gen, lens, 1, d, 16, BF)
    c.v[0][7, 0, 3] = math.nan
    c.store("v", 0, torch.arange(100, device="cuda"), c.v[0].float())
    x = c.k[1].clone()
    x[89, 0, 5] = math.nan
    c.store("k", 1, torch.arange(90, device="cuda"), x.float())
    q = randn(gen, 3, 2, d, dtype=BF)
    q[2, 1, 0] = math.inf
    out = c.layer(L, 2, 1, d, BF).decode_step(q, c.kv_len, c.table)
    quiet(L)
    nan = torch.isnan(out)
    assert bool(nan[0, :, 3].all()) and int(nan[0].sum()) == 2 and bool(nan[1].all()) and not bool(nan[2, 0].any()) and bool(nan[2, 1].all())
    check_attention(q[2, :1], [(c.k[2], c.v[2], None)], out[2, :1])


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 128), (F32, 32)])
def test_decode_bad_pages_are_reported(L, gen, dtype, page):
    lens = [300, 200]
    c = QPaged(gen, lens, 1, 64, page, dtype)
    q = randn(gen, 2, 2, 64, dtype=dtype)
    lay = c.layer(L, 2, 1, 64, dtype)
    table = c.table.clone()
    hidden = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in lens]
    for col, bad in ((0, -1), (1, c.n_pages), (2, 2 ** 31 - 1)):
        if col * page < 300:
            table[0, col] = bad
            hidden[0][col * page:(col + 1) * page] = True
    out = lay.decode_step(q, c.kv_len, table)
    assert L.lola_attn_status() == (L.LOLA_ERR_DEVICE, L.LOLA_ATTN_BAD_PAGE)
    check_decode(q, c, out, hidden=hidden)
    table.fill_(-7)
    out = lay.decode_step(q, c.kv_len, table)
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE and bool((out == 0).all())


def test_decode_pool_past_32_bits(L, gen):
    """Pools of more than 2^32 bytes, their last pages used: appended, read back and attended."""
    page, Hkv, d, n = 256, 2, 128, 700
    n_pages = (1 << 32) // (page * Hkv * d) + 40
    pools = [torch.empty(n_pages, Hkv, page, d, dtype=torch.uint8, device="cuda").view(E4) for _ in range(2)]
    scales = [torch.empty(n_pages, Hkv, page, dtype=torch.uint8, device="cuda").view(E8) for _ in range(2)]
    k, v = randn(gen, n, Hkv, d, dtype=BF), randn(gen, n, Hkv, d, dtype=BF)
    table = ints([[n_pages - 1, n_pages - 30, n_pages - 7]])
    lay = L.QuantizedAttention(4, Hkv, d, BF, *pools, *scales)
    lay.append(k, v, ints([n]), table, cu_new=offsets([n]))
    kk, vv, cu = lay.read(ints([n]), table, n)
    q = randn(gen, 1, 4, d, dtype=BF)
    out = lay.decode_step(q, ints([n]), table)
    quiet(L)
    kd, vd = decode(*encode(k)), decode(*encode(v))
    assert torch.equal(kk.double(), kd) and torch.equal(vv.double(), vd)
    check_attention(q[0], [(kd, vd, None)], out[0])


def test_decode_strides_and_graphs(L, gen):
    lens = [130, 999, 64, 5]
    c = QPaged(gen, lens, 2, 128, 64, BF, width=20)
    wide = randn(gen, 4, 11, 128, dtype=BF)
    q = wide[:, 3:11]
    lay = c.layer(L, 8, 2, 128, BF)
    out = torch.empty(8, 4, 128, dtype=BF, device="cuda").transpose(0, 1)
    lay.decode_step(q, c.kv_len, c.table[:, :17], out=out)
    quiet(L)
    check_decode(q, c, out)
    graphs = []
    for _ in range(2):
        qs, n, o = q.clone(), c.kv_len.clone(), torch.zeros(4, 8, 128, dtype=BF, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            lay.decode_step(qs, n, c.table, out=o)
        graphs.append((g, qs, n, o))
    new = [[1, 500, 63, 0], [130, 999, 64, 5]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (g, qs, n, o), x in zip(graphs, new):
        qs.copy_(randn(gen, 4, 8, 128, dtype=BF))
        n.copy_(ints(x))
    torch.cuda.synchronize()
    for _ in range(4):
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    quiet(L)
    for (g, qs, n, o), x in zip(graphs, new):
        c.lens = x
        check_decode(qs, c, o)


# ---------------------------------------------------------------------------------------
# shared prefixes
# ---------------------------------------------------------------------------------------

WIDE = False


@pytest.fixture
def wide(request):
    """Prefix tables so wide that a call reads every prefix once, for all sequences, however short it is; otherwise
    short ones are read for each sequence."""
    global WIDE
    WIDE = request.param
    yield
    WIDE = False


def pytest_generate_tests(metafunc):
    if "Shared" in metafunc.function.__code__.co_names:
        metafunc.fixturenames.insert(0, "wide")
        metafunc.parametrize("wide", [False, True], ids=["narrow", "wide"], indirect=True)


class Shared:
    """A cache of prefixes and sequences: sequence b sees prefix of[b] (-1: none) before its own tokens."""

    def __init__(self, gen, quant, prefixes, members, lens, Hkv, d, page, dtype, start=0, **kw):
        self.c = (QPaged if quant else Paged)(gen, prefixes + lens, Hkv, d, page, dtype, **({} if quant else dict(junk=math.nan)), **kw)
        c, k = self.c, len(prefixes)
        self.prefix_len, self.kv_len = c.kv_len[:k].clone(), c.kv_len[k:].clone()
        self.prefix_table, self.table = c.table[:k], c.table[k:]
        if WIDE:
            row = 2 * Hkv * d * (1 if quant else torch.finfo(dtype).bits // 8)
            junk = torch.randint(-9, 1 << 30, (k, 64_000_000 // (len(lens) * page * row) + 2), generator=gen, device="cuda").int()
            self.prefix_table = torch.cat([self.prefix_table, junk], 1)
        self.cu = offsets(members, start)
        self.of = [-1] * start
        for g, m in enumerate(members):
            self.of += [g] * m
        self.of += [-1] * (len(lens) - len(self.of))
        self.k, self.lens = k, lens

    def layer(self, L, Hq, Hkv, d, dtype, scale=None):
        if isinstance(self.c, QPaged):
            return self.c.layer(L, Hq, Hkv, d, dtype, scale)
        return L.ExactAttention(Hq, Hkv, d, dtype, self.c.k_pool, self.c.v_pool, scale)

    def check(self, q, out, lse=None, scale=None, hidden=None, only=None):
        """``hidden``: {index of a prefix, or k + index of a sequence: bool tensor}"""
        c, hidden = self.c, hidden or {}
        part = lambda i: (c.k[i], c.v[i], hidden.get(i))  # noqa: E731
        for b in only if only is not None else range(len(self.lens)):
            parts = ([part(self.of[b])] if self.of[b] >= 0 else []) + [part(self.k + b)]
            check_attention(q[b], parts, out[b], None if lse is None else lse[b], scale, f"sequence {b}")


KINDS = [(BF, False, 128, 8, 2), (BF, False, 64, 6, 6), (BF, False, 128, 5, 1), (BF, True, 128, 8, 2), (BF, True, 64, 6, 1),
         (F32, False, 64, 4, 2), (F32, False, 128, 3, 3), (F32, True, 128, 4, 2), (F32, True, 64, 5, 1)]


@pytest.mark.parametrize("dtype,quant,d,Hq,Hkv", KINDS)
@pytest.mark.parametrize("page,prefixes,members,lens", [
    (16, [1], [1], [1]), (16, [100], [3], [5, 0, 17]), (64, [1000], [40], [3] * 40), (32, [513, 1, 0, 64], [2, 3, 2, 1], [7] * 8),
    (128, [129, 700], [0, 5], [200, 1, 0, 64, 63]), (256, [255, 256, 257], [1, 1, 1], [0, 0, 300]), (16, [300], [70], [1] * 70)])
def test_shared_lengths(L, gen, dtype, quant, d, Hq, Hkv, page, prefixes, members, lens):
    s = Shared(gen, quant, prefixes, members, lens, Hkv, d, page, dtype)
    q = randn(gen, len(lens), Hq, d, dtype=dtype)
    lse = torch.empty(len(lens), Hq, dtype=F32, device="cuda")
    lay = s.layer(L, Hq, Hkv, d, dtype)
    args = (s.kv_len, s.table, s.prefix_len, s.prefix_table, s.cu)
    out = lay.decode_shared(q, *args, lse=lse)
    quiet(L)
    s.check(q, out, lse)
    assert torch.equal(out, lay.decode_shared(q, *args))
    if len(prefixes) == 1:
        assert torch.equal(out, lay.decode_shared(q, *args[:-1]))


@pytest.mark.parametrize("dtype,quant,d,Hq,Hkv,n,members", [
    (BF, False, 128, 8, 2, 20001, 33), (BF, False, 64, 12, 2, 9000, 21), (BF, True, 128, 8, 1, 30000, 17), (BF, True, 64, 24, 4, 7000, 40),
    (BF, True, 128, 8, 8, 30000, 34), (BF, True, 64, 32, 8, 40001, 10), (F32, False, 64, 4, 1, 6001, 9), (F32, True, 128, 4, 1, 5000, 9), (BF, False, 128, 7, 1, 3000, 150), (BF, True, 128, 20, 1, 2500, 30)])
def test_shared_longer(L, gen, dtype, quant, d, Hq, Hkv, n, members):
    """Long prefixes, whose length is cut; rows that are no multiple of a tile's; own parts of many lengths."""
    lens = [(i * 83) % 300 for i in range(members + 3)]
    s = Shared(gen, quant, [n], [members], lens, Hkv, d, 64, dtype, start=1)
    q = randn(gen, len(lens), Hq, d, dtype=dtype)
    lse = torch.empty(len(lens), Hq, dtype=F32, device="cuda")
    out = s.layer(L, Hq, Hkv, d, dtype).decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, s.cu, lse=lse)
    quiet(L)
    s.check(q, out, lse, only=[0, 1, 2, members // 2, members, members + 1, members + 2])


@pytest.mark.parametrize("quant", [False, True])
def test_shared_many_prefixes(L, gen, quant):
    """More prefixes than the GPU has SMs, most shared by few; sequences without one at both ends."""
    prefixes = [(i * 131) % 400 for i in range(330)]
    members = [1 + (i % 3 == 0) - (i % 7 == 0) for i in range(330)]
    lens = [(i * 29) % 90 for i in range(sum(members) + 5)]
    s = Shared(gen, quant, prefixes, members, lens, 1, 64, 16, BF, start=2)
    q = randn(gen, len(lens), 2, 64, dtype=BF)
    out = s.layer(L, 2, 1, 64, BF).decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, s.cu)
    quiet(L)
    s.check(q, out)


@pytest.mark.parametrize("dtype,quant", [(BF, False), (BF, True), (F32, False), (F32, True)])
def test_shared_equals_sequences_that_hold_the_prefix_themselves(L, gen, dtype, quant):
    """Page-aligned prefixes: the same call with the prefix' pages in each sequence's table, within the sum of both bounds."""
    page, P, lens = 32, 256, [40, 0, 7]
    s = Shared(gen, quant, [P], [3], lens, 2, 128, page, dtype)
    q = randn(gen, 3, 8, 128, dtype=dtype)
    lay = s.layer(L, 8, 2, 128, dtype)
    out = lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table)
    table = torch.cat([s.prefix_table[:1, :P // page].expand(3, -1), s.table], 1).contiguous()
    long = lay.decode_step(q, s.kv_len + P, table)
    quiet(L)
    s.check(q, out), s.check(q, long)


@pytest.mark.parametrize("dtype,quant", [(BF, False), (BF, True), (F32, False)])
def test_shared_nothing_to_see(L, gen, dtype, quant):
    """Rows of no prefix and no token: zeros, and minus infinity; negative lengths count as none."""
    s = Shared(gen, quant, [0, 50], [2, 2], [0, 9, 0, 4, 0], 2, 64, 16, dtype)
    q = randn(gen, 5, 4, 64, dtype=dtype)
    lse = torch.zeros(5, 4, dtype=F32, device="cuda")
    lay = s.layer(L, 4, 2, 64, dtype)
    out = lay.decode_shared(q, s.kv_len - (s.kv_len == 0).int() * 3, s.table, ints([-7, 50]), s.prefix_table, s.cu, lse=lse)
    quiet(L)
    s.check(q, out, lse)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all()) and bool((out[4] == 0).all())


@pytest.mark.parametrize("dtype,quant", [(BF, False), (BF, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("page", [16, 128])
def test_shared_bad_pages_are_reported(L, gen, dtype, quant, page):
    s = Shared(gen, quant, [400, 300], [3, 2], [60, 5, 0, 20, 33], 1, 64, page, dtype)
    q = randn(gen, 5, 3, 64, dtype=dtype)
    lay = s.layer(L, 3, 1, 64, dtype)
    prefix_table, table = s.prefix_table.clone(), s.table.clone()
    hide = lambda n, col: torch.arange(n, device="cuda") // page == col  # noqa: E731
    prefix_table[0, 1], prefix_table[1, 300 // page], table[3, 0] = -1, s.c.n_pages, 2 ** 31 - 1
    out = lay.decode_shared(q, s.kv_len, table, s.prefix_len, prefix_table, s.cu)
    assert L.lola_attn_status() == (L.LOLA_ERR_DEVICE, L.LOLA_ATTN_BAD_PAGE)
    s.check(q, out, hidden={0: hide(400, 1), 1: hide(300, 300 // page), 5: hide(20, 0)})
    prefix_table.fill_(-1)                                    # nothing of the prefixes is left to see
    out = lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, prefix_table, s.cu)
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    every = lambda n: torch.ones(n, dtype=torch.bool, device="cuda")  # noqa: E731
    s.check(q, out, hidden={0: every(400), 1: every(300)})
    out = lay.decode_shared(q, s.kv_len, s.table, ints([2 ** 31 - 1, 300]), s.prefix_table[:, :300 // page], s.cu)
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    short = 300 // page * page
    s.check(q, out, hidden={0: torch.arange(400, device="cuda") >= short, 1: torch.arange(300, device="cuda") >= short})


@pytest.mark.parametrize("dtype,quant", [(BF, False), (BF, True), (F32, False)])
def test_shared_bad_offsets_are_reported(L, gen, dtype, quant):
    """A prefix with malformed offsets has no sequences; the others' are right where they see one prefix only."""
    s = Shared(gen, quant, [90, 80, 70], [2, 2, 2], [5, 6, 7, 8, 9, 10], 1, 64, 16, dtype)
    q = randn(gen, 6, 2, 64, dtype=dtype)
    lay = s.layer(L, 2, 1, 64, dtype)
    for cu, of in (([0, 2, 4, 7], [0, 0, 1, 1, -1, -1]), ([-3, 2, 4, 6], [-1, -1, 1, 1, 2, 2])):
        out = lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, ints(cu))
        assert L.lola_attn_status() == (L.LOLA_ERR_DEVICE, L.LOLA_ATTN_BAD_OFFSETS), cu
        s.of = of
        s.check(q, out)
    for cu in ([0, 5, 2, 6], [6, 4, 2, 0], [2 ** 31 - 1, 0, -2 ** 31, 5]):    # (any result)
        lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, ints(cu))
        assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_OFFSETS, cu


@pytest.mark.parametrize("dtype,quant", [(BF, False), (BF, True), (F32, False)])
def test_shared_strides_streams_and_graphs(L, gen, dtype, quant):
    """Wide queries, outputs head-major or in the queries' place; captured calls replayed on two streams, with other
    lengths, prefixes and sharing than they were captured with."""
    s = Shared(gen, quant, [700, 300], [3, 3], [130, 99, 64, 5, 0, 77], 2, 128, 64, dtype, width=20)
    lay = s.layer(L, 8, 2, 128, dtype)
    q = randn(gen, 6, 11, 128, dtype=dtype)[:, 3:11]
    args = (s.kv_len, s.table[:, :17], s.prefix_len, s.prefix_table[:, :15], s.cu)
    out = torch.empty(8, 6, 128, dtype=dtype, device="cuda").transpose(0, 1)
    lay.decode_shared(q, *args, out=out)
    same = q.clone()
    lay.decode_shared(same, *args, out=same)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = lay.decode_shared(q, *args, stream=stream)
    torch.cuda.synchronize()
    quiet(L)
    s.check(q, out)
    assert torch.equal(same, out) and torch.equal(other, out)
    graphs = []
    for _ in range(2):
        qs, n, m, cu, o = q.clone(), s.kv_len.clone(), s.prefix_len.clone(), s.cu.clone(), torch.zeros(6, 8, 128, dtype=dtype, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            lay.decode_shared(qs, n, s.table, m, s.prefix_table, cu, out=o)
        graphs.append((g, qs, n, m, cu, o))
    full = [x.clone() for x in s.c.k], [x.clone() for x in s.c.v]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for new in ([([1, 50, 63, 0, 0, 70], [64, 299], [0, 1, 6], [0, 1, 1, 1, 1, 1]), ([130, 99, 64, 5, 0, 77], [700, 0], [0, 6, 6], [0] * 6)],
                [([0, 0, 0, 0, 0, 1], [1, 1], [1, 3, 4], [-1, 0, 0, 1, -1, -1]), ([9, 9, 9, 5, 0, 9], [690, 300], [0, 2, 6], [0, 0, 1, 1, 1, 1])]):
        for (g, qs, n, m, cu, o), (lens, pre, c, _) in zip(graphs, new):
            qs.copy_(randn(gen, 6, 8, 128, dtype=dtype))
            n.copy_(ints(lens)), m.copy_(ints(pre)), cu.copy_(ints(c))
        torch.cuda.synchronize()
        for _ in range(3):
            for (g, *_), st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        quiet(L)
        for (g, qs, n, m, cu, o), (lens, pre, c, of) in zip(graphs, new):
            s.c.k, s.c.v = ([x[i][:z] for i, z in enumerate(pre + lens)] for x in full)
            s.of = of
            s.check(qs, o)


@pytest.mark.parametrize("dtype,quant,d", [(BF, True, 128), (BF, True, 64), (F32, True, 128)])
@pytest.mark.parametrize("up", [-60, -20, 15, 60])
def test_shared_powers_of_many_sizes(L, gen, dtype, quant, d, up):
    """Keys and values of magnitudes far from one, of many different ones in a block, and queries that make up for it."""
    s = Shared(gen, quant, [700], [5], [40, 3, 0, 130, 17], 1, d, 32, dtype)
    c = s.c
    for b, n in enumerate(c.lens):
        pos = torch.arange(n, device="cuda")
        f, g = (2.0 ** torch.randint(-m, m, (n, 1, 1), generator=gen, device="cuda").double() for m in (3, 12))
        c.k[b] = c.store("k", b, pos, (c.k[b] * f * 2.0 ** -up).float())
        c.v[b] = c.store("v", b, pos, (c.v[b] * g * 2.0 ** up).float())
    q = (0.3 * randn(gen, 5, 3, d, dtype=F32) * 2.0 ** up).to(dtype)
    lse = torch.empty(5, 3, dtype=F32, device="cuda")
    out = s.layer(L, 3, 1, d, dtype).decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, lse=lse)
    quiet(L)
    s.check(q, out, lse)


@pytest.mark.parametrize("dtype,quant", [(BF, False), (BF, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("what", ["step", "shared"])
@pytest.mark.parametrize("prefix,lens", [(6000, [4000, 100, 1, 2500]), (40000, [7] * 30), (130, [200] * 400)], ids=["few", "long", "many"])
def test_calls_after_waits_that_gave_up(L, gen, dtype, quant, what, prefix, lens):
    """A call whose waits gave up says so, ends, and leaves nothing behind: neither in a replay of a captured call nor
    in the next call in its workspace."""
    if what == "step" and not quant:
        pytest.skip("the plain cache's own test")
    s = Shared(gen, quant, [prefix], [len(lens)], lens, 1, 128, 64, dtype)
    lay = s.layer(L, 4, 1, 128, dtype)
    q = randn(gen, len(lens), 4, 128, dtype=dtype)
    out = torch.zeros_like(q)
    size = L.lola_shared_decode_workspace_bytes(lay.cfg, len(lens)) if what == "shared" else L.lola_paged_decode_workspace_bytes(lay.cfg)
    ws = torch.randint(0, 255, (size,), dtype=torch.uint8, device="cuda", generator=gen)

    def call():
        if what == "shared":
            lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, out=out, workspace=ws)
        else:
            lay.decode_step(q, s.kv_len, s.table, out=out, workspace=ws)

    call()
    quiet(L)
    want, gave_up = out.clone(), 0
    try:
        for block in (0, 1, 2, 3, 5, 8, 1000):
            L.lola_selftest_attn_wait(block)
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                call()
            for _ in range(2):
                out.fill_(7.0)
                g.replay()
                st, bits = L.lola_attn_status()
                assert bits in (0, L.LOLA_ATTN_TIMEOUT)
                gave_up += bits != 0
                assert bits or torch.equal(out, want), block
            L.lola_selftest_attn_wait(-1)
            out.fill_(7.0)
            call()
            quiet(L)
            assert torch.equal(out, want), block
    finally:
        L.lola_selftest_attn_wait(-1)
    assert gave_up > 0


# ---------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,quant,d,Hq,Hkv,page", [(BF, False, 128, 8, 2, 64), (BF, True, 128, 8, 2, 64), (F32, True, 64, 4, 1, 16),
                                                       (F32, False, 64, 4, 2, 16)])
def test_users_behind_one_prompt(L, gen, dtype, quant, d, Hq, Hkv, page):
    """A prompt is appended and attended, its samples go on from it with own tokens (rotated behind it), all steps over
    the one prompt: against a float64 form over the numbers that the cache holds."""
    P, users, steps = 150, 5, 4
    need = -(-P // page)
    cls = L.QuantizedAttention if quant else L.ExactAttention
    lay = cls.allocate(Hq, Hkv, d, need + users + 2, page, dtype)
    prefix_table = torch.randperm(need + users, generator=torch.Generator().manual_seed(3))[:need].to(torch.int32).cuda()[None]
    rest = [p for p in range(need + users) if p not in prefix_table[0].tolist()]
    table = ints(rest)[:, None].contiguous()
    freq = 10000.0 ** (-torch.arange(0, d, 2, device="cuda").float() / d)
    prefix_len = ints([P])

    def cached(row, n):
        pos = torch.arange(n, device="cuda")
        at = row.long()[pos // page], pos % page
        if not quant:
            return lay.k_pool[at[0], :, at[1]].double(), lay.v_pool[at[0], :, at[1]].double()
        byte = torch.uint8
        return tuple(decode(p.view(byte)[at[0], :, at[1]].view(E4), s.view(byte)[at[0], :, at[1]])
                     for p, s in ((lay.k_pool, lay.k_scale), (lay.v_pool, lay.v_scale)))

    q, k, v = (randn(gen, P, h, d, dtype=dtype) for h in (Hq, Hkv, Hkv))
    qr = lay.append(k, v, prefix_len, prefix_table, cu_new=ints([0, P]), q=q, inv_freq=freq)
    o = lay.prefill_paged(qr, ints([0, P]), prefix_len, prefix_table, P)
    quiet(L)
    K, V = cached(prefix_table[0], P)
    for i in (0, 1, 70, P - 1):
        check_attention(qr[i], [(K[:i + 1], V[:i + 1], None)], o[i], what=f"prompt row {i}")
    for t in range(1, steps + 1):
        q, k, v = (randn(gen, users, h, d, dtype=dtype) for h in (Hq, Hkv, Hkv))
        n = ints([t] * users)
        qr = lay.append(k, v, n, table, q=q, inv_freq=freq, positions=n + (P - 1))
        want, tol = rotated(q, n.double() + (P - 1), freq, "halves")
        check(qr, want, tol, "q")
        o = lay.decode_shared(qr, n, table, prefix_len, prefix_table)
        quiet(L)
        for b in range(users):
            check_attention(qr[b], [(K, V, None), (*cached(table[b], t), None)], o[b], what=f"step {t}, user {b}")


def test_two_calls_at_once_do_not_share(L, gen):
    """Calls of one layer on two streams, none waiting for the other."""
    s = Shared(gen, True, [5000], [20], [40] * 20, 2, 128, 64, BF)
    lay = s.layer(L, 8, 2, 128, BF)
    args = (s.kv_len, s.table, s.prefix_len, s.prefix_table)
    qs = [randn(gen, 20, 8, 128, dtype=BF) for _ in range(2)]
    want = [(lay.decode_shared(q, *args), lay.decode_step(q, s.kv_len, s.table)) for q in qs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append((lay.decode_shared(qs[i], *args), lay.decode_step(qs[i], s.kv_len, s.table)))
    torch.cuda.synchronize()
    quiet(L)
    for i in range(2):
        for a, b in got[i]:
            assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_both_forms_of_the_binding_give_the_same_bits(L, dtype, d, monkeypatch):
    """The calls through the marshalling module, and their Python form, which serves without it."""
    def run():
        g = torch.Generator(device="cuda").manual_seed(3)
        s = Shared(g, True, [90, 40], [2, 1], [70, 300, 1], 2, d, 16, dtype)
        lay = s.layer(L, 4, 2, d, dtype)
        n = 371
        rows, cu = randn(g, n, 8, d, dtype=dtype), offsets(s.lens)
        q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
        inv = torch.rand(d // 2, generator=g, device="cuda")
        qr = lay.append(k, v, s.kv_len, s.table, cu_new=cu, q=q, inv_freq=inv, pairs="neighbours")
        assert lay.append(k[:3], v[:3], s.kv_len, s.table) is None
        out = [qr, *lay.read(s.kv_len, s.table, n), lay.prefill_paged(qr, cu, s.kv_len, s.table, n), lay.decode_step(q[:3], s.kv_len, s.table),
               lay.decode_shared(q[:3], s.kv_len, s.table, s.prefix_len, s.prefix_table, s.cu)]
        io = Shared(g, False, [90, 40], [2, 1], [70, 300, 1], 2, d, 16, dtype)
        out.append(io.layer(L, 4, 2, d, dtype).decode_shared(q[:3], io.kv_len, io.table, io.prefix_len, io.prefix_table, io.cu))
        return out + [x.view(torch.uint8) for x in (lay.k_pool, lay.v_pool, lay.k_scale, lay.v_scale)]

    fast = run()
    assert L._fast is not L._Declines
    monkeypatch.setattr(L, "_fast", L._Declines)
    with pytest.warns(RuntimeWarning):
        slow = run()
    quiet(L)
    assert all(torch.equal(a, b) for a, b in zip(fast, slow)) and len(fast) == len(slow)


def test_refused_calls_say_what_is_wrong(L, gen):
    """Arguments that do not fit are refused by both forms, with nothing enqueued."""
    s = Shared(gen, True, [90, 40], [2, 1], [70, 30, 1], 2, 64, 16, BF)
    lay = s.layer(L, 4, 2, 64, BF)
    q, k = randn(gen, 3, 4, 64, dtype=BF), randn(gen, 3, 2, 64, dtype=BF)
    bad = [lambda: lay.decode_step(q[:2], s.kv_len, s.table), lambda: lay.decode_step(q.float(), s.kv_len, s.table),
           lambda: lay.decode_step(q, s.kv_len.long(), s.table), lambda: lay.decode_step(q, s.kv_len, s.table[:, ::2]),
           lambda: lay.append(k, k.float(), s.kv_len, s.table), lambda: lay.append(k, k, s.kv_len, s.table, q=q[:, :3]),
           lambda: lay.read(s.kv_len[:2], s.table, 5), lambda: lay.read(s.kv_len, s.table.cpu(), 5), lambda: lay.read(s.kv_len, s.table, -1),
           lambda: lay.prefill_paged(q, offsets([1, 1, 1]), s.kv_len, s.table),
           lambda: lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table),
           lambda: lay.decode_shared(q, s.kv_len, s.table, s.prefix_len[:1], s.prefix_table, s.cu),
           lambda: lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, s.cu[:2]),
           lambda: lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table.cpu(), s.cu),
           lambda: lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, s.cu, workspace=torch.empty(0, dtype=torch.uint8)),
           lambda: L.ExactAttention(4, 2, 64, BF, lay.k_pool, lay.v_pool)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: lay.append(k, k, s.kv_len, s.table, q=q),                      # queries without a rotation
              lambda: lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table[:1].expand(2, -1), s.cu),
              lambda: lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, s.prefix_table, s.cu,
                                        workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(L.LolaError):
            f()
    quiet(L)
