"""Exact attention on the GPU against plain float64 forms: packed prompts, the paged cache's append
and its single-token read, and a run of them together.  Bounds: tests/attn_parity.py."""
import math

import pytest
import torch

from attn_parity import Paged, attend, check, check_decode, check_prefill, ints, offsets, randn, rotated

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
    return torch.Generator(device="cuda").manual_seed(17)


def quiet(L):
    st, bits = L.lola_attn_status()
    assert st == 0 and bits == 0, bits


# ---------------------------------------------------------------------------------------
# packed prompts
# ---------------------------------------------------------------------------------------

LENS = [
    ([1], None), ([2], None), ([64], None), ([65], None), ([128], None), ([129], None), ([256], None), ([257], None),
    ([300, 1, 0, 63, 500], None),                              # an empty sequence inside
    ([0, 0, 7], None),
    ([5, 130, 1], [700, 130, 513]),                            # later pieces of prompts
    ([200, 3], [60, 0]),                                       # rows that see nothing; no keys at all
    ([140], [139]),                                            # the first row sees nothing
    ([1, 1, 1, 1, 1], [1, 2, 127, 128, 129]),
    ([31] * 40, None),                                         # many short prompts
]


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF, 128, 4, 2), (BF, 64, 5, 1), (F32, 64, 2, 2), (F32, 128, 3, 1)])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x[0][:5])) + (":" if x[1] else ""))
def test_prefill_lengths(L, gen, dtype, d, Hq, Hkv, lens):
    lq, lk = lens[0], lens[1] or lens[0]
    q = randn(gen, sum(lq), Hq, d, dtype=dtype)
    k, v = randn(gen, sum(lk), Hkv, d, dtype=dtype), randn(gen, sum(lk), Hkv, d, dtype=dtype)
    lse = torch.empty(Hq, sum(lq), dtype=F32, device="cuda")
    lay = L.ExactAttention(Hq, Hkv, d, dtype)
    out = lay.prefill(q, k, v, offsets(lq), offsets(lk) if lens[1] else None, lse=lse)
    quiet(L)
    check_prefill(q, k, v, lq, lk, out, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [384, 512, 640, 768, 896, 1024, 1152])
def test_prefill_every_ring_length(L, gen, d, n):
    """Many sequences of three to nine key blocks: the ring of key and value blocks ends at every one
    of its stages (at four blocks of d = 64 the whole sequence fits the ring)."""
    B, H = 24, 4
    q, k, v = (randn(gen, B * n, H, d, dtype=BF) for _ in range(3))
    out = L.ExactAttention(H, H, d).prefill(q, k, v, offsets([n] * B))
    quiet(L)
    check_prefill(q, k, v, [n] * B, [n] * B, out, heads=[0, 3], rows=[0, 127, 128, 255, 256, n - 129, n - 1])


@pytest.mark.parametrize("dtype,d,Hq,Hkv,n", [(BF, 128, 8, 1, 2100), (BF, 64, 4, 4, 3001), (F32, 64, 2, 1, 1500)])
def test_prefill_longer(L, gen, dtype, d, Hq, Hkv, n):
    """Many key blocks; scores grow along the sequence, so the running maximum moves all the time."""
    q, v = randn(gen, n, Hq, d, dtype=dtype), randn(gen, n, Hkv, d, dtype=dtype)
    k = (randn(gen, n, Hkv, d, dtype=F32) * torch.linspace(0.1, 6.0, n, device="cuda")[:, None, None]).to(dtype)
    out = L.ExactAttention(Hq, Hkv, d, dtype).prefill(q, k, v, offsets([n]))
    quiet(L)
    check_prefill(q, k, v, [n], [n], out)


def test_prefill_long_sampled(L, gen):
    """40000 tokens, every kind of row sampled, on two heads."""
    n, Hq, Hkv, d = 40000, 4, 2, 128
    q, k, v = (randn(gen, n, h, d, dtype=BF) for h in (Hq, Hkv, Hkv))
    lse = torch.empty(Hq, n, dtype=F32, device="cuda")
    out = L.ExactAttention(Hq, Hkv, d).prefill(q, k, v, offsets([n]), lse=lse)
    quiet(L)
    check_prefill(q, k, v, [n], [n], out, lse, heads=[0, 3],
                  rows=[0, 1, 127, 128, 255, 256, 257, 8191, 8192, 20011, 39935, 39936, 39998, 39999])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [None, 0.02, 1.0])
def test_prefill_scales(L, gen, dtype, scale):
    n, d = 333, 64
    q, k, v = (randn(gen, n, 2, d, dtype=dtype) for _ in range(3))
    out = L.ExactAttention(2, 2, d, dtype, scale=scale).prefill(q, k, v, offsets([n]))
    check_prefill(q, k, v, [n], [n], out, scale=scale)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 128)])
def test_prefill_strides(L, gen, dtype, d):
    """Rows of one projection, head-major tensors, an output inside a wider one; the rest of that
    one stays as it was."""
    lens, Hq, Hkv = [130, 61], 6, 2
    n = sum(lens)
    rows = randn(gen, n, Hq + 2 * Hkv, d, dtype=dtype)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    lay = L.ExactAttention(Hq, Hkv, d, dtype)
    wide = torch.full((n, Hq + 3, d), 7.0, dtype=dtype, device="cuda")
    out = lay.prefill(q, k, v, offsets(lens), out=wide[:, 2:2 + Hq])
    check_prefill(q, k, v, lens, lens, out)
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + Hq:] == 7).all())
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]     # [H, n, d] in memory
    out2 = lay.prefill(*hm, offsets(lens), out=torch.empty(Hq, n, d, dtype=dtype, device="cuda").transpose(0, 1))
    assert torch.equal(out, out2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_leaves_rows_outside_the_sequences(L, gen, dtype):
    """Rows before the first and behind the last sequence: not read into any result, not written."""
    lens, d, Hq, Hkv = [100, 37], 128, 2, 1
    n = 11 + sum(lens) + 90
    q, k, v = (randn(gen, n, h, d, dtype=dtype) for h in (Hq, Hkv, Hkv))
    for t in (q, k, v):
        t[:11] = math.nan
        t[11 + sum(lens):] = math.nan
    out = torch.full((n, Hq, d), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((Hq, n), 5.0, dtype=F32, device="cuda")
    L.ExactAttention(Hq, Hkv, d, dtype).prefill(q, k, v, offsets(lens, 11), out=out, lse=lse)
    quiet(L)
    check_prefill(q, k, v, lens, lens, out, lse, start=11, start_k=11)
    for t in (out[:11], out[11 + sum(lens):], lse[:, :11], lse[:, 11 + sum(lens):]):
        assert bool((t == 5).all())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_prefill_values_that_are_not_finite_reach_only_who_sees_them(L, gen, dtype, d):
    """NaN and infinities in keys and values at several places of the tiles: rows before the token and
    other sequences are untouched, rows from it on show them."""
    lens, Hq, Hkv = [400, 290], 2, 1
    n = sum(lens)
    q, k, v = (randn(gen, n, h, d, dtype=dtype) for h in (Hq, Hkv, Hkv))
    for at, x in ((130, math.inf), (255, math.nan), (256, -math.inf), (399, math.nan)):
        v[at, 0, at % d] = x
    v[270, 0, :3] = math.inf
    k[399, 0, 5] = math.nan
    v[400 + 64, 0, 1] = math.nan
    v[400 + 289] = math.nan
    lay = L.ExactAttention(Hq, Hkv, d, dtype)
    out = lay.prefill(q, k, v, offsets(lens))
    quiet(L)
    r = torch.arange(n, device="cuda")
    first = r < 399                                           # (row 399 sees a NaN key: all of it is NaN)
    assert bool(torch.isnan(out[399]).all())
    o2 = out.clone()
    k2 = k.clone()
    k2[399] = 0
    q2 = torch.cat([q[:399], q[400:]])
    check_prefill(q2, torch.cat([k2[:399], k2[400:]]), torch.cat([v[:399], v[400:]]), [399, 290], [399, 290],
                  torch.cat([o2[:399], o2[400:]]))
    assert bool(torch.isfinite(out[:130][first[:130]]).all())


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_short_sequences_beside_a_long_one(L, gen, d):
    """A long sequence makes the whole call take two query tiles per CTA: the short ones' edges (lengths
    around the tiles, pieces with earlier keys, rows that see nothing, values that are not finite,
    rows of a wider tensor, rows outside the sequences) under that form."""
    lq = [20000, 512, 384, 1, 640, 257, 0, 130, 100, 3]
    lk = [20000, 512, 384, 700, 640, 300, 5, 129, 60, 0]
    Hq, Hkv, nq, nk = 16, 4, sum(lq) + 40, sum(lk) + 40
    rows = randn(gen, nq, Hq + 3, d, dtype=BF)
    q = rows[:, 2:2 + Hq]
    k, v = randn(gen, nk, Hkv, d, dtype=BF), randn(gen, nk, Hkv, d, dtype=BF)
    for t, used in ((rows, sum(lq)), (k, sum(lk)), (v, sum(lk))):
        t[:17] = math.nan
        t[17 + used:] = math.nan
    a = 17 + 20000                                              # the sequence of 512
    v[a + 130, 0, 3], v[a + 255, 1, 4], v[a + 300, 2, 5] = math.inf, math.nan, -math.inf
    b = a + 512 + 384 + 700                                     # ... of 640
    v[b + 5, 3, 0], v[b + 639, 0] = math.nan, math.nan
    out = torch.full((nq, Hq, d), 5.0, dtype=BF, device="cuda")
    lse = torch.full((Hq, nq), 5.0, dtype=F32, device="cuda")
    L.ExactAttention(Hq, Hkv, d).prefill(q, k, v, offsets(lq, 17), offsets(lk, 17), out=out, lse=lse)
    quiet(L)
    check_prefill(q, k, v, lq, lk, out, lse, start=17, start_k=17, heads=[0, 5, 10, 15],
                  rows=[0, 1, 2, 60, 99, 127, 128, 129, 130, 131, 254, 255, 256, 257, 300, 301, 383, 511, 512, 638, 639,
                        10000, 19967, 19968, 19999])
    for t in (out[:17], out[17 + sum(lq):], lse[:, :17], lse[:, 17 + sum(lq):]):
        assert bool((t == 5).all())


def test_prefill_offsets_past_32_bits(L, gen):
    """Rows so far apart that element offsets pass 2^31."""
    n, d, apart = 700, 128, 3_200_000
    base = torch.zeros(n * apart, dtype=BF, device="cuda")
    k = base.as_strided((n, 1, d), (apart, d, 1))
    v = base.as_strided((n, 1, d), (apart, d, 1), 256)
    q = base.as_strided((n, 2, d), (apart, d, 1), 1024)
    out = base.as_strided((n, 2, d), (apart, d, 1), 2048)
    for t in (k, v, q):
        t.copy_(randn(gen, *t.shape, dtype=BF))
    L.ExactAttention(2, 1, d).prefill(q, k, v, offsets([n]), out=out)
    quiet(L)
    check_prefill(q, k, v, [n], [n], out)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_bad_offsets_are_reported(L, gen, dtype):
    """Offsets that decrease or pass the rows: the sequence counts as empty, its neighbours do not."""
    n, d = 200, 64
    q, k, v = (randn(gen, n, 1, d, dtype=dtype) for _ in range(3))
    lay = L.ExactAttention(1, 1, d, dtype)
    out = torch.full((n, 1, d), 3.0, dtype=dtype, device="cuda")
    lay.prefill(q, k, v, ints([0, 50, 40]), out=out)
    st, bits = L.lola_attn_status()
    assert st == L.LOLA_ERR_DEVICE and bits == L.LOLA_ATTN_BAD_OFFSETS
    check_prefill(q[:50], k[:50], v[:50], [50], [50], out[:50])
    assert bool((out[50:] == 3).all())
    quiet(L)                                                  # reading clears
    for cu in ([0, 201], [-1, 50], [5, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1]):
        out.fill_(3.0)
        lay.prefill(q, k, v, ints(cu), out=out)
        assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_OFFSETS
        assert bool((out == 3).all())
    # bad key offsets: the queries see nothing
    lay.prefill(q, k, v, ints([0, 50]), ints([0, 201]), out=out)
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_OFFSETS
    assert bool((out[:50] == 0).all()) and bool((out[50:] == 3).all())


def test_prefill_on_streams_and_in_graphs(L, gen):
    """Two graphs of one layer replayed on two streams at once, with other inputs and lengths than
    were captured; and a call on a stream that is not the current one."""
    d, Hq, Hkv, cap = 128, 4, 2, 700
    lay = L.ExactAttention(Hq, Hkv, d)
    graphs = []
    for i in range(2):
        q, k, v = (randn(gen, cap, h, d, dtype=BF) for h in (Hq, Hkv, Hkv))
        cu, out = offsets([cap, 0]), torch.zeros(cap, Hq, d, dtype=BF, device="cuda")
        lay.prefill(q, k, v, cu, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lay.prefill(q, k, v, cu, out=out)
        graphs.append((g, q, k, v, cu, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    lens = [[333, 200], [5, 650]]
    for (g, q, k, v, cu, out), n in zip(graphs, lens):
        for t in (q, k, v):
            t.copy_(randn(gen, *t.shape, dtype=BF))
        cu.copy_(offsets(n))
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    quiet(L)
    for (g, q, k, v, cu, out), n in zip(graphs, lens):
        check_prefill(q, k, v, n, n, out)
    q, k, v = (randn(gen, 90, h, d, dtype=BF) for h in (Hq, Hkv, Hkv))
    torch.cuda.synchronize()
    for s in (streams[0], streams[0].cuda_stream):
        out = lay.prefill(q, k, v, offsets([90]), stream=s)
        streams[0].synchronize()
        check_prefill(q, k, v, [90], [90], out)


# ---------------------------------------------------------------------------------------
# the paged cache: one token per sequence
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF, 128, 8, 2), (BF, 64, 6, 6), (BF, 128, 5, 1), (F32, 64, 4, 2),
                                            (F32, 128, 3, 3)])
@pytest.mark.parametrize("page,lens", [(16, [1]), (16, [15, 16, 17, 0, 33]), (32, [63, 64, 65, 1]), (64, [127, 128, 129]),
                                       (128, [1, 300, 0, 513]), (256, [1000, 255, 257]), (16, [2000, 5])])
def test_decode_lengths(L, gen, dtype, d, Hq, Hkv, page, lens):
    c = Paged(gen, lens, Hkv, d, page, dtype, junk=math.nan)
    q = randn(gen, len(lens), Hq, d, dtype=dtype)
    lse = torch.empty(len(lens), Hq, dtype=F32, device="cuda")
    lay = L.ExactAttention(Hq, Hkv, d, dtype, c.k_pool, c.v_pool)
    out = lay.decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    check_decode(q, c, out, lse)


@pytest.mark.parametrize("dtype,Hq,Hkv", [(BF, 16, 1), (BF, 17, 1), (BF, 40, 1), (BF, 64, 2), (F32, 16, 1), (F32, 20, 1)])
def test_decode_many_query_heads_per_key_head(L, gen, dtype, Hq, Hkv):
    """Groups of 16 rows and more than one group of a key head."""
    c = Paged(gen, [700, 64], Hkv, 128, 64, dtype, junk=math.nan)
    q = randn(gen, 2, Hq, 128, dtype=dtype)
    lse = torch.empty(2, Hq, dtype=F32, device="cuda")
    out = L.ExactAttention(Hq, Hkv, 128, dtype, c.k_pool, c.v_pool).decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    check_decode(q, c, out, lse)


@pytest.mark.parametrize("dtype,d,n", [(BF, 128, 70001), (BF, 64, 30000), (F32, 64, 20001)])
def test_decode_long(L, gen, dtype, d, n):
    """One long sequence beside short ones: cut into pieces and joined; keys grow along it."""
    lens = [3, n, 200]
    c = Paged(gen, lens, 1, d, 128, dtype)
    c.k[1] = (c.k[1].float() * torch.linspace(0.1, 4.0, n, device="cuda")[:, None, None]).to(dtype)
    c.put(1, torch.arange(n, device="cuda"), c.k[1], c.v[1])
    q = randn(gen, 3, 4, d, dtype=dtype)
    lse = torch.empty(3, 4, dtype=F32, device="cuda")
    lay = L.ExactAttention(4, 1, d, dtype, c.k_pool, c.v_pool)
    out = lay.decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    check_decode(q, c, out, lse)
    for _ in range(3):                                        # the join's order is fixed
        assert torch.equal(out, lay.decode_step(q, c.kv_len, c.table))


def test_decode_many_sequences(L, gen):
    """More sequences than threads of a CTA, most of them empty or short."""
    lens = [(i * 37) % 90 if i % 3 else 0 for i in range(1500)]
    c = Paged(gen, lens, 1, 64, 16, BF, junk=math.nan)
    q = randn(gen, len(lens), 2, 64, dtype=BF)
    out = L.ExactAttention(2, 1, 64, BF, c.k_pool, c.v_pool).decode_step(q, c.kv_len, c.table)
    quiet(L)
    c.lens = lens
    check_decode(q, c, out)


def test_decode_values_that_are_not_finite(L, gen):
    """A NaN or infinite value shows in its own sequence and head only; the rest of the pool is NaN."""
    c = Paged(gen, [100, 100, 70], 2, 128, 32, BF, junk=math.nan)
    c.v[1][40, 0, 3] = math.inf
    c.v[1][41, 0, 4] = math.nan
    c.put(1, torch.arange(100, device="cuda"), c.k[1], c.v[1])
    q = randn(gen, 3, 4, 128, dtype=BF)
    out = L.ExactAttention(4, 2, 128, BF, c.k_pool, c.v_pool).decode_step(q, c.kv_len, c.table)
    quiet(L)
    check_decode(q, c, out)


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 128), (F32, 32)])
def test_decode_bad_pages_are_reported(L, gen, dtype, page):
    """A page outside the pool: its tokens are not seen, the others are; lengths past the table."""
    lens = [300, 200]
    c = Paged(gen, lens, 1, 64, page, dtype, junk=math.nan)
    q = randn(gen, 2, 2, 64, dtype=dtype)
    lay = L.ExactAttention(2, 1, 64, dtype, c.k_pool, c.v_pool)
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
    out = lay.decode_step(q, c.kv_len, table)                 # nothing is left to see
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    assert bool((out == 0).all())
    c2 = Paged(gen, [2 * page, 2 * page], 1, 64, page, dtype)
    lay2 = L.ExactAttention(2, 1, 64, dtype, c2.k_pool, c2.v_pool)
    out = lay2.decode_step(q, ints([2 * page + 1, 2 ** 31 - 1]), c2.table)
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    check_decode(q, c2, out)
    quiet(L)


def test_decode_negative_lengths_are_empty(L, gen):
    c = Paged(gen, [50, 60], 1, 64, 16, BF)
    q = randn(gen, 2, 1, 64, dtype=BF)
    lse = torch.zeros(2, 1, dtype=F32, device="cuda")
    out = L.ExactAttention(1, 1, 64, BF, c.k_pool, c.v_pool).decode_step(q, ints([-5, 60]), c.table, lse=lse)
    quiet(L)
    assert bool((out[0] == 0).all()) and float(lse[0, 0]) == -math.inf
    c.lens = [0, 60]
    c.k[0], c.v[0] = c.k[0][:0], c.v[0][:0]
    check_decode(q, c, out)


def test_decode_pool_past_32_bits(L, gen):
    """A pool of more than 2^31 elements, its last pages used."""
    page, Hkv, d = 256, 2, 128
    n_pages = (1 << 31) // (page * Hkv * d) + 40
    k_pool = torch.empty(n_pages, Hkv, page, d, dtype=BF, device="cuda")
    v_pool = torch.empty(n_pages, Hkv, page, d, dtype=BF, device="cuda")
    n = 700
    k, v = randn(gen, n, Hkv, d, dtype=BF), randn(gen, n, Hkv, d, dtype=BF)
    table = ints([[n_pages - 1, n_pages - 30, n_pages - 7]])
    lay = L.ExactAttention(4, Hkv, d, BF, k_pool, v_pool)
    lay.append(k, v, ints([n]), table, cu_new=offsets([n]))
    q = randn(gen, 1, 4, d, dtype=BF)
    out = lay.decode_step(q, ints([n]), table)
    quiet(L)
    for h in range(4):
        o, _, tol, _ = attend(q[0, h][None], k[:, h // 2], v[:, h // 2], torch.ones(1, n, dtype=torch.bool, device="cuda"))
        check(out[0, h][None], o, tol, f"head {h}")
    assert torch.equal(k_pool[n_pages - 1, :, 3], k[3]) and torch.equal(v_pool[n_pages - 7, 1, 700 - 513], v[699, 1])


def test_decode_strides_and_graphs(L, gen):
    """Queries of a wider tensor, an output head-major, two captured steps replayed on two streams
    with other lengths; the table a slice of a wider one."""
    lens = [130, 999, 64, 5]
    c = Paged(gen, lens, 2, 128, 64, BF, junk=math.nan, width=20)
    wide = randn(gen, 4, 11, 128, dtype=BF)
    q = wide[:, 3:11]
    lay = L.ExactAttention(8, 2, 128, BF, c.k_pool, c.v_pool)
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
    full_k, full_v = c.k, c.v
    for (g, qs, n, o), x in zip(graphs, new):
        c.lens, c.k, c.v = x, [t[:m] for t, m in zip(full_k, x)], [t[:m] for t, m in zip(full_v, x)]
        check_decode(qs, c, o)


# ---------------------------------------------------------------------------------------
# prompts over the paged cache
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF, 128, 4, 2), (BF, 64, 5, 1), (F32, 64, 2, 2), (F32, 128, 3, 1)])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens,keys", [([1], [1]), ([300, 1, 0, 63, 500], None), ([5, 130, 1, 17], [700, 130, 1300, 16]),
                                       ([200, 3, 40], [60, 0, 33]), ([700] * 12, None), ([31] * 40, [257] * 40)])
def test_paged_prefill_equals_packed(L, gen, dtype, d, Hq, Hkv, page, lens, keys):
    """The same bits as over the gathered rows (the same form of the kernel: it depends on the totals),
    those being checked against float64 for themselves; unused slots and pages hold NaN."""
    keys = keys or lens
    c = Paged(gen, keys, Hkv, d, page, dtype, junk=math.nan)
    lay = L.ExactAttention(Hq, Hkv, d, dtype, c.k_pool, c.v_pool)
    q = randn(gen, sum(lens), Hq, d, dtype=dtype)
    k, v = torch.cat(c.k), torch.cat(c.v)
    lse, want_lse = (torch.empty(Hq, sum(lens), device="cuda") for _ in range(2))
    out = lay.prefill_paged(q, offsets(lens), c.kv_len, c.table, sum(keys), lse=lse)
    want = lay.prefill(q, k, v, offsets(lens), offsets(keys), lse=want_lse)
    quiet(L)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    if page == 32:
        check_prefill(q, k, v, lens, keys, out)
        unknown = lay.prefill_paged(q, offsets(lens), c.kv_len, c.table)     # (perhaps the other form)
        quiet(L)
        check_prefill(q, k, v, lens, keys, unknown)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_paged_prefill_longer(L, gen, dtype, d):
    """Every place of the ring many times over, several items a CTA."""
    lens, keys = [1500, 2048, 700, 130] * 5, [4000, 2048, 5003, 131] * 5
    c = Paged(gen, keys, 2, d, 64, dtype)
    lay = L.ExactAttention(8, 2, d, dtype, c.k_pool, c.v_pool)
    q = randn(gen, sum(lens), 8, d, dtype=dtype)
    for tk in (sum(keys), 0):
        out = lay.prefill_paged(q, offsets(lens), c.kv_len, c.table, tk)
        quiet(L)
        k, v = torch.cat(c.k), torch.cat(c.v)
        if tk:
            assert torch.equal(out, lay.prefill(q, k, v, offsets(lens), offsets(keys)))
        else:
            check_prefill(q, k, v, lens, keys, out, heads=[0, 7], rows=[0, 1, 127, 128, 600, 1300, 1499, 2047])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
def test_paged_prefill_values_that_are_not_finite(L, gen, dtype, d):
    lens = [200, 300]
    c = Paged(gen, lens, 1, d, 16, dtype, junk=math.inf)
    for b, pos, x in ((0, 150, math.inf), (1, 131, math.nan), (1, 299, -math.inf)):
        c.v[b][pos, 0, 3] = x
        c.put(b, torch.tensor([pos], device="cuda"), c.k[b][pos:pos + 1], c.v[b][pos:pos + 1])
    lay = L.ExactAttention(2, 1, d, dtype, c.k_pool, c.v_pool)
    q = randn(gen, 500, 2, d, dtype=dtype)
    out = lay.prefill_paged(q, offsets(lens), c.kv_len, c.table, 500)
    want = lay.prefill(q, torch.cat(c.k), torch.cat(c.v), offsets(lens))
    quiet(L)
    assert torch.equal(out.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    assert out[:150].isfinite().all() and out[150:200, :, 3].isinf().all() and out[200:331].isfinite().all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_paged_prefill_bad_pages_are_reported(L, gen, dtype, d, page):
    """A page outside the cache stands for zeros; the other sequences do not notice.  A length beyond
    the table counts as the table's."""
    lens = [2 * page + 5, 300, 3 * page]
    c = Paged(gen, lens, 2, d, page, dtype)
    lay = L.ExactAttention(4, 2, d, dtype, c.k_pool, c.v_pool)
    q = randn(gen, sum(lens), 4, d, dtype=dtype)
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[0, 1] = bad
        out = lay.prefill_paged(q, offsets(lens), c.kv_len, table, sum(lens))
        assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
        k, v = c.k[0].clone(), c.v[0].clone()
        k[page:2 * page] = 0
        v[page:2 * page] = 0
        want = lay.prefill(q, torch.cat([k, *c.k[1:]]), torch.cat([v, *c.v[1:]]), offsets(lens))
        quiet(L)
        assert torch.equal(out, want)
    full = c.table.shape[1] * page
    one = ints([full + 9])
    i = max(range(3), key=lambda b: -(-lens[b] // page))
    if lens[i] == full:
        got = lay.prefill_paged(q[:7], offsets([7]), one, c.table[i:i + 1])
        assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
        assert torch.equal(got, lay.prefill_paged(q[:7], offsets([7]), ints([full]), c.table[i:i + 1]))
        quiet(L)


def test_paged_prefill_in_a_graph_with_other_lengths(L, gen):
    """A server's step: pieces of prompts appended and attended, captured once, replayed as the lengths
    grow; a table that is part of a wider one, queries a part of wider rows, rows behind the last
    sequence left."""
    Hq, Hkv, d, page, B, T = 8, 2, 128, 64, 3, 96
    lay = L.ExactAttention.allocate(Hq, Hkv, d, 40, page)
    table = ints([[13 * b + i for i in range(13)] + [-1] * 4 for b in range(B)])[:, :13]
    rows = torch.empty(B * T, Hq + 2 * Hkv, d, dtype=BF, device="cuda")
    cu, lens = ints([0] * (B + 1)), ints([0] * B)
    out = torch.full((B * T, Hq, d), 5.0, dtype=BF, device="cuda")
    inv = _freq(d)

    def step():
        q = lay.append(rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], lens, table, cu_new=cu, q=rows[:, :Hq], inv_freq=inv)
        lay.prefill_paged(q, cu, lens, table, out=out)
        return q

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = step()
    K, V = ([torch.empty(0, Hkv, d, dtype=BF, device="cuda") for _ in range(B)] for _ in range(2))
    done = [0] * B
    for new in ([96, 50, 1], [1, 96, 0], [90, 1, 96], [96, 96, 96]):
        done = [x + n for x, n in zip(done, new)]
        rows.copy_(randn(gen, B * T, Hq + 2 * Hkv, d, dtype=BF))
        cu.copy_(offsets(new))
        lens.copy_(ints(done))
        out.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        quiet(L)
        r = 0
        for b, n in enumerate(new):
            pos = torch.arange(done[b] - n, done[b], device="cuda")
            K[b] = torch.cat([K[b], lay.k_pool[table[b].long()[pos // page], :, pos % page]])
            V[b] = torch.cat([V[b], rows[r:r + n, Hq + Hkv:]])
            r += n
        check_prefill(q[:r], torch.cat(K), torch.cat(V), new, done, out[:r])
        assert (out[r:] == 5.0).all()


def test_kernels_behind_copies_sets_and_other_streams(L, gen):
    """The kernels start behind whatever the stream did last: copies, memsets, kernels of another stream,
    each other, in a stream and in a graph; every result is that of the same calls one by one."""
    lens, page = [300, 77, 1], 16
    c = Paged(gen, lens, 2, 64, page, BF)
    lay = L.ExactAttention(4, 2, 64, BF, c.k_pool, c.v_pool)
    src = [(randn(gen, 3, 4, 64, dtype=BF), randn(gen, 3, 2, 64, dtype=BF), randn(gen, 3, 2, 64, dtype=BF)) for _ in range(4)]
    q, k, v = (torch.empty_like(x) for x in src[0])
    cu, inv = offsets([1, 1, 1]), _freq(64)
    out = [torch.empty_like(q) for _ in range(3)]
    side = torch.cuda.Stream()

    def step(wait=lambda: None):
        out[0].zero_()                                         # a memset
        q.copy_(src_now[0])                                    # copies
        k.copy_(src_now[1])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            v.copy_(src_now[2].mul(0.5))                       # another stream's kernels
        torch.cuda.current_stream().wait_stream(side)
        wait()
        qr = lay.append(k, v, c.kv_len, c.table, q=q, inv_freq=inv)
        wait()
        lay.decode_step(qr, c.kv_len, c.table, out=out[0])
        wait()
        lay.prefill_paged(qr, cu, c.kv_len, c.table, out=out[1])
        wait()
        lay.decode_step(out[0], c.kv_len, c.table, out=out[2])
        wait()
        out[1].mul_(2.0)                                       # an ordinary kernel behind them

    src_now = [torch.empty_like(x) for x in src[0]]
    torch.cuda.synchronize()
    want = []
    for x in src:
        for a, b in zip(src_now, x):
            a.copy_(b)
        step(torch.cuda.synchronize)
        want.append([o.clone() for o in out])
    main = torch.cuda.Stream()
    with torch.cuda.stream(main):
        for x, w in zip(src, want):
            for a, b in zip(src_now, x):
                a.copy_(b)
            step()
            assert all(torch.equal(a, b) for a, b in zip(out, w))
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=main):
            step()
            step()
        for x, w in zip(src, want):
            for a, b in zip(src_now, x):
                a.copy_(b)
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, w))
    torch.cuda.synchronize()
    quiet(L)


# ---------------------------------------------------------------------------------------
# the paged cache: rotation and append
# ---------------------------------------------------------------------------------------

def _freq(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


@pytest.mark.parametrize("dtype,d,rot", [(BF, 128, 128), (BF, 64, 64), (BF, 128, 48), (F32, 128, 128), (F32, 64, 16)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("new,before", [([1, 1, 1], [0, 15, 4000]), ([5, 0, 200], [11, 3, 0]), ([1], [0])])
def test_append(L, gen, dtype, d, rot, pairs, new, before):
    Hq, Hkv, page = 6, 2, 16
    total = [a + b for a, b in zip(new, before)]
    c = Paged(gen, total, Hkv, d, page, dtype)
    k0, v0 = c.k_pool.clone(), c.v_pool.clone()
    t = sum(new)
    rows = randn(gen, t, Hq + 2 * Hkv, d, dtype=dtype)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    lay = L.ExactAttention(Hq, Hkv, d, dtype, c.k_pool, c.v_pool)
    inv = _freq(rot)
    cu = None if new == [1] * len(new) else offsets(new)
    qr = lay.append(k, v, c.kv_len, c.table, cu_new=cu, q=q, inv_freq=inv, pairs=pairs)
    quiet(L)
    r = 0
    for b, n in enumerate(new):
        pos = torch.arange(before[b], total[b], device="cuda")
        pages = c.table[b].long()[pos // page] if n else pos
        y, tol = rotated(q[r:r + n], pos, inv, pairs)
        check(qr[r:r + n], y, tol + 1e-30, "q")
        y, tol = rotated(k[r:r + n], pos, inv, pairs)
        check(c.k_pool[pages, :, pos % page], y, tol + 1e-30, "k")
        assert torch.equal(c.v_pool[pages, :, pos % page], v[r:r + n])
        k0[pages, :, pos % page] = c.k_pool[pages, :, pos % page]
        v0[pages, :, pos % page] = v[r:r + n]
        r += n
    assert torch.equal(c.k_pool, k0) and torch.equal(c.v_pool, v0)       # nothing else was written


def test_append_far_positions(L, gen):
    """Positions up to 2^31 - 1: the angle's reduction loses nothing."""
    pos = [0, 1, 131071, 1 << 20, 16777217, (1 << 31) - 1]
    n, d = len(pos), 128
    c = Paged(gen, [n], 1, d, 16, F32)
    q, k = randn(gen, n, 1, d, dtype=F32), randn(gen, n, 1, d, dtype=F32)
    lay = L.ExactAttention(1, 1, d, F32, c.k_pool, c.v_pool)
    inv = _freq(d)
    qr = lay.append(k, k, c.kv_len, c.table, cu_new=offsets([n]), q=q, inv_freq=inv, positions=ints(pos))
    quiet(L)
    y, tol = rotated(q, torch.tensor(pos, device="cuda"), inv, "halves")
    # (the kernel's turn w / 2 pi is a double product: 2^31 turns of it are 2^31 2^-53 off, and the
    # oracle's own double angle as much)
    tol = tol + (q.double()[..., :64].abs() + q.double()[..., 64:].abs()).repeat(1, 1, 2) * (4 * math.pi * 2.0 ** -21)
    check(qr, y, tol, "far positions")
    near = torch.tensor(pos, device="cuda") < 1 << 21
    y, tol = rotated(q[near], torch.tensor(pos, device="cuda")[near], inv, "halves")
    check(qr[near], y, tol, "near positions")


def test_append_without_rotation_and_in_place(L, gen):
    c = Paged(gen, [40, 3], 2, 64, 32, BF)
    k, v = randn(gen, 43, 2, 64, dtype=BF), randn(gen, 43, 2, 64, dtype=BF)
    lay = L.ExactAttention(4, 2, 64, BF, c.k_pool, c.v_pool)
    assert lay.append(k, v, c.kv_len, c.table, cu_new=offsets([40, 3])) is None
    quiet(L)
    pos = torch.arange(40, device="cuda")
    assert torch.equal(c.k_pool[c.table[0].long()[pos // 32], :, pos % 32], k[:40])
    q = randn(gen, 43, 4, 64, dtype=BF)
    want = lay.append(k, v, c.kv_len, c.table, cu_new=offsets([40, 3]), q=q, inv_freq=_freq(64))
    q2 = q.clone()
    got = lay.append(k, v, c.kv_len, c.table, cu_new=offsets([40, 3]), q=q2, inv_freq=_freq(64), q_out=q2)
    assert got is q2 and torch.equal(q2, want)


def test_append_padded_batches(L, gen):
    """Empty sequences of a padded batch and rows behind the last sequence: nothing is written."""
    c = Paged(gen, [20, 9], 1, 64, 16, BF)
    lay = L.ExactAttention(2, 1, 64, BF, c.k_pool, c.v_pool)
    k, v, q = randn(gen, 2, 1, 64, dtype=BF), randn(gen, 2, 1, 64, dtype=BF), randn(gen, 2, 2, 64, dtype=BF)
    k0, v0 = c.k_pool.clone(), c.v_pool.clone()
    qo = torch.full_like(q, 9.0)
    lay.append(k, v, ints([0, 9]), c.table, q=q, inv_freq=_freq(64), q_out=qo)
    quiet(L)
    assert bool((qo[0] == 9).all()) and not bool((qo[1] == 9).any())
    page = int(c.table[1, 0])
    k0[page, :, 8], v0[page, :, 8] = c.k_pool[page, :, 8], v[1]
    assert torch.equal(c.k_pool, k0) and torch.equal(c.v_pool, v0)
    # 12 rows, of which 2 .. 7 are new tokens of the two sequences
    k, v, q = randn(gen, 12, 1, 64, dtype=BF), randn(gen, 12, 1, 64, dtype=BF), randn(gen, 12, 2, 64, dtype=BF)
    qo = torch.full_like(q, 9.0)
    lay.append(k, v, c.kv_len, c.table, cu_new=ints([2, 5, 8]), q=q, inv_freq=_freq(64), q_out=qo)
    quiet(L)
    assert bool((qo[:2] == 9).all()) and bool((qo[8:] == 9).all()) and not bool((qo[2:8] == 9).any())
    for b, (lo, n) in enumerate(((2, 20), (5, 9))):
        pos = torch.arange(n - 3, n, device="cuda")
        pages = c.table[b].long()[pos // 16]
        v0[pages, :, pos % 16] = v[lo:lo + 3]
    assert torch.equal(c.v_pool, v0)


def test_append_tokens_without_a_slot_are_reported(L, gen):
    c = Paged(gen, [20, 20, 20], 1, 64, 16, BF)
    lay = L.ExactAttention(2, 1, 64, BF, c.k_pool, c.v_pool)
    k, v, q = randn(gen, 3, 1, 64, dtype=BF), randn(gen, 3, 1, 64, dtype=BF), randn(gen, 3, 2, 64, dtype=BF)
    table = c.table.clone()
    table[0, 1], table[2, 1] = -1, c.n_pages
    v0 = c.v_pool.clone()
    lay.append(k, v, ints([20, 33, 20]), table, q=q, inv_freq=_freq(64))       # 33: past the two columns
    assert L.lola_attn_status() == (L.LOLA_ERR_DEVICE, L.LOLA_ATTN_BAD_PAGE)
    assert torch.equal(c.v_pool, v0)
    quiet(L)


# ---------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d,Hq,Hkv,page", [(BF, 128, 8, 2, 64), (F32, 64, 4, 1, 16)])
def test_a_layer_serves_prompts_and_then_tokens(L, gen, dtype, d, Hq, Hkv, page):
    """Prompts in two pieces, then single tokens, as a server runs a layer: each output against the
    float64 attention over the layer's own rotated rows."""
    prompt, cut, steps, B = [150, 40, 301], [100, 40, 7], 5, 3
    total = [n + steps for n in prompt]
    need = [-(-n // page) for n in total]
    lay = L.ExactAttention.allocate(Hq, Hkv, d, sum(need), page, dtype)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).tolist()
    table = ints([[order.pop() for _ in range(n)] + [-1] * (max(need) - n) for n in need])
    inv = _freq(d)
    K = [torch.empty(0, Hkv, d, dtype=dtype, device="cuda") for _ in range(B)]
    V = [torch.empty(0, Hkv, d, dtype=dtype, device="cuda") for _ in range(B)]

    def put(new, length):
        """Appends new[b] tokens; returns the rotated queries, keys kept beside."""
        t = sum(new)
        q, k, v = (randn(gen, t, h, d, dtype=dtype) for h in (Hq, Hkv, Hkv))
        one = new == [1] * B
        qr = lay.append(k, v, ints(length), table, cu_new=None if one else offsets(new), q=q, inv_freq=inv)
        r = 0
        for b, n in enumerate(new):
            pos = torch.arange(length[b] - n, length[b], device="cuda")
            K[b] = torch.cat([K[b], lay.k_pool[table[b].long()[pos // page], :, pos % page]])
            V[b] = torch.cat([V[b], v[r:r + n]])
            r += n
        return qr

    done = [0] * B
    for piece in (cut, [n - c for n, c in zip(prompt, cut)]):
        done = [x + n for x, n in zip(done, piece)]
        qr = put(piece, done)
        k, v = torch.cat(K), torch.cat(V)
        out = lay.prefill(qr, k, v, offsets(piece), offsets(done))
        check_prefill(qr, k, v, piece, done, out)
        assert torch.equal(lay.prefill_paged(qr, offsets(piece), ints(done), table, sum(done)), out)
    for _ in range(steps):
        done = [x + 1 for x in done]
        qr = put([1] * B, done)
        out = lay.decode_step(qr, ints(done), table)
        for b in range(B):
            seen = torch.ones(1, done[b], dtype=torch.bool, device="cuda")
            for h in range(Hq):
                g = h * Hkv // Hq
                o, _, tol, _ = attend(qr[b, h][None], K[b][:, g], V[b][:, g], seen)
                check(out[b, h][None], o, tol, f"token of sequence {b} head {h}")
        # the single-token read and the prompt attention agree on the token
        o2 = lay.prefill(qr, torch.cat(K), torch.cat(V), offsets([1] * B), offsets(done))
        check_prefill(qr, torch.cat(K), torch.cat(V), [1] * B, done, o2)
    quiet(L)


def test_prompt_attention_is_the_limit_of_a_lola_layer(L, gen):
    """A LoLA layer whose window holds the whole prompt is exact causal attention: the two layers
    agree to the sum of their roundings (bf16: 2e-2, the library's bar for LoLA outputs)."""
    B, H, n, d = 2, 3, 500, 128
    q, k, v = (randn(gen, B, H, n, d, dtype=BF) for _ in range(3))
    W = torch.randn(d // 2, d, generator=gen, device="cuda") / 8
    Y = L.Lola(B, H, d, d, 512, 0, chunk=64, dtype=BF).prefill(q, k, v, W)
    rows = [t.permute(0, 2, 1, 3).reshape(B * n, H, d) for t in (q, k, v)]
    out = L.ExactAttention(H, H, d, BF).prefill(*rows, offsets([n] * B))
    got = out.reshape(B, n, H, d).permute(0, 2, 1, 3)
    assert float((got.float() - Y.float()).abs().max()) <= 2e-2


def test_refused_calls_say_what_is_wrong(L, gen):
    """The call's short form declines what it does not take for granted; the long one then raises, or
    handles it.  Neither keeps a reference."""
    import sys
    c = Paged(gen, [40, 30], 2, 64, 16, BF)
    lay = L.ExactAttention(4, 2, 64, BF, c.k_pool, c.v_pool)
    q, k = randn(gen, 2, 4, 64, dtype=BF), randn(gen, 2, 2, 64, dtype=BF)
    cu = offsets([1, 1])
    good = lay.decode_step(q, c.kv_len, c.table)
    for bad in (q.float(), q[:1], q[:, :3], q.cpu(), torch.empty(2, 64, 4, dtype=BF, device="cuda").transpose(1, 2)):
        with pytest.raises(ValueError):
            lay.decode_step(bad, c.kv_len, c.table)
        with pytest.raises(ValueError):
            lay.append(k, k, c.kv_len, c.table, q=bad, inv_freq=_freq(64))
    for args in ((q, c.kv_len.long(), c.table), (q, c.kv_len, c.table.long()), (q, c.kv_len[:1], c.table),
                 (q, c.kv_len, c.table.t().contiguous().t())):
        with pytest.raises(ValueError):
            lay.decode_step(*args)
    with pytest.raises(ValueError):
        lay.prefill(q, k, k[:1], cu)
    with pytest.raises(ValueError):
        lay.prefill(q, k, k, cu.long())
    with pytest.raises(L.LolaError):
        lay.prefill(q, k[:1], k[:1], cu)                       # other totals without offsets of their own
    for args in ((q.float(), cu, c.kv_len, c.table), (q, cu[:2], c.kv_len, c.table), (q, cu.long(), c.kv_len, c.table),
                 (q, cu, c.kv_len.long(), c.table), (q, cu, c.kv_len, c.table.t().contiguous().t())):
        with pytest.raises(ValueError):
            lay.prefill_paged(*args)
    with pytest.raises(L.LolaError):
        lay.prefill_paged(q, cu, c.kv_len, c.table, total_k=-1)
    with pytest.raises(L.LolaError):
        lay.append(k, k, c.kv_len, c.table, q=q)               # q without a rotation
    with pytest.raises(L.LolaError):
        lay.append(k[:1], k[:1], c.kv_len, c.table)            # one token for two sequences
    with pytest.raises(KeyError):
        lay.append(k, k, c.kv_len, c.table, pairs="both")
    odd = torch.zeros(2 * 4 * 64 + 4, dtype=BF, device="cuda")[4:].view(2, 4, 64)     # 8-byte aligned
    with pytest.raises(L.LolaError):
        lay.decode_step(odd, c.kv_len, c.table)
    big = L.ExactAttention(4, 2, 64, BF, torch.zeros(2, 2, 24, 64, dtype=BF, device="cuda"),
                           torch.zeros(2, 2, 24, 64, dtype=BF, device="cuda"))
    with pytest.raises(L.LolaError):
        big.decode_step(q, c.kv_len, c.table)                  # pages of 24 tokens
    quiet(L)
    held = [sys.getrefcount(x) for x in (q, k, c.kv_len, c.table, cu, c.k_pool)]
    for _ in range(50):
        again = lay.decode_step(q, c.kv_len, c.table)
        lay.prefill(q, k, k, cu)
        lay.prefill_paged(q, cu, c.kv_len, c.table, 70)
    assert held == [sys.getrefcount(x) for x in (q, k, c.kv_len, c.table, cu, c.k_pool)]
    assert torch.equal(again, good) and sys.getrefcount(again) == sys.getrefcount(good)


def test_page_tables_whose_rows_overlap_are_refused(L, gen):
    """One row of pages for every sequence, expanded: refused; a copy of it serves."""
    c = Paged(gen, [30], 2, 64, 16, BF)
    lay = L.ExactAttention(4, 2, 64, BF, c.k_pool, c.v_pool)
    q, k, lens = randn(gen, 3, 4, 64, dtype=BF), randn(gen, 3, 2, 64, dtype=BF), ints([30, 30, 30])
    shared = c.table[:1].expand(3, -1)
    with pytest.raises(L.LolaError):
        lay.decode_step(q, lens, shared)
    with pytest.raises(L.LolaError):
        lay.append(k, k, lens, shared)
    got = lay.decode_step(q, lens, shared.contiguous())
    quiet(L)
    assert torch.equal(got[1], lay.decode_step(q[1:2], lens[:1], shared[:1])[0])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
def test_outputs_in_place_of_the_queries(L, gen, dtype, d):
    """The same bits as into other memory, for prompts of both forms and for single tokens."""
    lay = L.ExactAttention(6, 2, d, dtype)
    for lens in ([700, 130, 1, 391], [3000, 2500, 1200, 17] * 4):
        q, k = randn(gen, sum(lens), 6, d, dtype=dtype), randn(gen, sum(lens), 2, d, dtype=dtype)
        want = lay.prefill(q, k, k, offsets(lens))
        assert lay.prefill(q, k, k, offsets(lens), out=q) is q and torch.equal(q, want)
    lens = [4000, 3, 0, 777]
    c = Paged(gen, lens, 2, d, 64, dtype)
    lay = L.ExactAttention(6, 2, d, dtype, c.k_pool, c.v_pool)
    q = randn(gen, 4, 6, d, dtype=dtype)
    want = lay.decode_step(q, c.kv_len, c.table)
    assert lay.decode_step(q, c.kv_len, c.table, out=q) is q and torch.equal(q, want)
    quiet(L)


def test_kernel_timing_counts_the_new_kernels(L, gen):
    c = Paged(gen, [200], 1, 64, 16, BF)
    lay = L.ExactAttention(1, 1, 64, BF, c.k_pool, c.v_pool)
    q, k = randn(gen, 1, 1, 64, dtype=BF), randn(gen, 1, 1, 64, dtype=BF)
    L.lola_kernel_timing(True)
    lay.append(k, k, c.kv_len, c.table)
    lay.decode_step(q, c.kv_len, c.table)
    lay.prefill(q, k, k, offsets([1]))
    L.lola_kernel_timing(False)
    for name in ("attn", "append", "paged"):
        ms, n = L.lola_kernel_time(name)
        assert n == 1 and ms > 0, name
