"""Single tokens behind shared prefixes on the GPU, at the places where a piece of the work begins or ends, and over powers
of two that lie far apart.  Bounds: tests/quant_parity.py, unless a test states its own."""
import math

import pytest
import torch

from attn_parity import Paged, ints, offsets, randn
from quant_parity import QPaged, check_attention

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
    return torch.Generator(device="cuda").manual_seed(31)


def quiet(L):
    st, bits = L.lola_attn_status()
    assert st == 0 and bits == 0, bits


class Behind:
    """A cache of prefixes and sequences: sequence b sees prefix of[b] (-1: none) before its own tokens.  ``once``: a prefix
    table so wide that each prefix is read once for all its sequences, whatever its length."""

    def __init__(self, gen, quant, prefixes, members, lens, Hkv, d, page, dtype, once=True, start=0):
        self.c = (QPaged if quant else Paged)(gen, prefixes + lens, Hkv, d, page, dtype, **({} if quant else dict(junk=math.nan)))
        c, k = self.c, len(prefixes)
        self.prefix_len, self.kv_len = c.kv_len[:k].clone(), c.kv_len[k:].clone()
        self.prefix_table, self.table = c.table[:k], c.table[k:]
        if once:
            row = 2 * Hkv * d * (1 if quant else torch.finfo(dtype).bits // 8)
            wide = int(100e6) // (len(lens) * page * row) + 1
            self.prefix_table = torch.full((k, max(wide, c.table.shape[1])), -1, dtype=torch.int32, device="cuda")
            self.prefix_table[:, :c.table.shape[1]] = c.table[:k]
        self.cu = offsets(members, start)
        self.of = [-1] * start + [g for g, m in enumerate(members) for _ in range(m)]
        self.of += [-1] * (len(lens) - len(self.of))
        self.k = k

    def layer(self, L, Hq, Hkv, d, dtype):
        if isinstance(self.c, QPaged):
            return self.c.layer(L, Hq, Hkv, d, dtype)
        return L.ExactAttention(Hq, Hkv, d, dtype, self.c.k_pool, self.c.v_pool)

    def args(self):
        return self.kv_len, self.table, self.prefix_len, self.prefix_table, self.cu

    def parts(self, b):
        c, g = self.c, self.of[b]
        return ([(c.k[g], c.v[g], None)] if g >= 0 else []) + [(c.k[self.k + b], c.v[self.k + b], None)]

    def check(self, q, out, only=None):
        for b in only if only is not None else range(len(self.of)):
            check_attention(q[b], self.parts(b), out[b], what=f"sequence {b}")


# ---------------------------------------------------------------------------------------
# pieces that begin and end anywhere
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("quant,d,Hq,Hkv", [(False, 128, 8, 2), (False, 64, 6, 3), (True, 128, 8, 2), (True, 64, 6, 3), (True, 128, 2, 1)])
@pytest.mark.parametrize("prefixes,members", [([100, 300] * 150, [1] * 300), ([128, 257, 1] * 70, [2, 1, 3] * 70),
                                              ([128 * 61], [12]), ([128 * 77 + 1, 128 * 40], [9, 8])])
def test_pieces_that_begin_at_an_items_last_block(L, gen, quant, d, Hq, Hkv, prefixes, members):
    """One tile of rows, whose blocks are dealt out to two halves: one of them has none in a piece's first segment, and
    rows of another prefix or key head in the next."""
    n = sum(members)
    s = Behind(gen, quant, prefixes, members, [b % 3 for b in range(n)], Hkv, d, 32, BF)
    q = randn(gen, n, Hq, d, dtype=BF)
    lay = s.layer(L, Hq, Hkv, d, BF)
    out = lay.decode_shared(q, *s.args())
    for _ in range(5):
        assert torch.equal(out, lay.decode_shared(q, *s.args()))
    quiet(L)
    s.check(q, out)


# ---------------------------------------------------------------------------------------
# powers of two that lie far apart
# ---------------------------------------------------------------------------------------
# A row's numbers and its power of two enter the products exactly, whatever the powers of other rows are.  What is left:
# float32 products (attn_parity's ds), q to 2^-39 of its row's largest number, weights of 11 bits (22 in float32 io) or,
# where they are small, to 2^-25 in the unit in which the largest of p_j 2^f_j (f_j: a value row's power) is at least 2^-1:
# it is kept times 2^15 below a maximum of 2^0, which is at most 8 bits above the blocks' maxima, and those 8 above the
# rows' where a block is taken as one.  Codes are at most 448 and a row's largest one at least 224: 2^-23 of the
# largest p_j max|v_j| a key (rows of zeros have no error).  Everything is relative to what the row sees with its weights.

def check_apart(q, k, v, out, lse, codes_most=448 / 224, what=""):
    Hq, d = q.shape
    c, u = 1 / math.sqrt(d), {BF: 2.0 ** -8, F32: 2.0 ** -24}[q.dtype]
    weights = {BF: 2.0 ** -11, F32: 2.0 ** -22}[q.dtype]
    n = k.shape[0]
    for h in range(Hq):
        g = h * k.shape[1] // Hq
        x, K, V = q[h].double(), k[:, g].double(), v[:, g].double()
        s = c * (K @ x)
        norm = torch.logsumexp(s, 0)
        p = torch.exp(s - norm)
        o, A = p @ V, p @ V.abs()
        B = (p * V.abs().amax(-1)).amax()
        # (a score counts as far as its weight does: 2^-40 of the largest is nothing)
        near = p > 2.0 ** -60 * p.amax()
        lost = 2.0 ** -38 * x.abs().amax() * (x != 0) if q.dtype == F32 else 0 * x      # (zeros, and bfloat16 numbers, whole)
        ds = c * (K.abs() @ ((d + 4) * 2.0 ** -23 * x.abs() + lost))[near].amax() + 2.0 ** -22
        if q.dtype == F32:
            ds = ds + 2.0 ** -17                          # (s + f and m in float32, |f| < 2^7, in K11's exponents)
        tol = u * o.abs() + (1 + u) * (2 * ds + weights + 2.0 ** -17 + (n + 8) * 2.0 ** -23) * A + n * codes_most * 2.0 ** -24 * B
        err = (out[h].double() - o).abs()
        assert bool(torch.isfinite(out[h]).all()), f"{what} head {h}: not finite"
        worst = float((err / tol.clamp(min=1e-300)).max())
        assert worst <= 1, f"{what} head {h}: {worst:.3g} of the bound"
        if lse is not None:
            assert abs(float(lse[h].double() - norm)) <= float(ds) + (n + 8) * 2.0 ** -23 + abs(float(norm)) * 2.0 ** -22, f"lse of {what} head {h}"


def place(c, w, b, codes, power):
    """Codes [n, Hkv, d] and biased powers [n, Hkv] of sequence b's rows, written as they are."""
    pos = torch.arange(codes.shape[0], device="cuda")
    at = c.table[b].long()[pos // c.page], pos % c.page
    getattr(c, w + "_pool").view(torch.uint8)[at[0], :, at[1]] = codes.view(torch.uint8)
    getattr(c, w + "_scale").view(torch.uint8)[at[0], :, at[1]] = power
    getattr(c, w)[b] = codes.double() * 2.0 ** (power.double() - 127)[..., None]


def far_apart(gen, c, kind, Hkv, d):
    """Rewrites every sequence of the cache.  Queries have 0 in channel 0 and 8 in channel 1."""
    for b, n in enumerate(c.lens):
        pos = torch.arange(n, device="cuda")
        k, v = randn(gen, n, Hkv, d, dtype=F32), randn(gen, n, Hkv, d, dtype=F32)
        k[..., 1] = 0.0
        unseen = torch.zeros(n, dtype=torch.bool, device="cuda")
        if kind == "one value":                              # one row 2^30 times the others, without weight
            unseen[n // 2:n // 2 + 1] = True
            v[unseen] *= 2.0 ** 30
        elif kind == "values":
            unseen = pos % 50 == 7
            v *= torch.exp2(torch.randint(-6, 3, (n, 1, 1), generator=gen, device="cuda").float())
            v[unseen] *= torch.exp2(torch.randint(9, 60, (int(unseen.sum()), 1, 1), generator=gen, device="cuda").float())
        elif kind == "keys":                                 # large in a channel that no query has
            big = pos % 77 == 5
            k[big] = 0.0
            k[big, :, 0] = torch.exp2(torch.randint(12, 40, (int(big.sum()), 1), generator=gen, device="cuda").float())
        elif kind == "zeros":                                # blocks of rows of zeros, and of large ones
            v *= torch.where(pos // 128 % 2 == 0, 0.0, 2.0 ** 60)[:, None, None]
        elif kind == "zero rows":
            v *= torch.where(pos % 2 == 0, 0.0, 2.0 ** 45)[:, None, None]
        elif kind == "apart":                                # small ones by blocks, and large ones, all of the same weight
            v *= torch.where(pos // 128 % 3 == 0, 2.0 ** -85, 2.0 ** 50)[:, None, None]
        elif kind == "top":                                  # sums far behind float32's range, means that are in it
            v = 2.5e38 + 0.4e38 * torch.rand(v.shape, generator=gen, device="cuda")
        k[unseen, :, 1] = -300.0
        if kind == "high":                                   # the largest powers that a caller may write, of small codes
            place(c, "v", b, v.clamp(-1, 1).to(torch.float8_e4m3fn), torch.full((n, Hkv), 254, dtype=torch.uint8, device="cuda"))
        else:
            c.v[b] = c.store("v", b, pos, v)
        c.k[b] = c.store("k", b, pos, k)


APART = ["one value", "values", "keys", "zeros", "zero rows", "apart", "high", "top"]


def apart_queries(gen, n, Hq, d, dtype):
    q = randn(gen, n, Hq, d, dtype=dtype)
    q[..., 0], q[..., 1] = 0.0, 8.0
    return q


@pytest.mark.parametrize("kind", APART)
@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF, 128, 8, 2), (BF, 64, 12, 1), (F32, 128, 4, 1), (F32, 64, 10, 1)])
def test_decode_powers_far_apart(L, gen, dtype, d, Hq, Hkv, kind):
    lens = [1500, 17, 300, 1]
    c = QPaged(gen, lens, Hkv, d, 32, dtype)
    far_apart(gen, c, kind, Hkv, d)
    q = apart_queries(gen, len(lens), Hq, d, dtype)
    lse = torch.empty(len(lens), Hq, dtype=F32, device="cuda")
    out = c.layer(L, Hq, Hkv, d, dtype).decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    for b in range(len(lens)):
        check_apart(q[b], c.k[b], c.v[b], out[b], lse[b], 1 if kind == "high" else 2, f"sequence {b}")


@pytest.mark.parametrize("kind", APART)
@pytest.mark.parametrize("once", [False, True], ids=["few", "once"])
@pytest.mark.parametrize("dtype,d,Hq,Hkv,members", [(BF, 128, 8, 2, 5), (BF, 128, 8, 1, 40), (BF, 64, 12, 1, 9), (BF, 64, 12, 1, 30),
                                                    (F32, 128, 4, 1, 5)])
def test_shared_powers_far_apart(L, gen, dtype, d, Hq, Hkv, members, once, kind):
    """Behind a prefix: rows of one tile and of two, both forms of the call."""
    lens = [(i * 37) % 140 for i in range(members)]
    s = Behind(gen, True, [2500], [members], lens, Hkv, d, 32, dtype, once)
    far_apart(gen, s.c, kind, Hkv, d)
    q = apart_queries(gen, members, Hq, d, dtype)
    lse = torch.empty(members, Hq, dtype=F32, device="cuda")
    out = s.layer(L, Hq, Hkv, d, dtype).decode_shared(q, *s.args(), lse=lse)
    quiet(L)
    for b in range(0, members, max(1, members // 6)):
        k, v = (torch.cat([x[i] for x in s.parts(b)]) for i in (0, 1))
        check_apart(q[b], k, v, out[b], lse[b], 1 if kind == "high" else 2, f"sequence {b}")


@pytest.mark.parametrize("d,Hq,Hkv,members", [(128, 8, 1, 5), (128, 8, 1, 40), (64, 12, 1, 30)])
def test_shared_powers_far_apart_beside_bad_pages(L, gen, d, Hq, Hkv, members):
    """Tokens on pages outside the cache have no weight, and their places' powers no say."""
    page, n = 16, 1300
    s = Behind(gen, True, [n], [members], [3] * members, Hkv, d, page, BF)
    far_apart(gen, s.c, "values", Hkv, d)
    table = s.prefix_table.clone()
    table[0, 2::5] = -1
    pos = torch.arange(n, device="cuda")
    seen = table[0, pos // page] >= 0
    q = apart_queries(gen, members, Hq, d, BF)
    lse = torch.empty(members, Hq, dtype=F32, device="cuda")
    lay = s.layer(L, Hq, Hkv, d, BF)
    out = lay.decode_shared(q, s.kv_len, s.table, s.prefix_len, table, s.cu, lse=lse)
    assert L.lola_attn_status() == (L.LOLA_ERR_DEVICE, L.LOLA_ATTN_BAD_PAGE)
    for b in range(0, members, 4):
        k, v = (torch.cat([x[0][seen], x[1 + b]]) for x in (s.c.k, s.c.v))
        check_apart(q[b], k, v, out[b], lse[b], 2, f"sequence {b}")


# ---------------------------------------------------------------------------------------
# malformed offsets
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("once", [False, True], ids=["few", "once"])
@pytest.mark.parametrize("dtype,quant", [(BF, False), (BF, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("cu,of", [([0, 2, 4, 0], [0, 0, 1, 1, -1, -1]), ([4, 2, 4, 6], [-1, -1, 1, 1, 2, 2]),
                                   ([5, 0, 3, 1], [1, 1, 1, -1, -1, -1]), ([0, 3, -1, 7], [0, 0, 0, -1, -1, -1])])
def test_prefixes_with_sound_offsets_keep_their_sequences(L, gen, dtype, quant, cu, of, once):
    """Offsets that decrease or leave the batch cost their own prefix its sequences, and no other."""
    s = Behind(gen, quant, [90, 80, 70], [2, 2, 2], [5, 6, 7, 8, 9, 10], 1, 64, 16, dtype, once)
    q = randn(gen, 6, 2, 64, dtype=dtype)
    s.cu, s.of = ints(cu), of
    out = s.layer(L, 2, 1, 64, dtype).decode_shared(q, *s.args())
    assert L.lola_attn_status() == (L.LOLA_ERR_DEVICE, L.LOLA_ATTN_BAD_OFFSETS)
    s.check(q, out)


@pytest.mark.parametrize("quant", [False, True])
def test_many_prefixes_with_sound_offsets_keep_their_sequences(L, gen, quant):
    """More prefixes than one look takes in, the last offset (or one in between) below the others."""
    k, n = 70, 80
    s = Behind(gen, quant, [20 + i for i in range(k)], [1] * k, [3] * n, 1, 64, 16, BF, start=4)
    q = randn(gen, n, 2, 64, dtype=BF)
    lay = s.layer(L, 2, 1, 64, BF)
    s.check(q, lay.decode_shared(q, *s.args()))
    quiet(L)
    well = s.cu.tolist()
    for at, to, lost in ((k, 0, [k - 1]), (0, 70, [0]), (33, -5, [32, 33]), (50, 999, [49, 50])):
        cu = list(well)
        cu[at] = to
        s.cu, s.of = ints(cu), [-1] * 4 + [-1 if g in lost else g for g in range(k)] + [-1] * (n - k - 4)
        out = lay.decode_shared(q, *s.args())
        assert L.lola_attn_status() == (L.LOLA_ERR_DEVICE, L.LOLA_ATTN_BAD_OFFSETS), cu
        s.check(q, out)


# ---------------------------------------------------------------------------------------
# many rows
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("quant,d,Hq,Hkv,prefixes,members,own", [
    (False, 128, 8, 1, [900, 400, 1300], [40, 3, 70], 5),      # several items of 256 rows, of prefixes that are not alone
    (True, 128, 8, 1, [900, 400, 1300], [40, 3, 70], 5), (True, 64, 32, 1, [500, 640], [17, 30], 3),
    (False, 64, 64, 1, [300], [310], 2),                       # one prefix, 78 items: more than half of the CTAs
    (True, 64, 64, 1, [300], [310], 2), (False, 64, 64, 1, [129], [150], 0)])
def test_shared_many_rows(L, gen, quant, d, Hq, Hkv, prefixes, members, own):
    n = sum(members)
    s = Behind(gen, quant, prefixes, members, [own] * n, Hkv, d, 64, BF)
    q = randn(gen, n, Hq, d, dtype=BF)
    out = s.layer(L, Hq, Hkv, d, BF).decode_shared(q, *s.args())
    quiet(L)
    s.check(q, out, only=range(0, n, 9))
