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
