"""Exact attention on the GPU at the edges of its types and of its kernels' forms.  Bounds:
tests/attn_parity.py, and beside the tests that need closer ones."""
import math

import pytest
import torch

from attn_parity import Paged, attend, check, check_prefill, ints, offsets, randn, rotated

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MAX = torch.finfo(F32).max


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_exact_kv_gb300 as lib
    return lib


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(23)


def _freq(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def quiet(L):
    st, bits = L.lola_attn_status()
    assert st == 0 and bits == 0, bits


def prompt(L, q, k, v, paged, dtype=F32, lse=None):
    """One prompt, its keys and values packed or in the pages of a cache."""
    n, Hq, Hkv, d = q.shape[0], q.shape[1], k.shape[1], q.shape[2]
    if not paged:
        return L.ExactAttention(Hq, Hkv, d, dtype).prefill(q, k, v, offsets([n]), lse=lse)
    page, need = 16, -(-n // 16)
    pools = []
    for x in (k, v):
        pool = torch.zeros(need * page, Hkv, d, dtype=dtype, device="cuda")
        pool[:n] = x
        pools.append(pool.view(need, page, Hkv, d).transpose(1, 2).contiguous())
    lay = L.ExactAttention(Hq, Hkv, d, dtype, *pools)
    return lay.prefill_paged(q, offsets([n]), ints([n]), ints([list(range(need))]), n, lse=lse)


# ---------------------------------------------------------------------------------------
# float32 prompts: the operands' two parts
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("paged", [False, True], ids=["packed", "paged"])
def test_f32_prompt_values_next_to_the_largest(L, gen, d, paged):
    """The largest finite values: rows before them are the same bits as without, rows from them on are
    finite (one such value a channel, so that no sum of theirs passes the type)."""
    n = 200
    q, k, v = (randn(gen, n, 1, d, dtype=F32) for _ in range(3))
    big = {(70, 3): MAX, (130, 9): -MAX, (131, 17): 3.4019938e38, (131, 18): -3.402e38, (199, 20): MAX}
    for (at, ch), x in big.items():
        v[at, 0, ch] = x
    out = prompt(L, q, k, v, paged)
    quiet(L)
    for first in (70, 130, 131, 199):
        v0 = v.clone()
        v0[first:] = 0.0
        assert torch.equal(out[:first], prompt(L, q, k, v0, paged)[:first])
    assert bool(torch.isfinite(out).all())
    check_prefill(q, k, v, [n], [n], out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("paged", [False, True], ids=["packed", "paged"])
def test_f32_prompt_unseen_keys_leave_the_bits(L, gen, d, bad, paged):
    """A key that is not finite changes no bit of the rows before it.  Behind it a score of minus infinity
    is a key of no weight; plus infinity or NaN makes the row NaN, as exp(inf - inf) is."""
    n = 300
    q, k, v = (randn(gen, n, 1, d, dtype=F32) for _ in range(3))
    want = prompt(L, q, k, v, paged)
    k[250, 0, 7] = bad
    lse = torch.empty(1, n, device="cuda")
    out = prompt(L, q, k, v, paged, lse=lse)
    quiet(L)
    assert torch.equal(out[:250], want[:250])
    none = torch.zeros(n, dtype=torch.bool, device="cuda")
    if not math.isnan(bad):                                    # the score is minus infinity: the key is not there
        none[250:] = q[250:, 0, 7] * bad < 0
    assert bool(torch.isnan(out[250:][~none[250:]]).all())
    for r in torch.nonzero(none).flatten().tolist():
        seen = torch.arange(r + 1, device="cuda") != 250
        o, ls, to, tl = attend(q[r, 0][None], k[:r + 1, 0], v[:r + 1, 0], seen[None])
        check(out[r, 0][None], o, to, f"row {r}")
        check(lse[0, r][None], ls, tl, f"lse of row {r}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("paged", [False, True], ids=["packed", "paged"])
def test_f32_prompt_sums_are_rounded(L, gen, d, paged):
    """One key with a weight near all and many with small ones, values of one: the output is one.

    Bound: of the keys' tiles of 32 a warp takes 16 keys each, N tiles in all, and adds their sum to its
    output and to its normaliser, which stay within [1, 2): half a step of 2^-23 each, N 2^-23 together.  The
    small weights' own sums and parts (0.3 of the whole, (9 terms + 54) 2^-23 of it at most), the
    joins and the division: 32 2^-23.  Sums cut off instead lose half a step on average for each of the four
    instructions of a tile, 2 N 2^-23."""
    n = 16000
    q = torch.zeros(n, 1, d, device="cuda")
    q[..., 0] = math.sqrt(d)
    k = torch.zeros(n, 1, d, device="cuda")
    k[1:, 0, 0] = -16 * math.log(2.0) + 0.3 * randn(gen, n - 1, dtype=F32)
    out = prompt(L, q, k, torch.ones(n, 1, d, device="cuda"), paged)
    quiet(L)
    tol = (torch.arange(n, device="cuda").double() / 32 + 1 + 32) * 2.0 ** -23
    over = (out[:, 0].double() - 1).abs().amax(-1) - tol
    assert float(over.max()) <= 0, f"{float(((out - 1).abs().amax()) * 2 ** 23)} steps"


# ---------------------------------------------------------------------------------------
# many sequences: several rounds of items, which cross the 32 sequences looked at together
# ---------------------------------------------------------------------------------------

MANY = [([(53 * i) % 400 for i in range(300)], None),                   # short ones, some empty: one tile a CTA
        ([2300 + 31 * (i % 40) for i in range(80)], None),             # long ones: two tiles
        ([1 + i % 3 for i in range(1100)], [1 + (7 * i) % 300 for i in range(1100)]),     # a few queries of many
        ([(5000 if i % 50 == 7 else i % 5) for i in range(130)], None)]


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("lens,keys", MANY, ids=["300-short", "80-long", "1100-pieces", "130-mixed"])
@pytest.mark.parametrize("paged", [False, True], ids=["packed", "paged"])
def test_prefill_many_sequences(L, gen, dtype, d, lens, keys, paged):
    Hq, Hkv, keys = 8, 2, keys or lens
    q = randn(gen, sum(lens), Hq, d, dtype=dtype)
    if paged:
        c = Paged(gen, keys, Hkv, d, 64, dtype, junk=math.nan)
        k, v = torch.cat(c.k), torch.cat(c.v)
        out = L.ExactAttention(Hq, Hkv, d, dtype, c.k_pool, c.v_pool).prefill_paged(q, offsets(lens), c.kv_len, c.table,
                                                                                    sum(keys))
    else:
        k, v = (randn(gen, sum(keys), Hkv, d, dtype=dtype) for _ in range(2))
        out = L.ExactAttention(Hq, Hkv, d, dtype).prefill(q, k, v, offsets(lens), offsets(keys))
    quiet(L)
    assert bool(torch.isfinite(out).all())
    check_prefill(q, k, v, lens, keys, out, heads=[0, 7], rows=[0, 1, 127, 128, 255, 300, 2299, 4999])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_bad_offsets_behind_many_sequences(L, gen, dtype):
    """The sequence that is wrong is not among the first 32 nor the last; its neighbours are whole.  The
    rows 3993 .. 3999 belong to two sequences (99 and 102) and hold either's result: they are not looked at."""
    n, d = 200 * 40, 64
    q, k, v = (randn(gen, n, 2, d, dtype=dtype) for _ in range(3))
    cu = [40 * i for i in range(201)]
    cu[101] = cu[102] = cu[100] - 7                            # 100 decreases, 101 is empty, 102 begins early
    out = torch.full((n, 2, d), 3.0, dtype=dtype, device="cuda")
    L.ExactAttention(2, 2, d, dtype).prefill(q, k, v, ints(cu), out=out)
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_OFFSETS
    quiet(L)
    check_prefill(q, k, v, [40] * 99, [40] * 99, out, rows=[0, 39])
    check_prefill(q[3960:4000], k[3960:4000], v[3960:4000], [40], [40], out[3960:4000], rows=[0, 32])
    first = cu[102]                                            # sequence 102 reaches from there to its end
    lens = [cu[103] - first] + [40] * 97
    check_prefill(q[first:], k[first:], v[first:], lens, lens, out[first:], rows=[10, 39, 60, 86])


# ---------------------------------------------------------------------------------------
# large values under a rising maximum
# ---------------------------------------------------------------------------------------

def _rising(n, H, d, dtype):
    """Scores that rise by 6.5 (log2) after the first block, and one value of 3e38 behind the rise."""
    q, k, v = (torch.zeros(n, H, d, dtype=dtype, device="cuda") for _ in range(3))
    q[..., 0] = 1.0
    k[n // 2:, :, 0] = 4.5 * math.sqrt(d)
    v[2 * n // 3, :, 5] = 3e38
    v[..., 6] = 1.0
    return q, k, v


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("beside", [0, 20000], ids=["one-tile", "two-tiles"])
def test_prompt_large_values_under_a_rising_maximum(L, gen, dtype, d, beside):
    """Weights are at most one, so a finite value with a weight below one stays finite."""
    if dtype == F32 and beside:
        beside = 500
    n, Hq, Hkv = 600, 16, 4
    q, k, v = _rising(n, Hkv, d, dtype)
    q = q.repeat_interleave(Hq // Hkv, 1)
    lens = [n] + [beside] * (beside > 0)
    if beside:
        q, k, v = (torch.cat([x, randn(gen, beside, x.shape[1], d, dtype=dtype)]) for x in (q, k, v))
    lse = torch.empty(Hq, sum(lens), device="cuda")
    out = L.ExactAttention(Hq, Hkv, d, dtype).prefill(q, k, v, offsets(lens), lse=lse)
    quiet(L)
    assert bool(torch.isfinite(out[:n]).all())
    check_prefill(q[:n], k[:n], v[:n], [n], [n], out[:n], lse[:, :n], heads=[0, 15])


@pytest.mark.parametrize("dtype,d,Hq", [(BF, 128, 2), (BF, 128, 12), (BF, 64, 2), (BF, 64, 12), (F32, 128, 2), (F32, 64, 5),
                                        (F32, 64, 12)])
def test_decode_large_values_under_a_rising_maximum(L, gen, dtype, d, Hq):
    """300 sequences, so that a warp sees several tiles of each."""
    n, B = 600, 300
    q, k, v = _rising(n, 1, d, dtype)
    c = Paged(gen, [n] * B, 1, d, 64, dtype)
    for b in range(B):
        c.k[b], c.v[b] = k, v
        c.put(b, torch.arange(n, device="cuda"), k, v)
    q = q[:1].expand(B, Hq, d).contiguous()
    lse = torch.empty(B, Hq, device="cuda")
    out = L.ExactAttention(Hq, 1, d, dtype, c.k_pool, c.v_pool).decode_step(q, c.kv_len, c.table, lse=lse)
    quiet(L)
    assert bool(torch.isfinite(out).all())
    o, ls, to, tl = attend(q[0], k[:, 0], v[:, 0], torch.ones(Hq, n, dtype=torch.bool, device="cuda"))
    for b in range(B):
        check(out[b], o, to, f"sequence {b}")
        check(lse[b], ls, tl, f"lse of sequence {b}")


@pytest.mark.parametrize("dtype,d,Hq", [(BF, 128, 2), (BF, 64, 12), (F32, 64, 2), (F32, 128, 5)])
@pytest.mark.parametrize("n", [1, 300, 5000])
def test_decode_scores_of_minus_infinity(L, gen, dtype, d, Hq, n):
    """Where all scores are minus infinity the softmax is 0 / 0, as in the prompt form; where some are,
    those tokens have no weight; a sequence without tokens is zero."""
    c = Paged(gen, [n, n, 0], 1, d, 16, dtype)
    q = randn(gen, 3, Hq, d, dtype=dtype)
    q[..., 0] = 1.0
    c.k[0][:, 0, 0] = -math.inf
    c.k[1][:, 0, 0] = -math.inf
    c.k[1][n // 2] = 1.0
    for b in (0, 1):
        c.put(b, torch.arange(n, device="cuda"), c.k[b], c.v[b])
    lse = torch.empty(3, Hq, device="cuda")
    lay = L.ExactAttention(Hq, 1, d, dtype, c.k_pool, c.v_pool)
    out = lay.decode_step(q, c.kv_len, c.table, lse=lse)
    lse2 = torch.empty(Hq, 3, device="cuda")
    same = lay.prefill_paged(q, offsets([1, 1, 1]), c.kv_len, c.table, lse=lse2)
    quiet(L)
    for o, l in ((out, lse), (same, lse2.t())):
        assert bool(torch.isnan(o[0]).all()) and bool((l[0] == -math.inf).all())
        assert bool((o[2] == 0).all()) and bool((l[2] == -math.inf).all())
    o, ls, to, tl = attend(q[1], c.k[1][n // 2:n // 2 + 1, 0], c.v[1][n // 2:n // 2 + 1, 0],
                           torch.ones(Hq, 1, dtype=torch.bool, device="cuda"))
    check(out[1], o, to, "one key of any weight")
    check(lse[1], ls, tl, "its lse")


# ---------------------------------------------------------------------------------------
# the paged cache: rotation and append
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("n", [700, 9001])
def test_append_cosines(L, gen, n, pairs):
    """Pairs (1, 0) and (0, 1) show the cosines and sines themselves, all around the circle.

    Bound: the rest of a quarter turn as float32, at most 2^-2 half turns: half a step 2^-27, times pi; what is cut
    off the 64-bit turn, 2^-31 half turns; a step of the functions' own, 2^-24 below one."""
    d, page = 128, 64
    c = Paged(gen, [n], 1, d, page, F32)
    x = torch.zeros(n, 2, d, device="cuda")
    a = slice(0, d // 2) if pairs == "halves" else slice(0, d, 2)
    b = slice(d // 2, d) if pairs == "halves" else slice(1, d, 2)
    x[:, 0, a] = 1.0
    x[:, 1, b] = 1.0
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    lay = L.ExactAttention(2, 1, d, F32, c.k_pool, c.v_pool)
    pos = torch.arange(n, device="cuda")
    y = lay.append(x[:, :1], x[:, 1:], c.kv_len, c.table, cu_new=offsets([n]), q=x, inv_freq=inv, pairs=pairs)
    quiet(L)
    angle = pos[:, None].double() * inv.double()
    tol = math.pi * (2.0 ** -27 + 2.0 ** -31) + 2.0 ** -24
    stored = c.k_pool[c.table[0].long()[pos // page], 0, pos % page]
    for got, want in ((y[:, 0, a], angle.cos()), (y[:, 0, b], angle.sin()), (y[:, 1, a], -angle.sin()),
                      (y[:, 1, b], angle.cos()), (stored[:, a], angle.cos()), (stored[:, b], angle.sin())):
        worst = float((got.double() - want).abs().max())
        assert worst <= tol, worst


def _append_case(gen, lens_new, before, Hq, Hkv, d, page, dtype, lead=0, tail=0):
    """A cache with room for the new tokens, their rows, and for each row its sequence and position (-1: not
    in a sequence)."""
    total = [a + b for a, b in zip(lens_new, before)]
    c = Paged(gen, [0] * len(total), Hkv, d, page, dtype, extra=sum(-(-t // page) for t in total) + 3,
              width=max(1, max(-(-t // page) for t in total)))
    order = torch.randperm(c.n_pages, generator=torch.Generator().manual_seed(7)).tolist()
    c.table = ints([[order.pop() if i * page < t else -1 for i in range(c.table.shape[1])] for t in total])
    c.kv_len = ints(total)
    n = lead + sum(lens_new) + tail
    rows = randn(gen, n, Hq + 2 * Hkv, d, dtype=dtype)
    seq = torch.full((n,), -1, dtype=torch.long, device="cuda")
    pos = torch.full((n,), -1, dtype=torch.long, device="cuda")
    new, at = torch.tensor(lens_new, device="cuda"), lead + sum(lens_new)
    seq[lead:at] = torch.arange(len(total), device="cuda").repeat_interleave(new)
    first = new.cumsum(0) - new
    pos[lead:at] = torch.arange(at - lead, device="cuda") - first[seq[lead:at]] + torch.tensor(before, device="cuda")[seq[lead:at]]
    return c, rows, seq, pos


def _check_append(c, k0, v0, q, k, v, qr, seq, pos, inv, pairs, slot):
    """Rows with a slot are in their pages, those without one have only their query; the rest of the pools is as
    it was."""
    live = torch.nonzero(seq >= 0).flatten()
    y, tol = rotated(q[live], pos[live], inv, pairs)
    check(qr[live], y, tol + 1e-30, "q")
    live = torch.nonzero(slot).flatten()
    p = pos[live]
    pages, at = c.table.long()[seq[live], p // c.page], p % c.page
    y, tol = rotated(k[live], p, inv, pairs)
    check(c.k_pool[pages, :, at], y, tol + 1e-30, "k")
    k0[pages, :, at], v0[pages, :, at] = c.k_pool[pages, :, at], v[live]
    assert torch.equal(c.k_pool, k0) and torch.equal(c.v_pool, v0)


@pytest.mark.parametrize("dtype,d,rot", [(BF, 128, 128), (BF, 64, 48), (F32, 128, 32), (F32, 64, 64)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("n", [760, 761, 762, 763, 764, 3001])
def test_append_prompts(L, gen, dtype, d, rot, pairs, n):
    """The form for many tokens (from 761 on four of them a CTA, the last CTA with one to four), one
    prompt behind earlier tokens."""
    Hq, Hkv = 6, 2
    c, rows, seq, pos = _append_case(gen, [n], [37], Hq, Hkv, d, 16, dtype)
    k0, v0 = c.k_pool.clone(), c.v_pool.clone()
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    inv = _freq(rot)
    qr = L.ExactAttention(Hq, Hkv, d, dtype, c.k_pool, c.v_pool).append(k, v, c.kv_len, c.table, cu_new=offsets([n]), q=q,
                                                                        inv_freq=inv, pairs=pairs)
    quiet(L)
    _check_append(c, k0, v0, q, k, v, qr, seq, pos, inv, pairs, seq >= 0)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("B,most", [(33, 1), (33, 90), (100, 60), (1100, 1), (1100, 9), (2100, 3)])
def test_append_many_sequences(L, gen, dtype, d, B, most):
    """The search for a row's sequence in one to three rounds, empty sequences, rows before the first and behind the
    last one, which stay as they were; in place."""
    Hq, Hkv, page, lead, tail = 3, 1, 32, 5, 6
    new = [(i * 7919) % (most + 1) for i in range(B)]
    before = [(i * 31) % 50 for i in range(B)]
    c, rows, seq, pos = _append_case(gen, new, before, Hq, Hkv, d, page, dtype, lead, tail)
    k0, v0 = c.k_pool.clone(), c.v_pool.clone()
    q, k, v = rows[:, :Hq].clone(), rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    inv, q0 = _freq(d), q.clone()
    lay = L.ExactAttention(Hq, Hkv, d, dtype, c.k_pool, c.v_pool)
    got = lay.append(k, v, c.kv_len, c.table, cu_new=offsets(new, lead), q=q, inv_freq=inv, q_out=q)
    quiet(L)
    assert got is q and torch.equal(q[:lead], q0[:lead]) and torch.equal(q[lead + sum(new):], q0[lead + sum(new):])
    _check_append(c, k0, v0, q0, k, v, q, seq, pos, inv, "halves", seq >= 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [500, 2000])
def test_append_bad_slots_among_many(L, gen, dtype, n):
    """Tokens without a slot in the middle of a call: reported, their queries written, their neighbours whole;
    positions of the caller's; no rotation."""
    Hq, Hkv, d, page = 2, 2, 64, 16
    c, rows, seq, pos = _append_case(gen, [n, 9], [0, 0], Hq, Hkv, d, page, dtype)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    lay = L.ExactAttention(Hq, Hkv, d, dtype, c.k_pool, c.v_pool)
    slot = seq >= 0
    for col, bad in ((3, -1), (11, c.n_pages), (20, 2 ** 31 - 1)):
        c.table[0, col] = bad
        slot &= ~((seq == 0) & (pos // page == col))
    k0, v0 = c.k_pool.clone(), c.v_pool.clone()
    inv, turns = _freq(d), torch.flip(pos, (0,)) * 3
    qr = lay.append(k, v, c.kv_len, c.table, cu_new=offsets([n, 9]), q=q, inv_freq=inv, positions=turns.int())
    assert L.lola_attn_status() == (L.LOLA_ERR_DEVICE, L.LOLA_ATTN_BAD_PAGE)
    y, tol = rotated(q, turns, inv, "halves")
    check(qr, y, tol + 1e-30, "q")
    live = torch.nonzero(slot).flatten()
    pages, at = c.table.long()[seq[live], pos[live] // page], pos[live] % page
    y, tol = rotated(k[live], turns[live], inv, "halves")
    check(c.k_pool[pages, :, at], y, tol + 1e-30, "k")
    k0[pages, :, at], v0[pages, :, at] = c.k_pool[pages, :, at], v[live]
    assert torch.equal(c.k_pool, k0) and torch.equal(c.v_pool, v0)
    assert lay.append(k, v, c.kv_len, c.table, cu_new=offsets([n, 9])) is None
    assert L.lola_attn_status()[1] == L.LOLA_ATTN_BAD_PAGE
    k0[pages, :, at] = k[live]
    assert torch.equal(c.k_pool, k0) and torch.equal(c.v_pool, v0)
    quiet(L)


def test_append_at_the_ends_of_one_form(L, gen):
    """The two forms, one token a CTA and four, give the same bits."""
    Hq, Hkv, d = 4, 2, 128
    c, rows, _, _ = _append_case(gen, [761], [0], Hq, Hkv, d, 64, BF)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    lay, inv = L.ExactAttention(Hq, Hkv, d, BF, c.k_pool, c.v_pool), _freq(d)
    many = lay.append(k, v, c.kv_len, c.table, cu_new=offsets([761]), q=q, inv_freq=inv)
    pool = c.k_pool.clone()
    few = [lay.append(k[a:b], v[a:b], ints([b]), c.table, cu_new=offsets([b - a]), q=q[a:b], inv_freq=inv)
           for a, b in ((0, 400), (400, 761))]
    quiet(L)
    assert torch.equal(torch.cat(few), many) and torch.equal(c.k_pool, pool)


# ---------------------------------------------------------------------------------------
# single tokens: every group size of every form
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 33])
def test_decode_group_sizes(L, gen, dtype, d, G):
    """Lengths around the tiles and the pieces, junk of NaN in the pools and behind the lengths; a batch small enough
    to be cut into pieces, and one whose segments hold several tiles and sequences."""
    Hkv = 2
    for lens in ([700, 1, 64, 0, 129], [(67 * i) % 300 for i in range(150)]):
        c = Paged(gen, lens, Hkv, d, 32, dtype, junk=math.nan)
        q = randn(gen, len(lens), G * Hkv, d, dtype=dtype)
        lse = torch.empty(len(lens), G * Hkv, device="cuda")
        lay = L.ExactAttention(G * Hkv, Hkv, d, dtype, c.k_pool, c.v_pool)
        out = lay.decode_step(q, c.kv_len, c.table, lse=lse)
        quiet(L)
        for b in range(len(lens)) if len(lens) < 9 else (0, 1, 9, 76, 148, 149):
            seen = torch.ones(G, lens[b], dtype=torch.bool, device="cuda")
            for g in range(Hkv):
                hs = slice(g * G, (g + 1) * G)
                o, ls, to, tl = attend(q[b, hs], c.k[b][:, g], c.v[b][:, g], seen)
                check(out[b, hs], o, to, f"sequence {b} group {g}")
                check(lse[b, hs], ls, tl, f"lse of sequence {b} group {g}")
        assert torch.equal(out, lay.decode_step(q, c.kv_len, c.table))


# ---------------------------------------------------------------------------------------
# anomalies
# ---------------------------------------------------------------------------------------

def test_status_bits_of_another_stream_are_not_lost(L, gen):
    """One stream's calls set one bit and then another while the status is read all the time: every bit shows
    in one of the readings."""
    d = 64
    c = Paged(gen, [100], 1, d, 16, BF)
    lay = L.ExactAttention(1, 1, d, BF, c.k_pool, c.v_pool)
    q = randn(gen, 100, 1, d, dtype=BF)
    bad_cu, cu, bad_table = ints([5, 3]), offsets([100]), torch.full_like(c.table, -1)
    out, side, here = torch.empty_like(q), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    quiet(L)
    both = L.LOLA_ATTN_BAD_OFFSETS | L.LOLA_ATTN_BAD_PAGE
    for i in range(1500):
        lay.prefill_paged(q, bad_cu, c.kv_len, c.table, out=out, stream=side)
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000 + 977 * (i % 61))           # (a moment of GPU time between the two)
        lay.prefill_paged(q, cu, c.kv_len, bad_table, out=out, stream=side)
        done, bits = torch.cuda.Event(), 0
        done.record(side)
        while not done.query():
            bits |= L.lola_attn_status(stream=here)[1]
        bits |= L.lola_attn_status(stream=side)[1]
        assert bits == both, i
    quiet(L)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("lens", [[20000], [3000, 5, 700, 0, 9000], [300] * 200], ids=["one", "some", "many"])
def test_decode_after_waits_that_gave_up(L, gen, dtype, d, lens):
    """A call whose waits gave up says so; wherever that was, the workspace's cells end at zero, in replays of a
    captured call too, whose mark stays the same; the next call in that workspace is right."""
    c = Paged(gen, lens, 1, d, 64, dtype)
    lay = L.ExactAttention(4, 1, d, dtype, c.k_pool, c.v_pool)
    q = randn(gen, len(lens), 4, d, dtype=dtype)
    size = L.lola_paged_decode_workspace_bytes(lay.cfg)
    ws = torch.randint(0, 255, (size,), dtype=torch.uint8, device="cuda", generator=gen)
    cells = ws[size - 152 * 4 * 8:]                            # behind 152 x 4 records of 16 x (d + 2) floats
    assert size == 152 * 4 * (16 * (d + 2) * 4 + 8)
    out = torch.zeros_like(q)
    want = lay.decode_step(q, c.kv_len, c.table)
    lay.decode_step(q, c.kv_len, c.table, out=out, workspace=ws)
    cells.zero_()
    gave_up = 0
    try:
        for block in [0, 1, 2, 3, 4, 5, 6, 8, 11, 15, 23, 1000]:
            L.lola_selftest_attn_wait(block)
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                lay.decode_step(q, c.kv_len, c.table, out=out, workspace=ws)
            for _ in range(3):
                out.fill_(7.0)
                g.replay()
                st, bits = L.lola_attn_status()
                assert bits in (0, L.LOLA_ATTN_TIMEOUT)
                gave_up += bits != 0
                assert bits or torch.equal(out, want), block
                assert not bool(cells.any()), block
            L.lola_selftest_attn_wait(-1)
            out.fill_(7.0)
            lay.decode_step(q, c.kv_len, c.table, out=out, workspace=ws)
            quiet(L)
            assert torch.equal(out, want) and not bool(cells.any()), block
    finally:
        L.lola_selftest_attn_wait(-1)
    assert gave_up > 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[4000, 100, 1, 2500], [200] * 400, [5000] * 16], ids=["few", "one-tile", "two-tiles"])
@pytest.mark.parametrize("paged", [False, True], ids=["packed", "paged"])
def test_prefill_after_waits_that_gave_up(L, gen, d, lens, paged):
    """A prompt call whose waits gave up says so, ends, and leaves nothing behind for the next one."""
    H, n = 4, sum(lens)
    q = randn(gen, n, H, d, dtype=BF)
    c = Paged(gen, lens, H, d, 64, BF)
    k, v = torch.cat(c.k), torch.cat(c.v)
    lay = L.ExactAttention(H, H, d, BF, c.k_pool, c.v_pool)
    out, cu = torch.empty_like(q), offsets(lens)
    call = (lambda: lay.prefill_paged(q, cu, c.kv_len, c.table, n, out=out)) if paged else (
        lambda: lay.prefill(q, k, v, cu, out=out))
    want, gave_up = call().clone(), 0
    quiet(L)
    try:
        for block in (0, 1, 2, 3, 4, 7, 12, 25, 1000):
            L.lola_selftest_attn_wait(block)
            for _ in range(3):
                out.fill_(7.0)
                call()
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
# the binding
# ---------------------------------------------------------------------------------------

def test_pools_in_place_of_a_layers_own(L, gen):
    """A layer's pools may be replaced by others that fit it; others are refused by every call."""
    c, c2 = (Paged(gen, [70, 40], 2, 64, page, BF) for page in (16, 32))
    lay = L.ExactAttention(4, 2, 64, BF, c.k_pool, c.v_pool)
    q, k = randn(gen, 2, 4, 64, dtype=BF), randn(gen, 2, 2, 64, dtype=BF)
    cu, inv = offsets([1, 1]), _freq(64)
    lay.k_pool, lay.v_pool = c2.k_pool, c2.v_pool
    out = lay.decode_step(q, c2.kv_len, c2.table)
    quiet(L)
    for b in range(2):
        for h in range(4):
            o, _, to, _ = attend(q[b, h][None], c2.k[b][:, h // 2], c2.v[b][:, h // 2],
                                 torch.ones(1, c2.lens[b], dtype=torch.bool, device="cuda"))
            check(out[b, h][None], o, to, f"sequence {b} head {h}")
    for kp, vp in ((c.k_pool, c2.v_pool), (c2.k_pool, c.v_pool), (c.k_pool, None), (None, c.v_pool), (c.k_pool[:, :1], c.v_pool[:, :1]),
                   (c.k_pool.float(), c.v_pool.float()), (c.k_pool.transpose(1, 2), c.v_pool.transpose(1, 2))):
        lay.k_pool, lay.v_pool = kp, vp
        for call in (lambda: lay.decode_step(q, c.kv_len, c.table), lambda: lay.append(k, k, c.kv_len, c.table, q=q, inv_freq=inv),
                     lambda: lay.prefill_paged(q, cu, c.kv_len, c.table)):
            with pytest.raises(ValueError):
                call()
    quiet(L)


def test_copies_of_a_layer_serve(L, gen):
    import copy
    c = Paged(gen, [70, 40], 2, 64, 16, BF)
    lay = L.ExactAttention(4, 2, 64, BF, c.k_pool, c.v_pool, scale=0.2)
    q = randn(gen, 2, 4, 64, dtype=BF)
    want = lay.decode_step(q, c.kv_len, c.table)
    for other in (copy.copy(lay), copy.deepcopy(lay)):
        assert torch.equal(other.decode_step(q, c.kv_len, c.table), want)
    quiet(L)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_both_forms_of_the_binding_give_the_same_bits(L, gen, dtype, d, monkeypatch):
    """The calls through the marshalling module, and their Python form, which serves without it."""
    lens = [70, 300, 1]
    n = sum(lens)

    def run():
        g = torch.Generator(device="cuda").manual_seed(3)
        c = Paged(g, lens, 2, d, 16, dtype)
        lay = L.ExactAttention(4, 2, d, dtype, c.k_pool, c.v_pool)
        rows, cu = randn(g, n, 8, d, dtype=dtype), offsets(lens)
        q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
        qr = lay.append(k, v, c.kv_len, c.table, cu_new=cu, q=q, inv_freq=_freq(d), pairs="neighbours")
        assert lay.append(k[:3], v[:3], c.kv_len, c.table) is None
        return [qr, lay.prefill(q, k, v, cu), lay.prefill_paged(qr, cu, c.kv_len, c.table),
                lay.decode_step(q[:3], c.kv_len, c.table), c.k_pool, c.v_pool]

    fast = run()
    assert L._fast is not L._Declines
    monkeypatch.setattr(L, "_fast", L._Declines)
    with pytest.warns(RuntimeWarning):
        slow = run()
    quiet(L)
    assert all(torch.equal(a, b) for a, b in zip(fast, slow))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["prefill", "prefill_paged", "decode_step", "append", "status"])
def test_first_call_of_a_new_thread(L, gen, dtype, what):
    """A host thread whose first use of the GPU is the call (a server's worker): nothing has made the device's
    context the thread's own before."""
    import threading
    c = Paged(gen, [300, 40], 2, 64, 16, dtype)
    lay = L.ExactAttention(4, 2, 64, dtype, c.k_pool, c.v_pool)
    q, cu, inv = randn(gen, 340, 4, 64, dtype=dtype), offsets([300, 40]), _freq(64)
    k, v = torch.cat(c.k), torch.cat(c.v)
    out = [torch.empty_like(q), torch.empty_like(q)]
    call = {"prefill": lambda i: lay.prefill(q, k, v, cu, out=out[i]),
            "prefill_paged": lambda i: lay.prefill_paged(q, cu, c.kv_len, c.table, out=out[i]),
            "decode_step": lambda i: lay.decode_step(q[:2], c.kv_len, c.table, out=out[i][:2]),
            "append": lambda i: lay.append(k, v, c.kv_len, c.table, cu_new=cu, q=q, inv_freq=inv, q_out=out[i]),
            "status": lambda i: L.lola_attn_status()}[what]
    fast = {"prefill": lambda: lay.prefill(q, k, v, cu), "prefill_paged": lambda: lay.prefill_paged(q, cu, c.kv_len, c.table),
            "decode_step": lambda: lay.decode_step(q[:2], c.kv_len, c.table),
            "append": lambda: lay.append(k, v, c.kv_len, c.table, cu_new=cu, q=q, inv_freq=inv),
            "status": lambda: L.lola_attn_status()}[what]
    want = call(0)
    torch.cuda.synchronize()
    for f in (lambda: call(1), fast):
        got = []

        def run():
            try:
                got.append(f())
            except Exception as e:
                got.append(e)

        t = threading.Thread(target=run)
        t.start()
        t.join()
        assert not isinstance(got[0], Exception), got
        torch.cuda.synchronize()
        assert got[0] == (0, 0) if what == "status" else torch.equal(got[0], want)
    quiet(L)


def test_first_call_of_a_new_thread_lola(L, gen):
    """... and the same for a LoLA layer's prefill on the tensor cores."""
    import threading
    lay = L.Lola(1, 2, 128, 128, 64, 64)
    q, k, v = (randn(gen, 1, 2, 200, 128, dtype=BF) for _ in range(3))
    W = torch.randn(64, 128, generator=gen, device="cuda") / 8
    want = lay.prefill(q, k, v, W).clone()
    L.lola_state_init(lay.cfg, lay.state)
    Y, got = torch.empty_like(v), []
    torch.cuda.synchronize()

    def run():
        try:
            got.append(lay.prefill(q, k, v, W, Y=Y))
        except Exception as e:
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not isinstance(got[0], Exception), got
    assert torch.equal(Y, want)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_calls_with_nothing_in_them(L, gen, dtype, d):
    """No queries, no keys, no new tokens; a batch of no sequences is refused."""
    lay = L.ExactAttention(4, 2, d, dtype, *(torch.zeros(3, 2, 16, d, dtype=dtype, device="cuda") for _ in range(2)))
    rows = lambda n, h: randn(gen, n, h, d, dtype=dtype)  # noqa: E731
    none, zeros, table, inv = ints([0, 0]), ints([0]), ints([[1]]), _freq(d)
    lse = torch.zeros(4, 5, device="cuda")
    assert lay.prefill(rows(0, 4), rows(0, 2), rows(0, 2), none).shape == (0, 4, d)
    out = lay.prefill(rows(5, 4), rows(0, 2), rows(0, 2), offsets([5]), none, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    assert bool((lay.prefill(rows(5, 4), rows(0, 2), rows(0, 2), offsets([5]), none) == 0).all())
    assert lay.prefill(rows(0, 4), rows(7, 2), rows(7, 2), none, offsets([7])).shape == (0, 4, d)
    assert lay.prefill_paged(rows(0, 4), none, ints([9]), table).shape == (0, 4, d)
    assert bool((lay.prefill_paged(rows(5, 4), offsets([5]), zeros, table) == 0).all())
    assert bool((lay.decode_step(rows(1, 4), zeros, table) == 0).all())
    assert lay.append(rows(0, 2), rows(0, 2), ints([9]), table, cu_new=none, q=rows(0, 4), inv_freq=inv).shape == (0, 4, d)
    assert lay.append(rows(0, 2), rows(0, 2), ints([9]), table, cu_new=none) is None
    assert not bool(lay.k_pool.any()) and not bool(lay.v_pool.any())
    for call in (lambda: lay.decode_step(rows(0, 4), zeros[:0], table[:0]), lambda: lay.prefill(rows(0, 4), rows(0, 2), rows(0, 2), none[:1]),
                 lambda: lay.prefill_paged(rows(0, 4), none[:1], zeros[:0], table[:0]),
                 lambda: lay.append(rows(0, 2), rows(0, 2), zeros[:0], table[:0])):
        with pytest.raises(L.LolaError):
            call()
    quiet(L)


def test_beside_a_lola_layer_on_another_stream(L, gen):
    """A stack's two kinds of layers on two streams at once, which share the SMs' tensor memory: the bits of each are
    those of its calls alone."""
    lola = [L.Lola(1, 8, 128, 128, 64, 64, alloc=L.LOLA_ALLOC_CHUNK) for _ in range(6)]
    q, k, v = (randn(gen, 1, 8, 1500, 128, dtype=BF) for _ in range(3))
    W = torch.randn(64, 128, generator=gen, device="cuda") / 8
    lens = [700, 130, 2000, 1]
    c = Paged(gen, lens, 2, 128, 64, BF)
    lay = L.ExactAttention(8, 2, 128, BF, c.k_pool, c.v_pool)
    qe, cu, out = randn(gen, sum(lens), 8, 128, dtype=BF), offsets(lens), []
    one = lola[0].prefill(q, k, v, W).clone()
    two, three = lay.prefill_paged(qe, cu, c.kv_len, c.table), lay.decode_step(qe[:4], c.kv_len, c.table)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for other in lola[1:]:
        other.workspace_for(1500)
        Y = torch.empty_like(v)
        with torch.cuda.stream(a):
            other.prefill(q, k, v, W, Y=Y)
        with torch.cuda.stream(b):
            for _ in range(20):
                out.append((lay.prefill_paged(qe, cu, c.kv_len, c.table), lay.decode_step(qe[:4], c.kv_len, c.table)))
        torch.cuda.synchronize()
        assert torch.equal(Y, one)
        assert all(torch.equal(x, two) and torch.equal(y, three) for x, y in out)
        out.clear()
    quiet(L)
