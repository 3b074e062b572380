"""Plain float64 forms of the exact-attention operators and the error bounds of the GPU's.

Bounds (u = half a step of the io type: bf16 2^-8, float32 2^-24):
  scores  |ds| <= (d + 4) 2^-23 c sum_i |q_i k_i| + 2^-22   (float32 products summed in any order,
          the scale's rounding, and 2^s's own error)
  o       u |o| for the final rounding, plus A = sum_j p_j |v_j| (p normalised) times
          the weights' relative error: 2 max|ds| (numerator and normaliser), u for the
          bf16 weights of the product with V, and (keys + 8) 2^-23 for the two sums
  lse     max|ds| + (keys + 8) 2^-23 + |lse| 2^-22
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attend(q, k, v, seen, scale=None):
    """q [R, d], k, v [M, d], seen [R, M] bool: (o, lse, bound of o, bound of lse) in float64; the
    keys a row does not see are left out whatever they hold."""
    dt, d = q.dtype, q.shape[-1]
    c = scale if scale else 1.0 / math.sqrt(d)
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:                                       # no key at all: one that nobody sees
        k, v, seen = k.new_zeros(1, d), v.new_zeros(1, d), seen.new_zeros(seen.shape[0], 1)
    any_seen = seen.any(0)
    k = torch.where(any_seen[:, None], k, torch.zeros_like(k))
    s = (q @ k.T) * c
    s = s.masked_fill(~seen, -math.inf)
    n = seen.sum(-1).double()
    none = n == 0
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(none, torch.zeros_like(lse), lse)[:, None])
    # values that are not finite reach only the rows that see them
    fin = torch.isfinite(v)
    vz = torch.where(fin, v, torch.zeros_like(v))
    o, A = p @ vz, p @ vz.abs()
    if not bool(fin.all()):
        for j in torch.nonzero(~fin.all(-1)).flatten().tolist():
            rows = seen[:, j]
            add = torch.where(fin[j], torch.zeros_like(v[j]), v[j])
            o[rows] += add
    ds = ((q.abs() @ k.abs().T) * c * (d + 4) * 2.0 ** -23).masked_fill(~seen, 0.0).amax(-1) + 2.0 ** -22
    u = U[dt]
    w = 2 * ds + (u if dt == torch.bfloat16 else 0.0) + (n + 8) * 2.0 ** -23
    tol_o = u * o.abs() + (1 + u) * w[:, None] * A + 1e-30
    tol_l = ds + (n + 8) * 2.0 ** -23 + lse.abs() * 2.0 ** -22
    o[none] = 0.0
    return o, lse, tol_o, tol_l


def check(got, want, tol, what):
    got = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    if bool(fin.any()):
        over = ((got - want).abs() - tol)[fin]
        worst = float(over.max())
        assert worst <= 0, f"{what}: {worst} over the bound ({float(((got - want).abs() / tol)[fin].max()):.3g} of it)"


def ints(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def offsets(lens, start=0, dev="cuda"):
    out = [start]
    for n in lens:
        out.append(out[-1] + n)
    return ints(out, dev)


def randn(gen, *shape, dtype, dev="cuda"):
    return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)


def check_prefill(q, k, v, lens_q, lens_k, out, lse=None, scale=None, start=0, start_k=0, heads=None, rows=None):
    """Every head (or those in ``heads``) and row (or ``rows`` of each sequence) of a packed call."""
    Hq, Hkv = q.shape[1], k.shape[1]
    r, c = start, start_k
    for b, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        at = torch.arange(lq, device=q.device)
        if rows is not None:
            at = at[torch.as_tensor([x for x in rows if x < lq], device=q.device, dtype=torch.long)]
        key = torch.arange(lk, device=q.device)
        seen = key[None] <= at[:, None] + (lk - lq)
        for h in heads or range(Hq):
            if at.numel() == 0:
                continue
            g = h * Hkv // Hq
            o, ls, to, tl = attend(q[r + at, h], k[c:c + lk, g], v[c:c + lk, g], seen, scale)
            check(out[r + at, h], o, to, f"sequence {b} head {h}")
            if lse is not None:
                check(lse[h, r + at], ls, tl, f"lse of sequence {b} head {h}")
        r, c = r + lq, c + lk


class Paged:
    """A paged cache over a shuffled pool: sequences' tokens k, v [n, Hkv, d] in pages."""

    def __init__(self, gen, lens, Hkv, d, page, dtype, extra=3, junk=None, width=None, dev="cuda"):
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + extra
        self.page, self.lens = page, lens
        perm = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(5)).tolist()
        width = width or max(1, max(need))
        table, at = [], 0
        for n in need:
            table.append(perm[at:at + n] + [-1] * (width - n))
            at += n
        self.host_table = table
        self.table = ints(table, dev)
        self.kv_len = ints(lens, dev)
        shape = (self.n_pages, Hkv, page, d)
        fill = junk if junk is not None else 0.0
        self.k_pool = torch.full(shape, fill, dtype=dtype, device=dev)
        self.v_pool = torch.full(shape, fill, dtype=dtype, device=dev)
        self.k = [randn(gen, n, Hkv, d, dtype=dtype, dev=dev) for n in lens]
        self.v = [randn(gen, n, Hkv, d, dtype=dtype, dev=dev) for n in lens]
        for b, n in enumerate(lens):
            self.put(b, torch.arange(n, device=dev), self.k[b], self.v[b])

    def put(self, b, pos, k, v):
        if pos.numel():
            pages = self.table[b].long()[pos // self.page]
            self.k_pool[pages, :, pos % self.page] = k
            self.v_pool[pages, :, pos % self.page] = v


def check_decode(q, cache, out, lse=None, scale=None, hidden=None):
    """``hidden``: per sequence a bool tensor of tokens that must not be seen."""
    Hq = q.shape[1]
    for b, n in enumerate(cache.lens):
        seen = torch.ones(1, n, dtype=torch.bool, device=q.device)
        if hidden is not None and hidden[b] is not None:
            seen = seen & ~hidden[b]
        for h in range(Hq):
            g = h * cache.k[b].shape[1] // Hq
            o, ls, to, tl = attend(q[b, h][None], cache.k[b][:, g], cache.v[b][:, g], seen, scale)
            check(out[b, h][None], o, to, f"sequence {b} head {h}")
            if lse is not None:
                check(lse[b, h][None], ls, tl, f"lse of sequence {b} head {h}")


def rotated(x, pos, inv_freq, pairs):
    """x [n, H, d], pos [n]: the rotation over the first 2 len(inv_freq) channels in float64, and the
    bound: u |y| for the rounding, and (|a| + |b|) 2^-21 for cos and sin (their argument's rounding
    pi 2^-25 and their own 2^-23) and the products and sum."""
    y = x.double().clone()
    rot = 2 * inv_freq.numel()
    ang = pos.double()[:, None] * inv_freq.double()
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    size = torch.zeros_like(y)
    if pairs == "halves":
        ia, ib = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        ia, ib = slice(0, rot, 2), slice(1, rot, 2)
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, U[x.dtype] * y.abs() + size * 2.0 ** -21
