"""Plain forms of the quantised cache's operators and of attention over shared prefixes, and their bounds.

A row x becomes e4m3 codes of x 2^-e, 2^e the smallest power with max |x| <= 448 2^e in [2^-100, 2^119]; e4m3 numbers are
2^-9 apart below 2^-6 and round by at most 2^-4 of themselves above, so that |code 2^e - x| <= max(2^-4 |x|, 2^(e - 10)).
Attention over codes: as attn_parity's bounds, over the numbers that the codes stand for, which enter the products
exactly.  Three terms more: q is kept to 2^-39 of its row's largest number (|ds| <= c 2^-38 max|q| sum |k|); behind a shared
prefix, keys and values are kept to half of 2^-24 of their block's largest power, which is at most 1 / 224 of its largest
number (|ds| <= c 2^-32 max|k| sum |q|, and 2^-32 max|v| in o); and a weight that is small against its row's largest one,
to 2^-33 of that: 2^-31 (keys + 8) of the largest column's sum of p |v|, which has room for the values' term too."""
import math

import torch

from attn_parity import Paged, attend, check, randn

E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def power_of(e):
    """2^e in float64, exactly (|e| < 1023)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def encode(x):
    """Rows x [..., d] (float32 or bfloat16): codes as e4m3, powers of two as biased bytes."""
    y = x.double()
    fin = torch.isfinite(y)
    top = torch.where(fin, y.abs(), torch.zeros_like(y)).amax(-1)
    m, e = torch.frexp(top)                                  # top = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-100, 119)
    e = torch.where(top == 0, torch.full_like(e, -100), e)
    z = (y * power_of(-e)[..., None]).clamp(-448.0, 448.0)
    z = torch.where(fin, z, torch.full_like(z, math.nan))
    return z.float().to(E4), (e + 127).to(torch.uint8)


def decode(codes, power):
    return codes.double() * power_of(power.long() - 127)[..., None]


class QPaged(Paged):
    """A quantised paged cache: ``k``, ``v`` hold the numbers that the codes stand for (float64).  Slots behind the
    sequences hold NaN codes and any power."""

    def __init__(self, gen, lens, Hkv, d, page, dtype, dev="cuda", spread=0.5, **kw):
        super().__init__(gen, lens, Hkv, d, page, dtype, dev=dev, **kw)
        shape = self.k_pool.shape
        byte = lambda *s: torch.randint(0, 256, s, generator=gen, device=dev, dtype=torch.uint8)  # noqa: E731
        self.k_scale, self.v_scale = (byte(*shape[:3]).view(E8) for _ in range(2))
        self.k_pool, self.v_pool = (torch.full(shape, 0x7f, dtype=torch.uint8, device=dev).view(E4) for _ in range(2))
        for b, n in enumerate(lens):
            for w in "kv":
                # rows of several magnitudes
                x = getattr(self, w)[b].float() * torch.exp(spread * randn(gen, n, Hkv, 1, dtype=torch.float32, dev=dev))
                getattr(self, w)[b] = self.store(w, b, torch.arange(n, device=dev), x)

    def put(self, b, pos, k, v):                             # (the parent's filling of its pools)
        pass

    def store(self, w, b, pos, x):
        codes, power = encode(x)
        if pos.numel():
            at = self.table[b].long()[pos // self.page], pos % self.page
            getattr(self, w + "_pool").view(torch.uint8)[at[0], :, at[1]] = codes.view(torch.uint8)
            getattr(self, w + "_scale").view(torch.uint8)[at[0], :, at[1]] = power
        return decode(codes, power)

    def layer(self, L, Hq, Hkv, d, dtype, scale=None):
        return L.QuantizedAttention(Hq, Hkv, d, dtype, self.k_pool, self.v_pool, self.k_scale, self.v_scale, scale)


def check_attention(q, parts, out, lse=None, scale=None, what=""):
    """One sequence's rows: q [Hq, d], ``parts`` a list of (k, v, hidden | None) of tokens [n, Hkv, d], all seen one
    behind the other."""
    Hq, d = q.shape
    c = scale if scale else 1.0 / math.sqrt(d)
    k, v = (torch.cat([p[i].double() for p in parts]) for i in (0, 1))
    hidden = torch.cat([p[2] if p[2] is not None else torch.zeros(p[0].shape[0], dtype=torch.bool, device=q.device) for p in parts])
    n = int((~hidden).sum())
    for h in range(Hq):
        g = h * k.shape[1] // Hq
        o, ls, to, tl = attend(q[h][None], k[:, g], v[:, g], ~hidden[None], scale)
        fk, fv = (torch.nan_to_num(x[~hidden][:, g]) for x in (k, v))
        fq = torch.nan_to_num(q[h].double()).abs()
        ds = c * (2.0 ** -38 * float(fq.max() * fk.abs().sum(-1).max()) + 2.0 ** -32 * float(fq.sum() * fk.abs().max())) if n else 0.0
        A = fv.abs().amax() if n else 0.0
        check(out[h][None], o, to + (2 * ds + 2.0 ** -31 * (n + 8)) * A, f"{what} head {h}")
        if lse is not None:
            check(lse[h][None], ls, tl + ds, f"lse of {what} head {h}")
