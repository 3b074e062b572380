"""Cases of the exact-attention operators: prompt attention over packed sequences, rotating and
appending keys and values to a paged cache, and single-token attention over that cache.

``own`` false: the operators in their plain form (elementary torch operations in float32).
``own`` true: the same results through this package's entry points."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_THETA = 10000.0


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # a handful of short prompts that arrive together: latency counts
        {"name": "prefill_short", "op": "prefill", "seqs": 5, "longest": 118, "spread": 100, "past": 0, "Hq": 32,
         "Hkv": 8, "d": 128, "dtype": "bf16", "fused": True},
        # the batched prompt workload: 4 sequences of 4096 tokens, 32 heads with their own keys
        {"name": "prefill_b4h32", "op": "prefill", "seqs": 4, "longest": 4096, "spread": 1, "past": 0, "Hq": 32,
         "Hkv": 32, "d": 128, "dtype": "bf16", "fused": False},
        # serving's usual packed batch: ragged prompts, grouped heads, rows of one projection
        {"name": "prefill_ragged", "op": "prefill", "seqs": 16, "longest": 4001, "spread": 40, "past": 0, "Hq": 32,
         "Hkv": 8, "d": 128, "dtype": "bf16", "fused": True},
        # a later piece of long prompts (keys of earlier pieces before the queries), narrow heads
        {"name": "prefill_pieces_d64", "op": "prefill", "seqs": 3, "longest": 1025, "spread": 3, "past": 6000,
         "Hq": 16, "Hkv": 4, "d": 64, "dtype": "bf16", "fused": False},
        # the long prompt: 131072 tokens, 8 heads
        {"name": "prefill_long", "op": "prefill", "seqs": 1, "longest": 131072, "spread": 1, "past": 0, "Hq": 8,
         "Hkv": 8, "d": 128, "dtype": "bf16", "fused": False},
        # float32 layers, as used to check a model's numerics
        {"name": "prefill_f32", "op": "prefill", "seqs": 3, "longest": 1024, "spread": 2, "past": 0, "Hq": 8,
         "Hkv": 2, "d": 64, "dtype": "f32", "fused": False},
        # one user, a short conversation: the smallest decode step
        {"name": "decode_one", "op": "decode", "seqs": 1, "longest": 1000, "spread": 1, "page": 16, "Hq": 32,
         "Hkv": 8, "d": 128, "dtype": "bf16"},
        # the batched decode workload: 64 sequences around 4096 tokens
        {"name": "decode_b64", "op": "decode", "seqs": 64, "longest": 8000, "spread": 8, "page": 64, "Hq": 32,
         "Hkv": 8, "d": 128, "dtype": "bf16"},
        # few very long contexts: the cache's length has to be split
        {"name": "decode_long", "op": "decode", "seqs": 3, "longest": 131072, "spread": 2, "page": 128, "Hq": 8,
         "Hkv": 8, "d": 128, "dtype": "bf16"},
        # float32 cache, narrow heads
        {"name": "decode_f32", "op": "decode", "seqs": 8, "longest": 2049, "spread": 4, "page": 32, "Hq": 8,
         "Hkv": 4, "d": 64, "dtype": "f32"},
        # one new token of every sequence of a decode batch
        {"name": "append_step", "op": "append", "seqs": 64, "longest": 1, "spread": 1, "past": 4000, "page": 64,
         "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "pairs": "halves"},
        # the tokens of a packed prompt batch
        {"name": "append_prompt", "op": "append", "seqs": 16, "longest": 4001, "spread": 40, "past": 0, "page": 16,
         "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "pairs": "neighbours"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "decode", "append"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    case = {"op": op, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype}
    if op == "prefill":
        case["longest"] = _log_int(rng, 1, 20000 if dtype == "bf16" else 4000)
        most = max(1, min(64, int(1.5e9 / (Hq * float(case["longest"] + 1000) ** 2))))
        case["seqs"] = _log_int(rng, 1, most)
        case["spread"] = _log_int(rng, 1, 50)
        case["past"] = rng.choice([0, 0, _log_int(rng, 1, 4000)])
        case["fused"] = rng.random() < 0.5
    elif op == "decode":
        case["longest"] = _log_int(rng, 1, 100000)
        most = max(1, min(128, int(6e8 / (case["longest"] * Hkv * d))))
        case["seqs"] = _log_int(rng, 1, most)
        case["spread"] = _log_int(rng, 1, 50)
        case["page"] = rng.choice([16, 32, 64, 128, 256])
    else:
        case["longest"] = _log_int(rng, 1, 4000)
        case["seqs"] = _log_int(rng, 1, max(1, min(100, 30000 // case["longest"])))
        case["spread"] = _log_int(rng, 1, 50)
        case["past"] = _log_int(rng, 1, 3000)
        case["page"] = rng.choice([16, 32, 64, 128, 256])
        case["pairs"] = rng.choice(["halves", "neighbours"])
    return case


def _lengths(case, key="longest"):
    """Sequence lengths from longest / spread to longest, spread evenly over their logarithm and
    then shuffled by a fixed rule; the first of the shuffled order is the longest."""
    n, top = case["seqs"], case[key]
    low = max(1, top // case["spread"])
    at = [(i * 7) % n if n % 7 else (i * 5) % n if n % 5 else i for i in range(n)]
    return [max(1, int(round(top * (low / top) ** (a / max(1, n - 1))))) for a in at]


def _past(case):
    """Tokens before the new ones of each sequence."""
    return [max(0, case["past"] - 37 * i) for i in range(case["seqs"])]


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _offsets(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)


def _table(lens, page, gen, dev):
    """A page table [seqs, widest] over a shuffled pool, -1 behind each sequence's pages, and the
    pool's page count (a few pages belong to nobody)."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    width = max(need)
    used = torch.tensor(need, device=dev)
    first = used.cumsum(0) - used
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    return torch.where(col < used[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32)), n_pages


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    s = dict(case)
    lens = _lengths(case)
    if case["op"] == "prefill":
        past = _past(case)
        klens = [a + b for a, b in zip(lens, past)]
        tq, tk = sum(lens), sum(klens)
        if case["fused"] and tq == tk:
            rows = normal(tq, Hq + 2 * Hkv, d)
            q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        else:
            q, k, v = normal(tq, Hq, d), normal(tk, Hkv, d), normal(tk, Hkv, d)
        s.update(q=q, k=k, v=v, cu_q=_offsets(lens, dev), cu_k=_offsets(klens, dev), lens_q=lens,
                 lens_k=klens, max_q=max(lens), max_k=max(klens))
    elif case["op"] == "decode":
        table, n_pages = _table(lens, case["page"], gen, dev)
        s.update(q=normal(case["seqs"], Hq, d), k_pool=normal(n_pages, Hkv, case["page"], d),
                 v_pool=normal(n_pages, Hkv, case["page"], d), table=table,
                 kv_len=torch.tensor(lens, dtype=torch.int32, device=dev))
    else:
        past = _past(case)
        total = [a + b for a, b in zip(lens, past)]
        table, n_pages = _table(total, case["page"], gen, dev)
        t = sum(lens)
        rows = normal(t, Hq + 2 * Hkv, d)
        inv = _THETA ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
        s.update(q=rows[:, :Hq], k=rows[:, Hq:Hq + Hkv], v=rows[:, Hq + Hkv:],
                 k_pool=normal(n_pages, Hkv, case["page"], d), v_pool=normal(n_pages, Hkv, case["page"], d),
                 table=table, kv_len=torch.tensor(total, dtype=torch.int32, device=dev), cu_new=_offsets(lens, dev),
                 inv_freq=inv.to(torch.float32).to(dev))
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def _softmax_read(S, seen, V):
    """softmax of S over the seen keys, times V; a row that sees nothing reads 0."""
    S = S.masked_fill(~seen, -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.exp(S - m)
    return (p @ V) / p.sum(-1, keepdim=True).clamp(min=1e-37)


def _plain_prefill(s):
    q, n = s["q"], s["seqs"]
    if n == 1 or s["max_q"] * s["max_k"] * s["Hq"] < 1 << 24:
        return _plain_batch(s, q, s["k"], s["v"], s["cu_q"].long(), s["cu_k"].long(), s["lens_q"], s["lens_k"])
    out, r, c = torch.empty(q.shape, dtype=q.dtype, device=q.device), 0, 0
    for i, (a, b) in enumerate(zip(s["lens_q"], s["lens_k"])):       # long sequences: no padding
        out[r:r + a] = _plain_batch(s, q[r:r + a], s["k"][c:c + b], s["v"][c:c + b], s["cu_q"][i:i + 2].long() - r,
                                    s["cu_k"][i:i + 2].long() - c, [a], [b])
        r, c = r + a, c + b
    return out


def _plain_batch(s, q, k, v, cu_q, cu_k, lens_q, lens_k):
    """Sequences padded to the longest."""
    Hq, Hkv, d, n, L, M = s["Hq"], s["Hkv"], s["d"], len(lens_q), max(lens_q), max(lens_k)
    G, dev, T = Hq // Hkv, q.device, q.shape[0]
    row, key = torch.arange(L, device=dev), torch.arange(M, device=dev)
    len_q, len_k = cu_q.diff(), cu_k.diff()
    at_q = (cu_q[:-1, None] + row).clamp(max=T - 1)
    at_k = (cu_k[:-1, None] + key).clamp(max=k.shape[0] - 1)
    Q = q[at_q].float().reshape(n, L, Hkv, G, d).permute(0, 2, 3, 1, 4)
    K = k[at_k].float().permute(0, 2, 3, 1)
    V = v[at_k].float().permute(0, 2, 1, 3)
    last = row + (len_k - len_q)[:, None]            # the last key that a row sees
    to = torch.where(row < len_q[:, None], at_q, T)  # padding rows go behind the last one
    out = torch.empty((T + 1, Hq, d), dtype=q.dtype, device=dev)
    step = max(1, min(L, (1 << 30) // (n * Hq * M)))
    for a in range(0, L, step):                      # as many rows at once as memory allows
        b = min(L, a + step)
        top = min(M, b + max(y - x for x, y in zip(lens_q, lens_k)))
        S = (Q[:, :, :, a:b].reshape(n, Hkv, G * (b - a), d) @ K[..., :top]) * (1.0 / math.sqrt(d))
        seen = (key[:top] <= last[:, a:b, None])[:, None, None]
        seen = seen.expand(n, Hkv, G, b - a, top).reshape(n, Hkv, G * (b - a), top)
        y = _softmax_read(S, seen, V[:, :, :top]).reshape(n, Hkv, G, b - a, d)
        out[to[:, a:b]] = y.permute(0, 3, 1, 2, 4).reshape(n, b - a, Hq, d).to(q.dtype)
    return out[:T]


def _plain_decode(s):
    q, table, kv_len = s["q"], s["table"].long().clamp(min=0), s["kv_len"].long()
    Hq, Hkv, d, n = s["Hq"], s["Hkv"], s["d"], s["seqs"]
    M = table.shape[1] * s["page"]
    K = s["k_pool"][table].permute(0, 2, 1, 3, 4).reshape(n, Hkv, M, d).float()
    V = s["v_pool"][table].permute(0, 2, 1, 3, 4).reshape(n, Hkv, M, d).float()
    S = (q.float().reshape(n, Hkv, Hq // Hkv, d) @ K.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    seen = torch.arange(M, device=q.device) < kv_len[:, None, None, None]
    return _softmax_read(S, seen, V).reshape(n, Hq, d).to(q.dtype)


def _turn(x, cos, sin, pairs):
    x = x.float()
    if pairs == "halves":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_append(s):
    q, k, v, cu, kv_len = s["q"], s["k"], s["v"], s["cu_new"].long(), s["kv_len"].long()
    t = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = kv_len[seq] - cu[seq + 1] + t
    page, slot = s["table"].long()[seq, pos // s["page"]], pos % s["page"]
    angle = pos[:, None].double() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s["k_pool"][page, :, slot] = _turn(k, cos, sin, s["pairs"]).to(k.dtype)
    s["v_pool"][page, :, slot] = v
    return {"q": _turn(q, cos, sin, s["pairs"]).to(q.dtype), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def run(state):
    s = state
    if own:
        import sparse_exact_kv_gb300 as L

        layer = L.ExactAttention(s["Hq"], s["Hkv"], s["d"], s["q"].dtype, s.get("k_pool"), s.get("v_pool"))
        if s["op"] == "prefill":
            return layer.prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
        if s["op"] == "decode":
            return layer.decode_step(s["q"], s["kv_len"], s["table"])
        q = layer.append(s["k"], s["v"], s["kv_len"], s["table"], cu_new=s["cu_new"], q=s["q"],
                         inv_freq=s["inv_freq"], pairs=s["pairs"])
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    return {"prefill": _plain_prefill, "decode": _plain_decode, "append": _plain_append}[s["op"]](s)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------------------

def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    io = 2 if case["dtype"] == "bf16" else 4
    lens = _lengths(case)
    if case["op"] == "prefill":
        past = _past(case)
        pairs = sum(n * (n + 1) // 2 + n * p for n, p in zip(lens, past))
        rows, keys = sum(lens), sum(lens) + sum(past)
        return {"bytes": io * d * (2 * rows * Hq + 2 * keys * Hkv), "flops": 4 * d * Hq * pairs}
    if case["op"] == "decode":
        keys = sum(lens)
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": io * d * (2 * keys * Hkv + 2 * case["seqs"] * Hq) + 4 * pages, "flops": 4 * d * Hq * keys}
    rows = sum(lens)
    # q read and written, k and v read and written; a rotation is 3 operations an element
    return {"bytes": io * d * rows * (2 * Hq + 4 * Hkv), "flops": 3 * d * rows * (Hq + Hkv)}


def exact(case, seed):
    lens = _lengths(case)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    past = _past(case) if "past" in case else [0] * len(lens)
    if case["op"] == "prefill" and 4 * d * Hq * sum(n * (n + p) for n, p in zip(lens, past)) > 4e12:
        return None
    s = prepare(case, seed)
    q = s["q"].double()
    if case["op"] == "append":
        k_pool, v_pool, out = s["k_pool"].double(), s["v_pool"].double(), torch.empty_like(q)
        freq = s["inv_freq"].double()
        r = 0
        for b, n in enumerate(lens):
            p = torch.arange(past[b], past[b] + n, device=q.device)
            turn = torch.polar(torch.ones(n, d // 2, dtype=torch.float64, device=q.device), p[:, None] * freq)[:, None]

            def turned(x):
                if case["pairs"] == "halves":
                    z = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn
                    return torch.cat([z.real, z.imag], -1)
                return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous())
                                          * turn).flatten(-2)

            out[r:r + n] = turned(q[r:r + n])
            at = s["table"][b].long()[p // case["page"]], p % case["page"]
            k_pool[at[0], :, at[1]] = turned(s["k"][r:r + n].double())
            v_pool[at[0], :, at[1]] = s["v"][r:r + n].double()
            r += n
        return {"q": out, "k_pool": k_pool, "v_pool": v_pool}
    out = torch.zeros_like(q)
    if case["op"] == "decode":
        for b, n in enumerate(lens):
            pages = s["table"][b, :-(-n // case["page"])].long()
            for h in range(Hkv):
                k = s["k_pool"][pages, h].reshape(-1, d)[:n].double()
                v = s["v_pool"][pages, h].reshape(-1, d)[:n].double()
                g = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                out[b, g] = torch.softmax(q[b, g] @ k.T / d ** 0.5, -1) @ v
        return out
    r = c = 0
    for n, p in zip(lens, past):
        hidden = torch.ones(n, n + p, dtype=torch.bool, device=q.device).triu(p + 1)
        for h in range(Hq):
            k, v = s["k"][c:c + n + p, h * Hkv // Hq].double(), s["v"][c:c + n + p, h * Hkv // Hq].double()
            w = torch.softmax((q[r:r + n, h] @ k.T / d ** 0.5).masked_fill(hidden, -math.inf), -1)
            out[r:r + n, h] = w @ v
        r, c = r + n, c + n + p
    return out
