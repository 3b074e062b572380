"""Cases of the operators on a quantised key-value cache and on shared prefixes: rotating, quantising and
appending keys and values, reading them back as rows, single-token attention over such a cache, and
single-token attention for batches whose sequences begin with a common prefix, held once.

The quantised cache holds a row (a token's key or value of one head) as e4m3 numbers with one power of two:
x ~ code * 2^(byte - 127), the power being the smallest whose 448-fold reaches the row's largest magnitude.

``own`` false: the operators in their plain form (elementary torch operations in float32).
``own`` true: the same results through this package's entry points."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_THETA = 10000.0
_LOW, _TOP = 27, 246        # the powers of two that are stored: 2^-100 .. 2^119


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one new token of every sequence of a decode batch
        {"name": "append_step", "op": "append", "seqs": 64, "longest": 1, "spread": 1, "past": 4000, "page": 64,
         "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "pairs": "halves"},
        # the tokens of a packed batch of ragged prompts
        {"name": "append_prompt", "op": "append", "seqs": 16, "longest": 4001, "spread": 40, "past": 0, "page": 16,
         "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "pairs": "neighbours"},
        # what a prompt's next piece attends to, read back for prompt attention: few short sequences
        {"name": "read_short", "op": "read", "seqs": 3, "longest": 1025, "spread": 3, "page": 32, "Hq": 16, "Hkv": 4,
         "d": 64, "dtype": "bf16"},
        # ... a serving batch's longer ones
        {"name": "read_batch", "op": "read", "seqs": 16, "longest": 8001, "spread": 8, "page": 64, "Hq": 32, "Hkv": 8,
         "d": 128, "dtype": "bf16"},
        # one user, a short conversation: the smallest decode step
        {"name": "decode_one", "op": "decode", "seqs": 1, "longest": 1000, "spread": 1, "page": 16, "Hq": 32,
         "Hkv": 8, "d": 128, "dtype": "bf16"},
        # the batched decode workload: 64 sequences around 4096 tokens
        {"name": "decode_b64", "op": "decode", "seqs": 64, "longest": 8000, "spread": 8, "page": 64, "Hq": 32,
         "Hkv": 8, "d": 128, "dtype": "bf16"},
        # few very long contexts: the cache's length has to be split
        {"name": "decode_long", "op": "decode", "seqs": 3, "longest": 131072, "spread": 2, "page": 128, "Hq": 40,
         "Hkv": 8, "d": 128, "dtype": "bf16"},
        # a handful of users behind one short instruction text: latency counts
        {"name": "shared_few", "op": "shared", "seqs": 4, "longest": 60, "spread": 10, "prefixes": 1, "prefix": 900,
         "prefix_spread": 1, "page": 16, "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "cache": "io"},
        # a decode batch whose requests all begin with the same long instructions and examples
        {"name": "shared_b64", "op": "shared", "seqs": 64, "longest": 700, "spread": 20, "prefixes": 1, "prefix": 16001,
         "prefix_spread": 1, "page": 64, "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "cache": "io"},
        # several documents, each asked about by some users; narrow heads, groups of six, quantised cache
        {"name": "shared_groups", "op": "shared", "seqs": 97, "longest": 900, "spread": 30, "prefixes": 5,
         "prefix": 20000, "prefix_spread": 6, "page": 32, "Hq": 24, "Hkv": 4, "d": 64, "dtype": "bf16",
         "cache": "e4m3"},
        # many samples drawn from one very long context, quantised cache
        {"name": "shared_long", "op": "shared", "seqs": 128, "longest": 500, "spread": 8, "prefixes": 1,
         "prefix": 131072, "prefix_spread": 1, "page": 128, "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16",
         "cache": "e4m3"},
        # float32 layers, as used to check a model's numerics
        {"name": "shared_f32", "op": "shared", "seqs": 8, "longest": 300, "spread": 4, "prefixes": 2, "prefix": 2049,
         "prefix_spread": 3, "page": 32, "Hq": 8, "Hkv": 4, "d": 64, "dtype": "f32", "cache": "io"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "shared", "shared", "shared"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    case = {"op": op, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]),
            "page": rng.choice([16, 32, 64, 128, 256])}
    case["spread"] = _log_int(rng, 1, 50)
    if op == "append":
        case["longest"] = _log_int(rng, 1, 4000)
        case["seqs"] = _log_int(rng, 1, min(100, 30000 // case["longest"]))
        case["past"] = _log_int(rng, 1, 3000)
        case["pairs"] = rng.choice(["halves", "neighbours"])
    elif op in ("read", "decode"):
        case["longest"] = _log_int(rng, 1, 20000 if op == "read" else 100000)
        most = int((1e8 if op == "read" else 6e8) / (case["longest"] * Hkv * d))
        case["seqs"] = _log_int(rng, 1, max(1, min(128, most)))
    else:
        # at most a third of the largest listed case's products, an eighth in float32
        budget = (1e9 if case["dtype"] == "f32" else 2.5e9) / d / Hq * 16
        case["prefix"] = _log_int(rng, 1, min(100000, budget))
        case["seqs"] = _log_int(rng, 1, max(1, min(200, int(budget / case["prefix"]))))
        case["prefixes"] = rng.choice([1, 1, _log_int(rng, 1, min(12, case["seqs"]))])
        case["prefix_spread"] = _log_int(rng, 1, 20)
        case["longest"] = _log_int(rng, 1, 1000)
        case["cache"] = rng.choice(["io", "e4m3"])
    return case


def _lengths(case, n_key="seqs", key="longest", spread="spread"):
    """Lengths from longest / spread to longest, spread evenly over their logarithm and then shuffled by
    a fixed rule; the first of the shuffled order is the longest."""
    n, top = case[n_key], case[key]
    low = max(1, top // case[spread])
    at = [(i * 7) % n if n % 7 else (i * 5) % n if n % 5 else i for i in range(n)]
    return [max(1, int(round(top * (low / top) ** (a / max(1, n - 1))))) for a in at]


def _past(case):
    """Tokens before the new ones of each sequence."""
    return [max(0, case["past"] - 37 * i) for i in range(case["seqs"])]


def _members(case):
    """How many sequences begin with each prefix: the later prefixes have fewer."""
    n, k = case["seqs"], case["prefixes"]
    weight = [k - i for i in range(k)]
    ends = [round(n * sum(weight[:i + 1]) / sum(weight)) for i in range(k)]
    return [b - a for a, b in zip([0] + ends, ends)]


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _int32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _offsets(lens, dev):
    return _int32([0] + lens, dev).cumsum(0).to(torch.int32)


def _tables(lens, page, gen, dev):
    """Page tables of several lists of sequences over one shuffled pool, -1 behind each sequence's pages,
    and the pool's page count (a few pages belong to nobody)."""
    need = [[-(-n // page) for n in part] for part in lens]
    n_pages = sum(map(sum, need)) + 3
    perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    tables, start = [], 0
    for part in need:
        used = torch.tensor(part, device=dev)
        first = used.cumsum(0) - used + start
        col = torch.arange(max(1, max(part)), device=dev)
        at = (first[:, None] + col).clamp(max=n_pages - 1)
        tables.append(torch.where(col < used[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32)))
        start += sum(part)
    return tables, n_pages


def _encode(x):
    """Rows of float32 x as e4m3 numbers and their powers of two (biased by 127, as bytes)."""
    bits = x.abs().amax(-1).view(torch.int32)
    # 448 = 1.75 * 2^8: the smallest power whose 448-fold is not below the largest magnitude
    power = ((bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000).to(torch.int32)).clamp(_LOW, _TOP)
    down = ((254 - power) << 23).view(torch.float32)
    return (x * down[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), power.to(torch.uint8)


def _decode(codes, power):
    return codes.float() * (power.int() << 23).view(torch.float32)[..., None]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    Hq, Hkv, d, page, n = case["Hq"], case["Hkv"], case["d"], case["page"], case["seqs"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    def pool(n_pages):
        """One pool's contents: rows of several magnitudes."""
        x = normal(n_pages, Hkv, page, d) * torch.exp(0.4 * normal(n_pages, Hkv, page, 1))
        if case.get("cache") == "io":
            return x.to(dt), None
        codes, power = _encode(x)
        return codes, power.view(torch.float8_e8m0fnu)

    s = dict(case)
    lens = _lengths(case)
    past = _past(case) if "past" in case else [0] * n
    total = [a + b for a, b in zip(lens, past)]
    prefixes = _lengths(case, "prefixes", "prefix", "prefix_spread") if case["op"] == "shared" else [1]
    (table, prefix_table), n_pages = _tables([total, prefixes], page, gen, dev)
    s["k_pool"], s["k_scale"] = pool(n_pages)
    s["v_pool"], s["v_scale"] = pool(n_pages)
    s.update(table=table, kv_len=_int32(total, dev), tokens=sum(total), widest=max(total))
    if case["op"] == "append":
        rows = normal(sum(lens), Hq + 2 * Hkv, d).to(dt)
        inv = _THETA ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
        s.update(q=rows[:, :Hq], k=rows[:, Hq:Hq + Hkv], v=rows[:, Hq + Hkv:], cu_new=_offsets(lens, dev),
                 inv_freq=inv.to(torch.float32).to(dev))
    elif case["op"] != "read":
        s["q"] = normal(n, Hq, d).to(dt)
    if case["op"] == "shared":
        members = _members(case)
        s.update(prefix_table=prefix_table, prefix_len=_int32(prefixes, dev), cu_prefix=_offsets(members, dev),
                 most=max(members), prefix_widest=max(prefixes))
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

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
    kc, kp = _encode(_turn(k, cos, sin, s["pairs"]))
    vc, vp = _encode(v.float())
    byte = torch.uint8
    s["k_pool"].view(byte)[page, :, slot] = kc.view(byte)
    s["v_pool"].view(byte)[page, :, slot] = vc.view(byte)
    s["k_scale"].view(byte)[page, :, slot] = kp
    s["v_scale"].view(byte)[page, :, slot] = vp
    return _appended(s, _turn(q, cos, sin, s["pairs"]).to(q.dtype))


def _appended(s, q):
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _rows_of(s, x, scale, table, width):
    """[sequences, Hkv, width, d] in float32: the tokens of the table's pages."""
    at = table.long().clamp(min=0)
    n, m = at.shape
    byte = torch.uint8
    if scale is None:
        y = x[at].float()
    else:
        y = _decode(x.view(byte)[at].view(x.dtype), scale.view(byte)[at])
    return y.permute(0, 2, 1, 3, 4).reshape(n, s["Hkv"], m * s["page"], s["d"])[:, :, :width]


def _plain_read(s):
    kv_len, dt = s["kv_len"].long(), _DTYPES[s["dtype"]]
    seen = torch.arange(s["widest"], device=kv_len.device) < kv_len[:, None]

    def rows(x, scale):
        return _rows_of(s, x, scale, s["table"], s["widest"]).transpose(1, 2)[seen].to(dt)

    cu = torch.cat([kv_len.new_zeros(1), kv_len.cumsum(0)]).to(torch.int32)
    return {"k": rows(s["k_pool"], s["k_scale"]), "v": rows(s["v_pool"], s["v_scale"]), "cu": cu}


def _part(s, q, table, length, width):
    """Largest score, sum and unnormalised output of queries q [n, Hkv, rows, d] over a table's tokens."""
    K = _rows_of(s, s["k_pool"], s["k_scale"], table, width)
    S = (q @ K.transpose(-1, -2)) * (1.0 / math.sqrt(s["d"]))
    seen = torch.arange(width, device=q.device) < length.long()[:, None, None, None]
    S = S.masked_fill(~seen, -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.exp(S - m)
    return m, p.sum(-1, keepdim=True), p @ _rows_of(s, s["v_pool"], s["v_scale"], table, width)


def _plain_decode(s):
    q = s["q"].float().reshape(s["seqs"], s["Hkv"], -1, s["d"])
    _, l, o = _part(s, q, s["table"], s["kv_len"], s["widest"])
    return (o / l).reshape(s["q"].shape).to(s["q"].dtype)


def _plain_shared(s):
    """The prefix' part for all sequences that share it at once, then each sequence's own part, joined."""
    n, Hkv, d, k, most = s["seqs"], s["Hkv"], s["d"], s["prefixes"], s["most"]
    q = s["q"].float().reshape(n, Hkv, -1, d)
    cu, G = s["cu_prefix"].long(), q.shape[2]
    seq = torch.arange(n, device=q.device)
    of = torch.searchsorted(cu, seq, right=True) - 1                     # a sequence's prefix, and its place there
    at = of * most + seq - cu[of]
    Q = q.new_zeros(k * most, Hkv, G, d)
    Q[at] = q
    Q = Q.reshape(k, most, Hkv, G, d).transpose(1, 2).reshape(k, Hkv, most * G, d)
    m, l, o = (x.reshape(k, Hkv, most, G, -1).transpose(1, 2).reshape(k * most, Hkv, G, -1)[at]
               for x in _part(s, Q, s["prefix_table"], s["prefix_len"], s["prefix_widest"]))
    m1, l1, o1 = _part(s, q, s["table"], s["kv_len"], s["widest"])
    top = torch.maximum(m, m1)
    f, f1 = torch.exp(m - top), torch.exp(m1 - top)
    return ((f * o + f1 * o1) / (f * l + f1 * l1)).reshape(n, -1, d).to(s["q"].dtype)


def run(state):
    s = state
    if own:
        import sparse_exact_kv_gb300 as L

        dt = _DTYPES[s["dtype"]]
        if s["k_scale"] is None:
            layer = L.ExactAttention(s["Hq"], s["Hkv"], s["d"], dt, s["k_pool"], s["v_pool"])
        else:
            layer = L.QuantizedAttention(s["Hq"], s["Hkv"], s["d"], dt, s["k_pool"], s["v_pool"], s["k_scale"],
                                         s["v_scale"])
        if s["op"] == "append":
            return _appended(s, layer.append(s["k"], s["v"], s["kv_len"], s["table"], cu_new=s["cu_new"], q=s["q"],
                                             inv_freq=s["inv_freq"], pairs=s["pairs"]))
        if s["op"] == "read":
            return dict(zip(("k", "v", "cu"), layer.read(s["kv_len"], s["table"], s["tokens"])))
        if s["op"] == "decode":
            return layer.decode_step(s["q"], s["kv_len"], s["table"])
        return layer.decode_shared(s["q"], s["kv_len"], s["table"], s["prefix_len"], s["prefix_table"],
                                   s["cu_prefix"])
    return {"append": _plain_append, "read": _plain_read, "decode": _plain_decode,
            "shared": _plain_shared}[s["op"]](s)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------------------

def work(case):
    Hq, Hkv, d, n = case["Hq"], case["Hkv"], case["d"], case["seqs"]
    io = 2 if case["dtype"] == "bf16" else 4
    row = io * d if case.get("cache") == "io" else d + 1        # a token's key (or value) of one head
    lens = _lengths(case)
    tokens = sum(lens)
    if case["op"] == "append":
        # q read and written, k and v read, their codes written; a rotation is 3 operations an element, a
        # quantisation 2 (magnitude, scaling)
        return {"bytes": tokens * (2 * io * d * Hq + 2 * Hkv * (io * d + row)), "flops": tokens * d * (3 * Hq + 7 * Hkv)}
    if case["op"] == "read":
        return {"bytes": tokens * 2 * Hkv * (row + io * d), "flops": 2 * tokens * Hkv * d}
    pairs, keys = tokens, tokens
    if case["op"] == "shared":
        prefixes = _lengths(case, "prefixes", "prefix", "prefix_spread")
        pairs += sum(a * b for a, b in zip(_members(case), prefixes))
        keys += sum(prefixes)
    return {"bytes": 2 * Hkv * keys * row + 2 * n * Hq * d * io, "flops": 4 * d * Hq * pairs}


def _codes64(x):
    """e4m3 numbers and powers of two (values, in 64 bits) of the rows x."""
    top = x.abs().amax(-1, keepdim=True)
    power = torch.ceil(torch.log2(top / 448)).clamp(_LOW - 127, _TOP - 127)
    power = torch.where(top <= 448 * 2.0 ** (power - 1), power - 1, power).clamp(_LOW - 127, _TOP - 127)
    y = x / 2.0 ** power
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448), 2.0 ** power[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    lens = _lengths(case)
    dev = s["table"].device

    def cached(which, row, n, h):
        """Tokens 0 .. n - 1 of a page table's row, one head."""
        pages = row[:-(-n // page)].long()
        x = s[which + "_pool"][:, h].view(torch.uint8)[pages].view(s[which + "_pool"].dtype).double()
        if s[which + "_scale"] is not None:
            x = x * 2.0 ** (s[which + "_scale"].view(torch.uint8)[pages, h].double() - 127)[..., None]
        return x.reshape(-1, d)[:n]

    if case["op"] == "append":
        past, freq = _past(case), s["inv_freq"].double()
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        held = {w: s[w + "_pool"].double() for w in "kv"}
        powers = {w: 2.0 ** (s[w + "_scale"].view(torch.uint8).double() - 127) for w in "kv"}
        r = 0
        for b, n in enumerate(lens):
            p = torch.arange(past[b], past[b] + n, device=dev)
            turn = torch.polar(torch.ones(n, d // 2, dtype=torch.float64, device=dev), p[:, None] * freq)[:, None]

            def turned(x):
                if case["pairs"] == "halves":
                    z = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn
                    return torch.cat([z.real, z.imag], -1)
                return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous())
                                          * turn).flatten(-2)

            out[r:r + n] = turned(s["q"][r:r + n].double())
            at = s["table"][b].long()[p // page], p % page
            for w, x in (("k", turned(s["k"][r:r + n].double())), ("v", s["v"][r:r + n].double())):
                held[w][at[0], :, at[1]], powers[w][at[0], :, at[1]] = _codes64(x)
            r += n
        return {"q": out, "k_pool": held["k"], "v_pool": held["v"], "k_scale": powers["k"], "v_scale": powers["v"]}
    if case["op"] == "read":
        k, v = (torch.cat([torch.stack([cached(w, s["table"][b], n, h) for h in range(Hkv)], 1)
                           for b, n in enumerate(lens)]) for w in "kv")
        return {"k": k, "v": v, "cu": None}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    members = _members(case) if case["op"] == "shared" else [1] * len(lens)
    prefixes = _lengths(case, "prefixes", "prefix", "prefix_spread") if case["op"] == "shared" else [0] * len(lens)
    for h in range(Hkv):
        g, b = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)), 0
        for i, count in enumerate(members):
            k0, v0 = (cached(w, s["prefix_table"][i], prefixes[i], h) for w in "kv") if prefixes[i] else (None, None)
            for b in range(b, b + count):
                k, v = (cached(w, s["table"][b], lens[b], h) for w in "kv")
                q = s["q"][b, g].double()
                S = q @ k.T
                if k0 is not None:
                    S = torch.cat([q @ k0.T, S], -1)
                P = torch.softmax(S / d ** 0.5, -1)
                out[b, g] = P[:, S.shape[1] - lens[b]:] @ v
                if k0 is not None:
                    out[b, g] += P[:, :S.shape[1] - lens[b]] @ v0
            b += 1 if count else 0
    return out
