"""The serving-side operators: what is timed, on which sizes, and their plain
forms.

* ``prompt``: causal attention over packed prompts of different lengths, on
  the seq-sharded shards of a Ulysses group (P virtual ranks on one GPU);
* ``append``: the k and v rows of new tokens quantised into the pages of an
  8-bit cache (e4m3, one scale for each page and head);
* ``cached``: attention of the newest tokens of every sequence over such a
  cache.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the
library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F32_SCORES = 1 << 31  # score-matrix elements that the plain form of `prompt` holds at a time (a chunk of heads)
LEAST = -60  # smallest exponent of a page's scale


# ------------------------------------------------------------------ cases --
def _prompt(name, shards, seqs, Hq, Hkv, D, std=1.0, first=0):
    """shards: rows of each shard; seqs: lengths of the packed prompts, which begin at row `first`."""
    return {"name": name, "op": "prompt", "shards": ",".join(map(str, shards)), "seqs": ",".join(map(str, seqs)),
            "first": first, "Hq": Hq, "Hkv": Hkv, "D": D, "std": std}


def _append(name, old, new, Hkv, D, page, packed=False):
    """old: tokens in the cache of every sequence; new: tokens that join it."""
    return {"name": name, "op": "append", "old": ",".join(map(str, old)), "new": ",".join(map(str, new)), "Hkv": Hkv,
            "D": D, "page": page, "packed": packed}


def _cached(name, old, new, Hq, Hkv, D, page, std=1.0):
    return {"name": name, "op": "cached", "old": ",".join(map(str, old)), "new": ",".join(map(str, new)), "Hq": Hq,
            "Hkv": Hkv, "D": D, "page": page, "std": std}


def _spread(n, lo, hi, seed):
    r = random.Random(seed)
    return [_log(r, lo, hi) for _ in range(n)]


def listed():
    return [
        # one short prompt: latency counts
        _prompt("prompt short", (17,), (17,), 4, 2, 64),
        # two dozen requests of different lengths in one batch of a grouped-query model, the token budget not filled
        _prompt("prompt batch", (8192,), _spread(24, 30, 900, 1), 32, 8, 128),
        # one long document, a single token and a middling prompt over four shards
        _prompt("prompt long", (4096,) * 4, (12000, 1, 4383), 32, 8, 128, std=0.7),
        # the whole sequence of the largest video workload generated in causal order: every head its own k and v
        _prompt("prompt wan14b", (6820,) * 4, (27280,), 40, 40, 128),
        # 64-wide heads, uneven shards, empty sequences, rows before the first and behind the last
        _prompt("prompt odd", (1213, 700), (333, 0, 1, 900, 127, 0, 411), 12, 4, 64, first=5),
        # the newest token of each of eight sequences, middle of a page, first of a page: latency
        _append("append token", (700, 64, 63, 5, 1023, 130, 127, 0), (1,) * 8, 8, 128, 64),
        # four prompts go into an empty cache
        _append("append prompts", (0,) * 4, (9000, 1, 4383, 3000), 8, 128, 64),
        # a few tokens of each sequence join half-filled small pages, read in place from a packed projection
        _append("append odd", (17, 0, 250, 16, 1000), (3, 40, 1, 16, 7), 3, 64, 16, packed=True),
        # one sequence, one token: latency
        _cached("cached token", (499,), (1,), 32, 8, 128, 64),
        # a serving batch of 64 sequences of different lengths, one token each
        _cached("cached batch", _spread(64, 200, 8000, 2), (1,) * 64, 32, 8, 128, 64),
        # two long contexts, one token each
        _cached("cached long", (119999, 131071), (1, 1), 32, 8, 128, 128, std=0.7),
        # a few guessed tokens a sequence, checked at once; 64-wide heads, small pages, short and empty sequences
        _cached("cached odd", (0, 1, 15, 300, 2000, 777, 4096), (3, 3, 1, 3, 3, 0, 3), 12, 4, 64, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "append", "cached", "cached"))
    D, G = rng.choice((64, 128, 128)), rng.choice((1, 2, 3, 4, 5, 8))
    if op == "prompt":
        P = rng.choice((1, 1, 2, 4))
        Hkv = P * rng.choice((1, 2, 3, 8 // P))
        total = _log(rng, P, 14000)
        seqs, left = [], total - rng.choice((0, 0, rng.randrange(0, total)))
        first = min(left - 1, rng.choice((0, 0, rng.randrange(0, 200))))
        left -= first
        most = _log(rng, 1, 2 * total)
        while left > 0 and len(seqs) < 200:
            n = min(left, rng.randrange(0, most + 1))
            seqs.append(n)
            left -= n
        shards = [max(1, total // P)] * P
        if P > 1 and rng.random() < 0.5:  # uneven shards
            shards[0] += shards[-1] // 3
        shards[-1] += max(0, total - sum(shards))
        if not any(seqs):
            seqs.append(1)
        c = _prompt("", shards, seqs, min(Hkv * G, 40 // P * P // Hkv * Hkv or Hkv), Hkv, D,
                    rng.choice((1.0, 0.6)), first)
    else:
        Hkv, page, n = rng.choice((1, 2, 3, 8)), rng.choice((16, 32, 64, 128)), _log(rng, 1, 64)
        if op == "append":
            most = _log(rng, 1, 16000 // n)
            c = _append("", [rng.randrange(0, 400) for _ in range(n)], [rng.randrange(0, most + 1) for _ in range(n)],
                        Hkv, D, page, rng.random() < 0.4)
            if not any(int(x) for x in c["new"].split(",")):
                c["new"] = ",".join(["1"] * n)
        else:
            most = _log(rng, 4, 200000 // n)
            T = rng.choice((1, 1, 1, 2, 3, 5, 8))
            new = [T if rng.random() < 0.8 else rng.randrange(0, T + 1) for _ in range(n)]
            new[0] = max(1, new[0])
            c = _cached("", [rng.randrange(most // 4, most) for _ in range(n)], new, Hkv * G, Hkv, D, page,
                        rng.choice((1.0, 0.6)))
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes --
def _ints(c, key):
    return [int(x) for x in c[key].split(",")]


def work(c):
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "prompt":
        seqs, Hq = _ints(c, "seqs"), c["Hq"]
        rows = sum(seqs)
        return {"bytes": rows * (4 * D * (Hq + Hkv) + 4 * Hq) + 4 * len(seqs),
                "flops": 2 * Hq * D * sum(n * (n + 1) for n in seqs)}
    old, new, page = _ints(c, "old"), _ints(c, "new"), c["page"]
    rows = sum(new)
    if c["op"] == "append":
        blocks = sum(-(-(a + n) // page) - a // page for a, n in zip(old, new) if n)
        return {"bytes": rows * Hkv * D * 6 + 2 * blocks * (4 * Hkv + 2) + 8 * len(new), "flops": 4 * rows * Hkv * D}
    Hq = c["Hq"]
    lens = [a + n for a, n in zip(old, new)]
    kept = sum(n for n, t in zip(lens, new) if t)  # (a sequence without a new token is not read)
    pages = sum(-(-n // page) for n, t in zip(lens, new) if t)
    return {"bytes": 2 * Hkv * (kept * D + 4 * pages) + 4 * pages + rows * Hq * (4 * D + 4) + 8 * len(lens),
            "flops": 4 * Hq * D * sum(a * t + t * (t + 1) // 2 for a, t in zip(old, new))}


# ------------------------------------------------------------------ inputs --
def _randn(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _keys(g, shape):
    """Keys with a few channels much larger than the rest, as projections have them."""
    big = torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device=DEV))
    return (torch.randn(shape, generator=g, device=DEV) * big).to(torch.bfloat16)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return _int32(at)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, at least LEAST."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e.clamp(min=LEAST), LEAST)


def _filled(g, c, lens, width, extra):
    """Pages of a cache that holds lens[s] tokens of every sequence, and the table that says where; pages are taken in
    no order, and a table's entries behind the last page are -1."""
    H, D, page, n = c["Hkv"], c["D"], c["page"], len(lens)
    used = [-(-a // page) for a in lens]
    total = sum(used) + extra
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(width, device=DEV)[None] + (_starts(used)[:-1])[:, None]
    have = torch.arange(width, device=DEV)[None] < _int32(used)[:, None]
    table = torch.where(have, order[at.clamp(max=total - 1)], -1).to(torch.int32).contiguous()
    free = order[sum(used):]
    pools = []
    for make in (_keys, _randn):
        x = make(g, (total, page, H, D)).float().permute(0, 2, 1, 3)
        e = _exponent(x.abs().amax((2, 3)))
        codes = (x * torch.exp2(-e.float())[..., None, None]).to(torch.float8_e4m3fn)
        pools += [codes.contiguous(), torch.exp2(e.float())]
    return pools, table, free


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    D, Hkv = c["D"], c["Hkv"]
    s = {"case": c}
    if c["op"] == "prompt":
        shards, Hq = _ints(c, "shards"), c["Hq"]
        s["q"] = [_randn(g, (1, n, Hq, D), c["std"]) for n in shards]
        s["k"] = [_randn(g, (1, n, Hkv, D), c["std"]) for n in shards]
        s["v"] = [_randn(g, (1, n, Hkv, D)) for n in shards]
        # rows of no sequence keep what they hold
        s["o"] = [_randn(g, (1, n, Hq, D)) for n in shards]
        s["lse"] = [torch.randn((1, n, Hq), generator=g, device=DEV) for n in shards]
        s["starts"] = _starts(_ints(c, "seqs"), c["first"])
        s["scale"] = 1.0 / math.sqrt(D)
        if own:
            from ulysses_sequence_attention_uly_gb300 import Plan
            s["plan"] = Plan(1, len(shards), shards[0], 0, "none", Hq, Hkv, D,
                             shard_lens=shards if len(set(shards)) > 1 else None)
        return s
    old, new, page = _ints(c, "old"), _ints(c, "new"), c["page"]
    lens = [a + n for a, n in zip(old, new)]
    rows = sum(new)
    width = max(-(-n // page) for n in lens) + 1
    s["starts"], s["lens"] = _starts(new), _int32(lens)
    s["pools"], s["table"], _ = _filled(g, c, lens, width, 3)
    if c["op"] == "append":
        if c["packed"]:  # the k and v parts of one projection's output, next to a q part as wide
            qkv = torch.cat((_randn(g, (rows, Hkv, D)), _keys(g, (rows, Hkv, D)), _randn(g, (rows, Hkv, D))), 1)
            s["k"], s["v"] = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
        else:
            s["k"], s["v"] = _keys(g, (rows, Hkv, D)), _randn(g, (rows, Hkv, D))
    else:
        s["q"] = _randn(g, (rows, c["Hq"], D), c["std"])
        s["o"] = torch.empty((rows, c["Hq"], D), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((rows, c["Hq"]), device=DEV)
        s["scale"] = 1.0 / math.sqrt(D)
    if own:
        from ulysses_sequence_attention_uly_gb300 import Cache
        k, ks, v, vs = s["pools"]
        s["cache"] = Cache(k, v, ks, vs)
    return s


# ------------------------------------------------------------- plain forms --
def _plain_prompt(s):
    c = s["case"]
    q, k, v = (torch.cat(s[n], 1)[0].float() for n in ("q", "k", "v"))
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    row = torch.arange(N, device=DEV)
    seq = torch.searchsorted(s["starts"][1:].long().contiguous(), row, right=True)
    inside = (row >= s["starts"][0]) & (row < s["starts"][-1])
    ok = (seq[:, None] == seq[None]) & (row[:, None] >= row[None]) & inside[None]
    q = q.view(N, Hkv, G, D).permute(1, 2, 0, 3)
    k, v = k.transpose(0, 1), v.transpose(0, 1)
    n = max(1, F32_SCORES // (G * N * N))
    o, lse = [], []
    for i in range(0, Hkv, n):  # a chunk of heads: all score matrices together would not fit the GPU
        sc = (q[i:i + n] * s["scale"]).reshape(-1, G * N, D) @ k[i:i + n].transpose(1, 2)
        sc = sc.view(-1, G, N, N).masked_fill_(~ok, -math.inf)
        top = sc.amax(-1, keepdim=True).clamp_(min=-3e38)
        e = sc.sub_(top).exp_()
        z = e.sum(-1, keepdim=True)
        o.append((e.view(-1, G * N, N) @ v[i:i + n]).view(-1, G, N, D) / z)
        lse.append((top + z.log())[..., 0])
    o, lse = (torch.cat(x) for x in (o, lse))
    o = torch.where(inside[:, None, None], o.permute(2, 0, 1, 3).reshape(N, Hq, D).to(torch.bfloat16),
                    torch.cat(s["o"], 1)[0])
    lse = torch.where(inside[:, None], lse.permute(2, 0, 1).reshape(N, Hq), torch.cat(s["lse"], 1)[0])
    shards = _ints(c, "shards")
    return {"o": o[None].split(shards, 1), "lse": lse[None].split(shards, 1)}


def _rows_of(s):
    """Sequence and position in the cache of every new row."""
    starts, lens = s["starts"].long(), s["lens"].long()
    row = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    return seq, lens[seq] - starts[seq + 1] + row, row == starts[seq]


def _plain_append(s):
    page = s["case"]["page"]
    seq, pos, first = _rows_of(s)
    at, slot = s["table"].long()[seq, pos // page], pos % page
    lead = first | (slot == 0)  # the first new row of its page
    pages, slot0 = at[lead], slot[lead]
    out = []
    for x, codes, scale in ((s["k"], *s["pools"][:2]), (s["v"], *s["pools"][2:])):
        x = x.float()
        amax = torch.zeros_like(scale).index_reduce_(0, at, x.abs().amax(-1), "amax")[pages]
        need = torch.exp2(_exponent(amax).float())
        have = scale[pages]
        now = torch.where(slot0[:, None] == 0, need, torch.maximum(have, need))
        # tokens that were in the page before
        was = codes[pages].float()
        again = (was * (have / now)[..., None, None]).to(torch.float8_e4m3fn)
        keep = torch.arange(page, device=DEV) < slot0[:, None]
        codes[pages] = torch.where(keep[:, None, :, None], again.float(), was).to(torch.float8_e4m3fn)
        scale[pages] = now
        codes[at, :, slot] = (x / scale[at][..., None]).to(torch.float8_e4m3fn)
        out += [codes, scale]
    return dict(zip(("k", "k_scale", "v", "v_scale"), out))


def _plain_cached(s):
    c = s["case"]
    D, Hq, Hkv, page = c["D"], c["Hq"], c["Hkv"], c["page"]
    G = Hq // Hkv
    kc, ks, vc, vs = s["pools"]
    at = s["table"].long().clamp(min=0)
    n, width = at.shape
    k, v = ((codes[at].float() * scale[at][..., None, None]).permute(0, 2, 1, 3, 4).reshape(n, Hkv, width * page, D)
            for codes, scale in ((kc, ks), (vc, vs)))
    starts, lens = s["starts"].long(), s["lens"].long()
    T = max(_ints(c, "new"))
    t = torch.arange(T, device=DEV)
    count = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    live = t < count[:, None]
    q = s["q"][row].float().view(n, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, G * T, D)
    sc = (q * s["scale"]) @ k.transpose(2, 3)
    limit = (lens - count)[:, None] + t + 1  # keys that a token sees
    ok = torch.arange(width * page, device=DEV) < limit[..., None]
    sc = sc.view(n, Hkv, G, T, -1).masked_fill_(~ok[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True).clamp_(min=-3e38)
    e = (sc - top).exp()
    z = e.sum(-1, keepdim=True)
    v = torch.where((torch.arange(width * page, device=DEV) < lens[:, None])[:, None, :, None], v, 0.0)
    o = (e.view(n, Hkv, G * T, -1) @ v).view(n, Hkv, G, T, D) / z
    lse = (top + z.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, T, Hq, D)[live]
    return {"o": o.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(n, T, Hq)[live]}


def run(state):
    s, c = state, state["case"]
    if own:
        if c["op"] == "prompt":
            s["plan"].prompt_attention(s["q"], s["k"], s["v"], s["o"], s["starts"], scale=s["scale"], lse=s["lse"])
            return {"o": s["o"], "lse": s["lse"]}
        if c["op"] == "append":  # the values of the codes, and the scales that multiply them
            s["cache"].append(s["k"], s["v"], s["starts"], s["lens"], s["table"])
            return dict(zip(("k", "k_scale", "v", "v_scale"), s["pools"]))
        s["cache"].attention(s["q"], s["o"], s["starts"], s["lens"], s["table"], scale=s["scale"], lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    return {"prompt": _plain_prompt, "append": _plain_append, "cached": _plain_cached}[c["op"]](s)


# ----------------------------------------------------------- in 64 bits --
def exact(case, seed):
    c = case
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "prompt":
        seqs = _ints(c, "seqs")
        if 4 * c["Hq"] * D * sum(n * n for n in seqs) > 8e12:
            return None  # over ten seconds in 64 bits
        s = prepare(c, seed)
        q, k, v, o, lse = (torch.cat(s[n], 1)[0].double() for n in ("q", "k", "v", "o", "lse"))
        at = c["first"]
        for n in seqs:
            for h in range(c["Hq"]):
                g = h * Hkv // c["Hq"]
                z = torch.einsum("id,jd->ij", q[at:at + n, h], k[at:at + n, g]) * s["scale"]
                z += torch.full_like(z, -math.inf).triu(1)
                lse[at:at + n, h] = z.logsumexp(1)
                o[at:at + n, h] = z.softmax(1) @ v[at:at + n, g]
            at += n
        shards = _ints(c, "shards")
        return {"o": o[None].split(shards, 1), "lse": lse[None].split(shards, 1)}
    s = prepare(c, seed)
    page, old, new = c["page"], _ints(c, "old"), _ints(c, "new")
    table = s["table"].tolist()
    kc, ks, vc, vs = (x.double() for x in s["pools"])
    if c["op"] == "append":
        out = {}
        for name, codes, scale in (("k", kc, ks), ("v", vc, vs)):
            x, at = s[name].double(), 0
            for i, (a, n) in enumerate(zip(old, new)):
                for j in range(a // page, -(-(a + n) // page) if n else 0):
                    p, lo, hi = table[i][j], max(a - j * page, 0), min(a + n - j * page, page)
                    part = x[at:at + hi - lo].transpose(0, 1)
                    at += hi - lo
                    # the least power of two with which the largest new value and the old ones fit
                    top = part.abs().amax((1, 2)) / 448
                    m, e = torch.frexp(top)  # (a logarithm would miss exact powers)
                    e = torch.where(top > 0, e - (m == 0.5).int(), LEAST).clamp(min=LEAST).double()
                    now = 2.0 ** e if lo == 0 else torch.maximum(2.0 ** e, scale[p])
                    codes[p, :, :lo] *= (scale[p] / now)[:, None, None]
                    codes[p, :, lo:hi] = part / now[:, None, None]
                    scale[p] = now
            out[name], out[name + "_scale"] = codes, scale
        return out
    o, lse = [], []
    k, v = kc * ks[..., None, None], vc * vs[..., None, None]
    q = s["q"].double().split(new)
    for i, (a, n) in enumerate(zip(old, new)):
        for t in range(n):
            m = a + t + 1
            pages = torch.tensor(table[i][:-(-m // page)], device=DEV)
            kk, vv = (x[pages].transpose(0, 1).flatten(1, 2)[:, :m] for x in (k, v))
            z = torch.einsum("hgd,hjd->hgj", q[i][t].view(Hkv, -1, D), kk) * s["scale"]
            lse.append(z.logsumexp(2).flatten())
            o.append((z.softmax(2) @ vv).flatten(0, 1))
    return {"o": torch.stack(o), "lse": torch.stack(lse)}
