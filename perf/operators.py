"""The training-side operators of the sequence-parallel path: what is timed,
on which sizes, and their plain forms.

Four operators over the shards of a Ulysses group (P virtual ranks on one
GPU):

* ``norm_rope``: the RMS norm of every query and key head and the rotation by
  the row's position, in one pass over the q and k shards;
* ``norm_rope_backward``: its gradient (dq, dk and the two norm weights');
* ``sp_backward``: the gradient of the fused attention on the seq-sharded
  shards;
* ``backward``: the gradient of the attention on the head-sharded layout.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the
library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
F32_SCORES = 1 << 31  # score-matrix elements that the plain form holds at a time (a chunk of heads)


# ------------------------------------------------------------------ cases --
def _attn(name, op, B, P, lens, R, mode, Hq, Hkv, D, rows="sdpa", mask="all", rep_valid=-1, img_valid=-1, std=1.0):
    return {"name": name, "op": op, "B": B, "P": P, "lens": ",".join(map(str, lens)), "R": R, "mode": mode, "Hq": Hq,
            "Hkv": Hkv, "D": D, "rows": rows, "mask": mask, "rep_valid": rep_valid, "img_valid": img_valid,
            "std": std}


def _norm(name, op, B, P, lens, R, mode, Hq, Hkv, D, pairs="interleaved", packed=False, per_batch=False):
    return {"name": name, "op": op, "B": B, "P": P, "lens": ",".join(map(str, lens)), "R": R, "mode": mode, "Hq": Hq,
            "Hkv": Hkv, "D": D, "pairs": pairs, "packed": packed, "per_batch": per_batch}


def listed():
    return [
        # the smallest training step: two ranks, a short text prefix with masked padding; latency counts
        _attn("sp_backward tiny", "sp_backward", 1, 2, (56, 56), 16, "prefix", 4, 4, 64, mask="ranges", rep_valid=10),
        # joint text+image layer of the largest video workload: 40 heads over 4 ranks, padded text prefix
        _attn("sp_backward wan14b", "sp_backward", 1, 4, (6820,) * 4, 512, "prefix", 40, 40, 128, mask="ranges",
              rep_valid=226),
        # grouped-query layer with text keys only (no text queries): dk, dv summed over four query heads
        _attn("sp_backward gqa", "sp_backward", 2, 4, (4096,) * 4, 256, "kv_prefix", 32, 8, 128, std=0.7),
        # ragged last shards, text suffix, padded rows as a sequence of their own
        _attn("sp_backward ragged", "sp_backward", 2, 2, (700, 1213), 100, "suffix", 8, 4, 128, rows="self",
              mask="ranges", rep_valid=63, img_valid=1850),
        # self-attention layer after the exchange (head-sharded tensors), no text
        _attn("backward wan1.3b", "backward", 1, 4, (8190,) * 4, 0, "none", 12, 12, 128, std=0.5),
        # 64-wide heads, odd rows, scattered key mask whose rows give no output
        _attn("backward odd", "backward", 2, 2, (1111, 1111), 77, "suffix", 12, 4, 64, rows="zero", mask="random"),
        # one new token of each of eight sequences before attention: latency
        _norm("norm_rope token", "norm_rope", 8, 1, (1,), 0, "none", 40, 8, 128, pairs="half"),
        # every q and k row of the largest video workload
        _norm("norm_rope wan14b", "norm_rope", 1, 4, (6820,) * 4, 512, "prefix", 40, 40, 128),
        # 64-wide heads read in place from a packed qkv projection, positions of their own per sequence
        _norm("norm_rope packed", "norm_rope", 3, 2, (1777, 901), 0, "none", 24, 8, 64, pairs="half", packed=True,
              per_batch=True),
        # the gradients of the same passes
        _norm("norm_rope_backward wan14b", "norm_rope_backward", 1, 4, (6820,) * 4, 512, "prefix", 40, 40, 128),
        _norm("norm_rope_backward odd", "norm_rope_backward", 2, 2, (333, 333), 19, "kv_prefix", 6, 2, 64,
              pairs="half"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sp_backward", "sp_backward", "backward", "norm_rope", "norm_rope_backward"))
    B, P, D = rng.choice((1, 1, 2, 3)), rng.choice((1, 2, 4)), rng.choice((64, 128, 128))
    Hkv = P * rng.choice((1, 1, 2, 3))
    Hq = Hkv * rng.choice((1, 1, 2, 4))
    # (attention from four rows on: over a single key the gradients of q and k are zero)
    total = _log(rng, P if op.startswith("norm_rope") else 4, 12000)
    lens = [max(1, total // P)] * P
    if P > 1 and rng.random() < 0.5:  # uneven shards
        lens[-1] = max(1, lens[-1] - rng.randrange(0, lens[-1] + 1) // 2)
        lens[0] += rng.randrange(0, 1 + lens[0] // 3)
    mode = rng.choice(("none", "prefix", "suffix", "kv_prefix"))
    R = 0 if mode == "none" else _log(rng, 1, 600)
    if op.startswith("norm_rope"):
        c = _norm("", op, B, P, lens, R, mode, Hq, Hkv, D, rng.choice(("interleaved", "half")),
                  rng.random() < 0.4, rng.random() < 0.4)
    else:
        mask = rng.choice(("all", "ranges", "ranges", "random"))
        c = _attn("", op, B, P, lens, R, mode, Hq, Hkv, D, rng.choice(("sdpa", "sdpa", "zero", "self")), mask,
                  rng.randrange(0, R + 1), rng.randrange(2, sum(lens) + 1) if rng.random() < 0.5 else -1,
                  rng.choice((1.0, 0.5)))
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes --
def _lens(c):
    return [int(x) for x in c["lens"].split(",")]


def _rep(c):
    """(replicated q rows, replicated k/v rows)"""
    return (c["R"] if c["mode"] in ("prefix", "suffix") else 0), c["R"]


def _totals(c):
    n = sum(_lens(c))
    rq, rk = _rep(c)
    return n + rq, n + rk


def work(c):
    B, P, Hq, Hkv, D, lens = c["B"], c["P"], c["Hq"], c["Hkv"], c["D"], _lens(c)
    rq, rk = _rep(c)
    if c["op"].startswith("norm_rope"):
        back = c["op"] == "norm_rope_backward"
        el = B * D * (Hq * (sum(lens) + P * rq) + Hkv * (sum(lens) + P * rk))
        table = (B if c["per_batch"] else 1) * _totals(c)[1] * D * 4
        return {"bytes": (6 if back else 4) * el + table + (16 if back else 8) * D, "flops": (20 if back else 10) * el}
    nq, nk = _totals(c)
    adm = nk
    if c["mask"] == "ranges":
        adm = (rk if c["rep_valid"] < 0 else c["rep_valid"]) + (sum(lens) if c["img_valid"] < 0 else c["img_valid"])
    elif c["mask"] == "random":
        adm = int(0.7 * nk)
    # query rows whose own token is masked: zero or a sequence of their own
    dead = (nk - adm) * nq / nk if c["rows"] != "sdpa" else 0
    pairs = (nq - dead) * adm + (dead * (nk - adm) if c["rows"] == "self" else 0)
    if c["op"] == "sp_backward":
        sq, sk = sum(lens) + P * rq, sum(lens) + P * rk
    else:
        sq, sk = nq, nk
    el = B * D * (4 * Hq * sq + 4 * Hkv * sk)  # q, o, do, dq; k, v, dk, dv
    return {"bytes": 2 * el + 4 * B * Hq * sq, "flops": 10 * B * Hq * D * pairs}


# ------------------------------------------------------------------ inputs --
def _randn(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _to_shards(c, x, is_kv):
    """Global rows (replicated ones where the mode has them) -> one contiguous tensor per shard."""
    lens, R = _lens(c), _rep(c)[is_kv]
    if c["mode"] == "suffix":
        img, rep = x[:, :sum(lens)], x[:, sum(lens):]
        return [torch.cat([i, rep], 1) for i in img.split(lens, 1)]
    return [torch.cat([x[:, :R], i], 1) for i in x[:, R:].split(lens, 1)]


def _to_ranks(c, x):
    return [y.contiguous() for y in x.chunk(c["P"], 2)]


def _key_mask(c, g):
    """[B, Nk] truth values, and the arguments that say so."""
    nk, n = _totals(c)[1], sum(_lens(c))
    R = c["R"]
    if c["mask"] == "random":
        m = torch.rand((c["B"], nk), generator=g, device=DEV) < 0.7
        return m, {"key_mask": m}
    if c["mask"] == "all":
        return torch.ones((c["B"], nk), dtype=torch.bool, device=DEV), {}
    rv, iv = (R if c["rep_valid"] < 0 else c["rep_valid"]), (n if c["img_valid"] < 0 else c["img_valid"])
    r0, i0 = (n, 0) if c["mode"] == "suffix" else (0, R)
    pairs = torch.tensor([[r0, r0 + rv], [i0, i0 + iv]], dtype=torch.int32, device=DEV)
    m = torch.zeros((c["B"], nk), dtype=torch.bool, device=DEV)
    m[:, r0:r0 + rv] = True
    m[:, i0:i0 + iv] = True
    return m, {"key_ranges": pairs[None].expand(c["B"], 2, 2).contiguous()}


def _own_token(c, m):
    """[B, Nq]: is the row's own token an admitted key?"""
    return m[:, c["R"]:] if c["mode"] == "kv_prefix" else m


def _allowed(c, m, own_q):
    """[B, Nq or 1, Nk] truth values of admitted (query, key) pairs."""
    if c["rows"] == "self":
        return m[:, None, :] == own_q[:, :, None]
    if c["rows"] == "zero":
        return m[:, None, :] & own_q[:, :, None]
    return m[:, None, :]


def _forward(c, q, k, v, m):
    """Attention's output and log-sum-exp (bf16 [B, Nq, Hq, D], f32 [B, Nq, Hq]) of global tensors."""
    B, nq, Hq, D = q.shape
    G = Hq // c["Hkv"]
    o, lse = torch.empty_like(q), torch.empty((B, nq, Hq), device=DEV)
    ok = _allowed(c, m, _own_token(c, m))
    for b in range(B):
        for h in range(Hq):
            s = (q[b, :, h].float() @ k[b, :, h // G].float().T) / math.sqrt(D)
            s.masked_fill_(~ok[b], -math.inf)
            l = torch.logsumexp(s, 1)
            lse[b, :, h] = l
            o[b, :, h] = (torch.exp(s - torch.where(l == -math.inf, 0.0, l)[:, None]) @ v[b, :, h // G].float())
    return o, lse


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, P, Hq, Hkv, D, lens = c["B"], c["P"], c["Hq"], c["Hkv"], c["D"], _lens(c)
    nq, nk = _totals(c)
    s = {"case": c}
    if c["op"].startswith("norm_rope"):
        rq, rk = _rep(c)
        rows = [(n + rq, n + rk) for n in lens]
        if c["packed"] and rq == rk:
            # one projection output per shard, q and k read in place: [B, rows, Hq + 2 Hkv, D]
            qkv = [_randn(g, (B, a, Hq + 2 * Hkv, D)) for a, _ in rows]
            s["q"], s["k"] = [x[:, :, :Hq] for x in qkv], [x[:, :, Hq:Hq + Hkv] for x in qkv]
        else:
            s["q"], s["k"] = [_randn(g, (B, a, Hq, D)) for a, _ in rows], [_randn(g, (B, a, Hkv, D)) for _, a in rows]
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
        # positions in global key order; text rows are not rotated
        pos = torch.arange(nk, device=DEV, dtype=torch.float64)
        pos = pos - rk if c["mode"] != "suffix" else torch.where(pos < nk - rk, pos, -1.0)
        pos = pos.clamp(min=0)[None].expand(B if c["per_batch"] else 1, nk).clone()
        if c["per_batch"]:
            pos += torch.randint(0, 5000, (B, 1), generator=g, device=DEV)
        ang = pos[..., None] * 10000.0 ** (-2.0 * torch.arange(D // 2, device=DEV, dtype=torch.float64) / D)
        s["cos"], s["sin"] = (f(ang).float() if c["per_batch"] else f(ang)[0].float() for f in (torch.cos, torch.sin))
        if c["op"] == "norm_rope_backward":
            s["gq"], s["gk"] = [_randn(g, tuple(x.shape)) for x in s["q"]], [_randn(g, tuple(x.shape)) for x in s["k"]]
            s["dwq"], s["dwk"] = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
        s["oq"], s["ok"] = ([torch.empty(tuple(x.shape), dtype=torch.bfloat16, device=DEV) for x in s[n]]
                            for n in ("q", "k"))
    else:
        q = _randn(g, (B, nq, Hq, D), c["std"])
        k, v = (_randn(g, (B, nk, Hkv, D), c["std"]) for _ in range(2))
        m, s["mask_args"] = _key_mask(c, g)
        s["adm"] = m
        o, lse = _forward(c, q, k, v, m)
        fused = c["op"] == "sp_backward"
        s["scale"] = 1.0 / math.sqrt(D)
        for name, x, is_kv in (("q", q, 0), ("k", k, 1), ("v", v, 1), ("o", o, 0), ("lse", lse, 0)):
            s[name] = _to_shards(c, x, is_kv) if fused else _to_ranks(c, x)
        # each shard's copy of the replicated rows has a gradient of its own
        s["do"] = [_randn(g, tuple(x.shape)) for x in s["o"]]
        s["dq"], s["dk"], s["dv"] = ([torch.empty_like(x) for x in s[n]] for n in ("q", "k", "v"))
    if own:
        from ulysses_sequence_attention_uly_gb300 import Plan
        s["plan"] = Plan(B, P, lens[0], c["R"], c["mode"], Hq, Hkv, D, masked_rows=c.get("rows", "sdpa"),
                         shard_lens=lens if len(set(lens)) > 1 else None)
    return s


# ------------------------------------------------------------- plain forms --
def _rot_rows(c, t, p, is_kv):
    """Shard p's rows of a table in global key order, as [1 or B, rows, 1, D / 2]."""
    lens = _lens(c)
    a, b = sum(lens[:p]), sum(lens[:p + 1])
    R = _rep(c)[is_kv]
    t = t if t.dim() == 3 else t[None]
    if c["mode"] == "suffix":
        t = torch.cat([t[:, a:b], t[:, sum(lens):sum(lens) + R]], 1)
    else:
        off = c["R"]
        t = torch.cat([t[:, :R], t[:, off + a:off + b]], 1)
    return t[:, :, None]


def _split(c, x):
    return (x[..., 0::2], x[..., 1::2]) if c["pairs"] == "interleaved" else x.chunk(2, -1)


def _join(c, a, b):
    return torch.stack((a, b), -1).flatten(-2) if c["pairs"] == "interleaved" else torch.cat((a, b), -1)


EPS = 1e-6


def _norm_rope(c, x, w, cos, sin):
    x = x.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    a, b = _split(c, n)
    return _join(c, a * cos - b * sin, a * sin + b * cos).to(torch.bfloat16)


def _norm_rope_backward(c, x, w, cos, sin, g):
    x, g = x.float(), g.float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    z = x * rstd
    a, b = _split(c, g)
    dn = _join(c, a * cos + b * sin, b * cos - a * sin)
    dz = dn * w
    return ((dz - z * (dz * z).mean(-1, keepdim=True)) * rstd).to(torch.bfloat16), (dn * z).sum((0, 1, 2))


def _gather(c, shards, is_kv, total=False):
    """Shards -> global rows: replicated rows from the copy of the shard that owns the head, or the sum of all copies."""
    R = _rep(c)[is_kv]
    lens = _lens(c)
    suffix = c["mode"] == "suffix"
    img = torch.cat([(x[:, :n] if suffix else x[:, R:]).float() for x, n in zip(shards, lens)], 1)
    if not R:
        return img
    reps = torch.stack([(x[:, n:] if suffix else x[:, :R]).float() for x, n in zip(shards, lens)])
    H = reps.shape[3]
    if total:
        rep = reps.sum(0)
    else:
        rep = torch.cat([r[:, :, i * (H // c["P"]):(i + 1) * (H // c["P"])] for i, r in enumerate(reps)], 2)
    return torch.cat([img, rep] if suffix else [rep, img], 1)


def _scatter(c, x, is_kv):
    """The gradient of _gather: replicated rows go to the owner's copy, the other copies get zero."""
    x = x.to(torch.bfloat16)
    R, P = _rep(c)[is_kv], c["P"]
    lens = _lens(c)
    suffix = c["mode"] == "suffix"
    img = (x[:, :sum(lens)] if suffix else x[:, R:]).split(lens, 1)
    rep = x[:, sum(lens):] if suffix else x[:, :R]
    owner = torch.arange(x.shape[2], device=x.device)[:, None] // (x.shape[2] // P)
    reps = [torch.where(owner == p, rep, torch.zeros((), dtype=x.dtype, device=x.device)) for p in range(P)]
    return [torch.cat([i, r] if suffix else [r, i], 1) for i, r in zip(img, reps)]


def _attention_backward(c, s, q, k, v, o, lse, do):
    """dq, dk, dv of global f32 tensors [B, N, H, D].  A kv head's query heads are rows of one matrix; a chunk of
    (batch, kv head) pairs at a time, since all score matrices together would not fit the GPU."""
    B, nq, Hq, D = q.shape
    nk, Hkv = k.shape[1], c["Hkv"]
    G = Hq // Hkv
    rows = lambda x: x.view(B, nq, Hkv, G, -1).permute(0, 2, 3, 1, 4).reshape(B * Hkv, G * nq, -1)  # noqa: E731
    keys = lambda x: x.permute(0, 2, 1, 3).reshape(B * Hkv, nk, D)  # noqa: E731
    delta = rows((o * do).sum(-1, keepdim=True))
    l = rows(torch.where(lse == -math.inf, math.inf, lse)[..., None])
    q, do, k, v = rows(q), rows(do), keys(k), keys(v)
    ok = _allowed(c, s["adm"], _own_token(c, s["adm"]))
    n = max(1, min(B * Hkv, F32_SCORES // (G * nq * nk)))
    got = []
    for i in range(0, B * Hkv, n):
        j = slice(i, i + n)
        sc = torch.baddbmm(l[j], q[j], k[j].transpose(1, 2), beta=-1, alpha=s["scale"])
        p = sc.exp_().view(-1, G, nq, nk)
        if c["mask"] != "all":
            b = torch.arange(i, min(i + n, B * Hkv), device=q.device) // Hkv
            p.mul_(ok[b][:, None])
        p = p.view(-1, G * nq, nk)
        dv = p.transpose(1, 2) @ do[j]
        ds = p.mul_(torch.baddbmm(delta[j], do[j], v[j].transpose(1, 2), beta=-1))
        got.append(((ds @ k[j]) * s["scale"], (ds.transpose(1, 2) @ q[j]) * s["scale"], dv))
    dq, dk, dv = (torch.cat(x) for x in zip(*got))
    dq = dq.view(B, Hkv, G, nq, D).permute(0, 3, 1, 2, 4).reshape(B, nq, Hq, D)
    return [dq] + [x.view(B, Hkv, nk, D).permute(0, 2, 1, 3) for x in (dk, dv)]


def run(state):
    s, c = state, state["case"]
    if own:
        p = s["plan"]
        if c["op"] == "norm_rope":
            p.norm_rope(s["q"], s["k"], s["oq"], s["ok"], s["wq"], s["wk"], s["cos"], s["sin"], pairs=c["pairs"],
                        eps=EPS)
            return {"q": s["oq"], "k": s["ok"]}
        if c["op"] == "norm_rope_backward":
            p.norm_rope_backward(s["q"], s["k"], s["gq"], s["gk"], s["oq"], s["ok"], s["wq"], s["wk"], s["cos"],
                                 s["sin"], s["dwq"], s["dwk"], pairs=c["pairs"], eps=EPS)
            return {"dq": s["oq"], "dk": s["ok"], "dwq": s["dwq"], "dwk": s["dwk"]}
        call = p.sp_attention_backward if c["op"] == "sp_backward" else p.attention_backward
        call(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"], scale=s["scale"],
             **s["mask_args"])
        return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    if c["op"].startswith("norm_rope"):
        args = [(n, p, x, _rot_rows(c, s["cos"], p, i), _rot_rows(c, s["sin"], p, i))
                for i, n in enumerate("qk") for p, x in enumerate(s[n])]
        if c["op"] == "norm_rope":
            out = [_norm_rope(c, x, s["w" + n], cos, sin) for n, p, x, cos, sin in args]
            return {"q": out[:c["P"]], "k": out[c["P"]:]}
        out = [_norm_rope_backward(c, x, s["w" + n], cos, sin, s["g" + n][p]) for n, p, x, cos, sin in args]
        dx, dw = [d for d, _ in out], [d for _, d in out]
        P = c["P"]
        return {"dq": dx[:P], "dk": dx[P:], "dwq": torch.stack(dw[:P]).sum(0), "dwk": torch.stack(dw[P:]).sum(0)}
    if c["op"] == "sp_backward":
        args = [_gather(c, s[n], i, total=n == "do")
                for n, i in (("q", 0), ("k", 1), ("v", 1), ("o", 0), ("lse", 0), ("do", 0))]
        g = _attention_backward(c, s, *args)
        return {n: _scatter(c, x, i) for n, x, i in zip(("dq", "dk", "dv"), g, (0, 1, 1))}
    g = _attention_backward(c, s, *(torch.cat(s[n], 2).float() for n in ("q", "k", "v", "o", "lse", "do")))
    return {n: [y.to(torch.bfloat16) for y in x.chunk(c["P"], 2)] for n, x in zip(("dq", "dk", "dv"), g)}


# ----------------------------------------------------------- in 64 bits --
def _exact_norm(c, s):
    """Norm and rotation as complex products in 64 bits; the gradient by differentiating that."""
    P, D = c["P"], c["D"]
    lens = _lens(c)
    start = [sum(lens[:p]) for p in range(P)]
    n = sum(lens)
    turn = torch.complex(s["cos"].double(), s["sin"].double())
    out, grads = {"q": [], "k": []}, {"q": [], "k": []}
    dw = {}
    for t in "qk":
        R = _rep(c)[t == "k"]
        dw[t] = torch.zeros(D, dtype=torch.float64, device=DEV)
        for p in range(P):
            img = list(range(start[p], start[p] + lens[p]))
            if c["mode"] == "suffix":
                rows = img + list(range(n, n + R))
            else:
                rows = list(range(R)) + [c["R"] + r for r in img]
            tr = turn[..., torch.tensor(rows, device=DEV, dtype=torch.long), :].unsqueeze(-2)
            x = s[t][p].double().requires_grad_(c["op"] != "norm_rope")
            w = s["w" + t].double().requires_grad_(c["op"] != "norm_rope")
            y = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w
            pairs = y.unflatten(-1, (D // 2, 2)) if c["pairs"] == "interleaved" else y.unflatten(-1, (2, D // 2)).mT
            z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * tr)
            y = z.flatten(-2) if c["pairs"] == "interleaved" else z.mT.flatten(-2)
            if c["op"] == "norm_rope":
                out[t].append(y)
            else:
                gx, gw = torch.autograd.grad(y, (x, w), s["g" + t][p].double())
                grads[t].append(gx)
                dw[t] += gw
    if c["op"] == "norm_rope":
        return out
    return {"dq": grads["q"], "dk": grads["k"], "dwq": dw["q"], "dwk": dw["k"]}


def exact(case, seed):
    c = case
    if c["op"].startswith("norm_rope"):
        return _exact_norm(c, prepare(c, seed))
    if work(c)["flops"] > 3e12:
        return None  # most of a minute in 64 bits
    s = prepare(c, seed)
    B, P, Hq, Hkv = c["B"], c["P"], c["Hq"], c["Hkv"]
    lens, n = _lens(c), sum(_lens(c))
    out = {"d" + t: [torch.zeros(x.shape, dtype=torch.float64, device=DEV) for x in s[t]] for t in "qkv"}
    # where each global row lives: a list of (tensor, row) parts per head, by the operator's row order
    adm = s["adm"]

    def parts(h, H, is_kv):
        if c["op"] == "backward":
            return [(h // (H // P), slice(None))], h % (H // P)
        R, r = _rep(c)[is_kv], h // (H // P)
        img = [(p, slice(0, lens[p]) if c["mode"] == "suffix" else slice(R, R + lens[p])) for p in range(P)]
        rep = [(r, slice(lens[r], lens[r] + R) if c["mode"] == "suffix" else slice(0, R))] if R else []
        return (img + rep if c["mode"] == "suffix" else rep + img), h

    def get(ts, b, where, hh):
        return torch.cat([ts[p][b, sl, hh].double() for p, sl in where])

    def put(ts, b, where, hh, x):
        at = 0
        for p, sl in where:
            view = ts[p][b, sl, hh]
            view += x[at:at + view.shape[0]]
            at += view.shape[0]

    rq = _rep(c)[0]
    for b in range(B):
        for h in range(Hq):
            wq, hq = parts(h, Hq, 0)
            wk, hk = parts(h // (Hq // Hkv), Hkv, 1)
            q, o, do = (get(s[t], b, wq, hq) for t in ("q", "o", "do"))
            lse = get(s["lse"], b, wq, hq)
            if c["op"] == "sp_backward" and rq:
                # the replicated rows' output goes to every shard: their gradients add up
                sl = slice(n, n + rq) if c["mode"] == "suffix" else slice(0, rq)
                do[sl] = sum(s["do"][p][b, lens[p]:lens[p] + rq, h].double() if c["mode"] == "suffix"
                             else s["do"][p][b, :rq, h].double() for p in range(P))
            k, v = (get(s[t], b, wk, hk) for t in "kv")
            prob = (q @ k.T * s["scale"] - lse[:, None]).exp()
            mine = adm[b, c["R"]:] if c["mode"] == "kv_prefix" else adm[b]
            if c["rows"] == "self":
                keep = torch.outer(mine, adm[b]) | torch.outer(~mine, ~adm[b])
            else:
                keep = adm[b].expand(len(mine), -1) if c["rows"] == "sdpa" else torch.outer(mine, adm[b])
            prob = torch.where(keep & (lse > -math.inf)[:, None], prob, 0.0)
            ds = prob * (do @ v.T - torch.einsum("nd,nd->n", o, do)[:, None])
            put(out["dq"], b, wq, hq, ds @ k * s["scale"])
            put(out["dk"], b, wk, hk, ds.T @ q * s["scale"])
            put(out["dv"], b, wk, hk, prob.T @ do)
    return out
