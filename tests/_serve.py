"""The causal attention over packed prompts and the 8-bit cache in 64 bits, from
the definitions in include/uly.h: what the tests compare the kernels with.
Shares no code with the library."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch


@dataclass(frozen=True)
class Prompt:
    name: str
    shards: tuple
    seqs: tuple
    Hq: int
    Hkv: int
    D: int
    first: int = 0
    std: float = 1.0

    @property
    def n(self):
        return sum(self.shards)

    @property
    def bounds(self):
        at = [self.first]
        for x in self.seqs:
            at.append(at[-1] + x)
        return at


def plan_of(c):
    from ulysses_sequence_attention_uly_gb300 import Plan
    return Plan(1, len(c.shards), c.shards[0], 0, "none", c.Hq, c.Hkv, c.D,
                shard_lens=c.shards if len(set(c.shards)) > 1 else None)


def prompt_inputs(c, seed, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)

    def rows(H, std=1.0):
        x = (torch.randn((1, c.n, H, c.D), generator=g, device=dev) * std).to(torch.bfloat16)
        return [y.contiguous() for y in x.split(list(c.shards), 1)]

    d = {"q": rows(c.Hq, c.std), "k": rows(c.Hkv, c.std), "v": rows(c.Hkv)}
    # what rows of no sequence hold before the call, and after it
    d["o"] = [torch.full_like(x, 7.0) for x in d["q"]]
    d["lse"] = [torch.full(x.shape[:3], 7.0, device=dev) for x in d["q"]]
    d["starts"] = torch.tensor(c.bounds, dtype=torch.int32, device=dev)
    return d


def prompt_reference(c, d, scale=None):
    """o and lse in 64 bits as [rows, Hq, ...], the bound of o's error, and which
    rows are a sequence's.

    The bound: the probabilities are operands of a bf16 product (u = 2^-8 each,
    while their sum takes them unrounded) and the output is rounded once (u);
    r = 2^-13 stands for the 32-bit arithmetic, as sums of up to 2^14 terms of
    2^-24 each and the error of the exponential's argument, 2^-23 |s| for |s| up
    to about 60, stay below it."""
    scale = 1.0 / math.sqrt(c.D) if scale is None else scale
    u, r = 2.0 ** -8, 2.0 ** -13
    q, k, v = (torch.cat(d[n], 1)[0].double() for n in "qkv")
    G = c.Hq // c.Hkv
    o, lse, err = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device), torch.zeros_like(q)
    inside = torch.zeros(c.n, dtype=torch.bool, device=q.device)
    for a, b in zip(c.bounds, c.bounds[1:]):
        if a == b:
            continue
        inside[a:b] = True
        kk, vv = (x[a:b].repeat_interleave(G, 1) for x in (k, v))
        s = torch.einsum("ihd,jhd->hij", q[a:b], kk) * scale
        s = s.masked_fill(torch.ones((b - a, b - a), device=q.device).triu(1).bool(), -math.inf)
        lse[a:b] = s.logsumexp(-1).T
        p = s.softmax(-1)
        o[a:b] = torch.einsum("hij,jhd->ihd", p, vv)
        err[a:b] = torch.einsum("hij,jhd->ihd", p, vv.abs()) * (u + r)
    err = err * (1 + u) + u * o.abs() + 1e-30
    return o, lse, err, inside


def check_rows(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), what + ": not finite or not written"
    bad = (got - want).abs() > bound
    assert not bad.any(), "%s: %d elements, worst %.3g of its bound at %s" % (
        what, int(bad.sum()), float(((got - want).abs() / bound).max()), bad.nonzero()[0].tolist())


def check_prompt(c, d, o, lse, scale=None, what="o"):
    """Rows of sequences against the reference, all others as they were."""
    want, wl, err, inside = prompt_reference(c, d, scale)
    got = torch.cat(o, 1)[0]
    check_rows(got[inside], want[inside], err[inside], what)
    assert (got[~inside] == 7.0).all(), what + ": a row of no sequence was written"
    if lse is not None:
        gl = torch.cat(lse, 1)[0]
        check_rows(gl[inside], wl[inside], 2.0 ** -13 + 2.0 ** -22 * wl[inside].abs(), "lse")
        assert (gl[~inside] == 7.0).all(), "lse: a row of no sequence was written"
    return want


# ------------------------------------------------------------------ cache --
@dataclass(frozen=True)
class Cached:
    name: str
    old: tuple
    new: tuple
    H: int
    D: int
    page: int
    G: int = 1
    std: float = 1.0

    @property
    def rows(self):
        return sum(self.new)

    @property
    def lens(self):
        return tuple(a + n for a, n in zip(self.old, self.new))


def ints(v, dev="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def starts_of(new, dev="cuda"):
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    return ints(at, dev)


def cache_inputs(c, seed, dev="cuda", powers=True, spare=2):
    """Random codes in every slot (NaN codes in slots that no token of `old`
    takes), scales, a table of pages in no order with bad entries behind the last
    page, and new rows."""
    g = torch.Generator(device=dev).manual_seed(seed)
    used = [-(-n // c.page) for n in c.lens]
    n = sum(used) + spare
    width = max(max(used), 1) + 1
    order = torch.randperm(n, generator=g, device=dev).tolist()
    table, at = [], 0
    for x in used:
        table.append(order[at:at + x] + [-1, n, 2 ** 31 - 1, -2 ** 31][:1 + (at % 4)][-1:] * (width - x))
        at += x
    d = {"table": ints(table, dev), "starts": starts_of(c.new, dev), "lens": ints(c.lens, dev)}
    shape = (n, c.H, c.page, c.D)
    for t in "kv":
        codes = (torch.randn(shape, generator=g, device=dev) * 30).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        live = torch.zeros((n, c.page), dtype=torch.bool, device=dev)
        for s, m in enumerate(c.old):
            for i in range(-(-m // c.page)):
                live[table[s][i], :min(c.page, m - i * c.page)] = True
        codes = torch.where(live[:, None, :, None], codes, 0x7F).contiguous()
        e = torch.randint(-7, -3, (n, c.H), generator=g, device=dev).float()
        scale = torch.exp2(e)
        if not powers:
            scale = scale * (1 + torch.rand((n, c.H), generator=g, device=dev))
        d[t + "_pages"], d[t + "_scale"] = codes.view(torch.float8_e4m3fn), scale
        d[t] = torch.randn((c.rows, c.H, c.D), generator=g, device=dev).to(torch.bfloat16)
    d["q"] = (torch.randn((c.rows, c.H * c.G, c.D), generator=g, device=dev) * c.std).to(torch.bfloat16)
    return d


def cache_of(d):
    from ulysses_sequence_attention_uly_gb300 import Cache
    return Cache(d["k_pages"], d["v_pages"], d["k_scale"], d["v_scale"])


def least_power(amax):
    """The least 2^e, e >= -60, with amax <= 448 * 2^e, by trying."""
    e = -60
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def appended(c, d):
    """Codes (as 64-bit values, NaN where a code is one) and scales after the call."""
    n_pages = d["k_pages"].shape[0]
    table, starts, lens = (d[n].tolist() for n in ("table", "starts", "lens"))
    out = {}
    for t in "kv":
        codes, scale = d[t + "_pages"].to(torch.float64).cpu(), d[t + "_scale"].double().cpu()
        x = d[t].double().cpu()
        for s in range(len(lens)):
            a, b = starts[s], starts[s + 1]
            parts = {}
            for r in range(a, b):
                pos = lens[s] - (b - a) + r - a
                if 0 <= pos < len(table[s]) * c.page and 0 <= table[s][pos // c.page] < n_pages:
                    parts.setdefault(table[s][pos // c.page], []).append((pos % c.page, r))
            for g, rows in parts.items():
                slot0 = rows[0][0]
                for h in range(c.H):
                    new = x[[r for _, r in rows], h]
                    need = least_power(float(new[~new.isnan()].abs().max()) if (~new.isnan()).any() else 0.0)
                    had = float(scale[g, h])
                    now = need if slot0 == 0 else max(need, had)
                    if slot0 and now != had:
                        codes[g, h, :slot0] = to_e4m3(codes[g, h, :slot0] * (had / now))
                    for (slot, _), row in zip(rows, new):
                        codes[g, h, slot] = to_e4m3(row / now)
                    scale[g, h] = now
        out[t + "_pages"], out[t + "_scale"] = codes, scale
    return out


def to_e4m3(x):
    """Rounded to e4m3 (ties to even), by its grid: steps of 2^(e - 3) from 2^e on, 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return ((x / step).round() * step).clamp(-448, 448)


def cached_reference(c, d, scale=None):
    """o [rows, Hq, D], lse and the bound of o's error.

    The bound: the weights (the exponentials times their pages' scales) are
    operands of an f16 product, 2^-11 of each, or half an f16 step of 2^-24 of the
    largest weight where they are small against it; the output is rounded to bf16
    once (2^-8); r = 2^-13 as for prompts."""
    scale = 1.0 / math.sqrt(c.D) if scale is None else scale
    n_pages = d["k_pages"].shape[0]
    table, starts, lens = (d[n].tolist() for n in ("table", "starts", "lens"))
    k, v = (d[t + "_pages"].to(torch.float64) * d[t + "_scale"].double()[..., None, None] for t in "kv")
    q = d["q"].double()
    o, err = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    inside = torch.zeros(q.shape[0], dtype=torch.bool, device=q.device)
    for s in range(len(lens)):
        a, b = starts[s], starts[s + 1]
        if a == b:
            continue
        inside[a:b] = True
        m = min(max(lens[s], 0), len(table[s]) * c.page)
        pos = torch.arange(m, device=q.device)
        pages = torch.tensor(table[s], device=q.device)[pos // c.page]
        good = (pages >= 0) & (pages < n_pages)
        pos, pages = pos[good], pages[good]
        if not len(pos):
            continue
        kk, vv = (x[pages, :, pos % c.page].repeat_interleave(c.G, 1) for x in (k, v))  # [keys, Hq, D]
        vs = d["v_scale"].double()[pages].repeat_interleave(c.G, 1)  # [keys, Hq]
        z = torch.einsum("ihd,jhd->hij", q[a:b], kk) * scale
        limit = lens[s] - (b - a) + torch.arange(b - a, device=q.device) + 1
        ok = pos[None] < limit[:, None]
        z = z.masked_fill(~ok, -math.inf)
        some = ok.any(1)
        lse[a:b] = torch.where(some[:, None], z.logsumexp(-1).T, -math.inf)
        p = torch.where(ok, z - z.amax(-1, keepdim=True).clamp(min=-1e300), -math.inf).exp()
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
        o[a:b] = torch.einsum("hij,jhd->ihd", p, vv)
        err[a:b] = torch.einsum("hij,jhd->ihd", p, vv.abs()) * (2.0 ** -11 + 2.0 ** -13) + \
            2.0 ** -25 * (p * vs.T[:, None]).amax(-1).T[..., None] * \
            torch.einsum("ij,jhd->ihd", ok.double(), vv.abs() / vs[..., None])
    return o, lse, err * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs() + 1e-30, inside


def check_cached(c, d, o, lse, scale=None, what="o"):
    want, wl, err, inside = cached_reference(c, d, scale)
    check_rows(o[inside], want[inside], err[inside], what)
    assert (o[~inside] == 7.0).all(), what + ": a row of no sequence was written"
    if lse is not None:
        none = wl == -math.inf
        assert torch.equal((lse == -math.inf) & inside[:, None], none & inside[:, None])
        assert (o[(none & inside[:, None])] == 0).all()
        ok = ~none & inside[:, None]
        check_rows(lse[ok], wl[ok], 2.0 ** -13 + 2.0 ** -22 * wl[ok].abs(), "lse")
        assert (lse[~inside] == 7.0).all(), "lse: a row of no sequence was written"
    return want


def attend(cache, c, d, **kw):
    o = torch.full_like(d["q"], 7.0) if d["q"].is_contiguous() else torch.full(d["q"].shape, 7.0, dtype=torch.bfloat16,
                                                                              device=d["q"].device)
    lse = torch.full(d["q"].shape[:2], 7.0, device=o.device)
    cache.attention(d["q"], o, d["starts"], d["lens"], d["table"], lse=lse, **kw)
    return o, lse
