"""The attention, and the norm and rotation of q and k heads, of P shards in 64
bits with torch operations that autograd differentiates: what the gradient
tests compare the kernels with.  Written from the definitions in
include/uly.h; shares no code with the library."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch


@dataclass(frozen=True)
class Case:
    name: str
    B: int
    lens: tuple
    R: int
    mode: str
    Hq: int
    Hkv: int
    D: int
    rows: str = "sdpa"
    mask: str = "all"  # all, ranges, random, none (no admitted key), tail (a few keys of the last tile)
    std: float = 1.0

    @property
    def P(self):
        return len(self.lens)

    @property
    def n(self):
        return sum(self.lens)

    @property
    def rep_q(self):
        return self.R if self.mode in ("prefix", "suffix") else 0

    @property
    def nk(self):
        return self.n + self.R

    @property
    def nq(self):
        return self.n + self.rep_q


def plan_of(c, dtype="bf16"):
    from ulysses_sequence_attention_uly_gb300 import Plan
    return Plan(c.B, c.P, c.lens[0], c.R, c.mode, c.Hq, c.Hkv, c.D, dtype=dtype, masked_rows=c.rows,
                shard_lens=c.lens if len(set(c.lens)) > 1 else None)


def key_mask(c, g, dev):
    nk = c.nk
    if c.mask == "all":
        return None
    if c.mask == "none":
        return torch.zeros((c.B, nk), dtype=torch.bool, device=dev)
    if c.mask == "random":
        return torch.rand((c.B, nk), generator=g, device=dev) < 0.6
    m = torch.zeros((c.B, nk), dtype=torch.bool, device=dev)
    if c.mask == "tail":
        m[:, -min(3, nk):] = True
        return m
    for b in range(c.B):  # ranges: two of them, other ones for each batch
        m[b, nk // 7 + b:nk // 2] = True
        m[b, nk // 2 + nk // 5 + b:nk - nk // 9] = True
    return m


def shard_rows(c, p, is_kv):
    return c.lens[p] + (c.R if is_kv else c.rep_q)


def _bf16(g, shape, dev, std=1.0):
    return (torch.randn(shape, generator=g, device=dev) * std).to(torch.bfloat16)


def inputs(c, seed, dev="cuda"):
    """q, k, v shards and one output gradient per shard; every shard's copy of
    the replicated rows has values of its own."""
    g = torch.Generator(device=dev).manual_seed(seed)
    d = {"q": [_bf16(g, (c.B, shard_rows(c, p, False), c.Hq, c.D), dev, c.std) for p in range(c.P)],
         "k": [_bf16(g, (c.B, shard_rows(c, p, True), c.Hkv, c.D), dev, c.std) for p in range(c.P)],
         "v": [_bf16(g, (c.B, shard_rows(c, p, True), c.Hkv, c.D), dev, c.std) for p in range(c.P)],
         "do": [_bf16(g, (c.B, shard_rows(c, p, False), c.Hq, c.D), dev) for p in range(c.P)]}
    d["mask"] = key_mask(c, g, dev)
    return d


def _parts(c, x, p, R):
    """(replicated rows, image rows) of shard p's tensor."""
    return (x[:, c.lens[p]:], x[:, :c.lens[p]]) if c.mode == "suffix" else (x[:, :R], x[:, R:])


def to_global(c, shards, is_kv):
    """[B, N, H, ...] in the global row order; replicated rows of a head from its owner's shard."""
    R = c.R if is_kv else c.rep_q
    parts = [_parts(c, x, p, R) for p, x in enumerate(shards)]
    img = torch.cat([i for _, i in parts], 1)
    per = shards[0].shape[2] // c.P
    rep = torch.cat([r[:, :, p * per:(p + 1) * per] for p, (r, _) in enumerate(parts)], 2)
    return torch.cat([img, rep] if c.mode == "suffix" else [rep, img], 1)


def to_shards(c, x, is_kv):
    """Global rows to the shards; replicated rows to every one of them."""
    R = c.R if is_kv else c.rep_q
    n = c.n
    rep, img = (x[:, n:], x[:, :n]) if c.mode == "suffix" else (x[:, :R], x[:, R:])
    out = []
    for i in img.split(list(c.lens), 1):
        out.append(torch.cat([i, rep] if c.mode == "suffix" else [rep, i], 1))
    return out


def admitted(c, mask, dev):
    """[B, Nq, Nk] pairs that attend."""
    m = torch.ones((c.B, c.nk), dtype=torch.bool, device=dev) if mask is None else mask
    own = m[:, c.R:] if c.mode == "kv_prefix" else m
    a = m[:, None, :].expand(c.B, c.nq, c.nk)
    if c.rows == "zero":
        a = a & own[:, :, None]
    elif c.rows == "self":
        a = m[:, None, :] == own[:, :, None]
    return a


def attention(c, q, k, v, mask, scale):
    """Output and log-sum-exp of global 64-bit tensors (autograd through them)."""
    G = c.Hq // c.Hkv
    a = admitted(c, mask, q.device)[:, None]  # [B, 1, Nq, Nk]
    s = torch.einsum("bnhd,bmhd->bhnm", q, k.repeat_interleave(G, 2)) * scale
    s = torch.where(a, s, -math.inf)
    top = s.detach().amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.where(a, torch.exp(torch.where(a, s - top, 0.0)), 0.0)
    z = e.sum(-1, keepdim=True)
    p = e / torch.where(z == 0, 1.0, z)
    o = torch.einsum("bhnm,bmhd->bnhd", p, v.repeat_interleave(G, 2))
    lse = torch.where(z == 0, -math.inf, torch.log(torch.where(z == 0, 1.0, z)) + top)[..., 0].transpose(1, 2)
    return o, lse, p


def reference(c, d, scale=None):
    """Everything a test compares with: the forward's o (bf16) and lse (f32)
    as shards and rank tensors, and gradients with their error bounds for both
    layouts.

    The bounds count roundings of at most half a step, u = 2^-8 for bf16:
    dv = sum P do with P rounded (u each); dS = P (dP - delta) rounded, with o
    in delta rounded by the forward; dq and dk are sums of dS k and dS q; and
    the output.  r64 stands for the 32-bit arithmetic: sums of up to 2^14 terms
    (2^-24 each, added pairwise or in order by the MMA in chunks of 16) and the
    exponential's argument, |s| up to about 60: together below 2^-13.  Fused,
    replicated rows: the sum of the shards' do enters as two bf16 parts, off by
    u^2."""
    scale = 1.0 / math.sqrt(c.D) if scale is None else scale
    u, r = 2.0 ** -8, 2.0 ** -13
    shards = [[x.double().requires_grad_() for x in d[n]] for n in "qkv"]
    q, k, v = (to_global(c, x, i) for x, i in zip(shards, (False, True, True)))
    o, lse, p = attention(c, q, k, v, d["mask"], scale)
    os = to_shards(c, o, False)
    do = [x.double() for x in d["do"]]
    g = torch.autograd.grad(os, shards[0] + shards[1] + shards[2], do)
    P = c.P
    ref = {"dq": g[:P], "dk": g[P:2 * P], "dv": g[2 * P:], "o": [x.detach().to(torch.bfloat16) for x in os],
           "lse": [x.float() for x in to_shards(c, lse.detach(), False)], "scale": scale}
    with torch.no_grad():
        # global gradient of o: replicated rows of every shard added up
        tot = torch.zeros_like(o)
        rep_u = torch.zeros((1, c.nq, 1, 1), dtype=torch.float64, device=o.device)
        img_at = c.rep_q if c.mode != "suffix" else 0
        at = img_at
        for i, x in enumerate(do):
            rr, im = _parts(c, x, i, c.rep_q)
            tot[:, at:at + c.lens[i]] = im
            at += c.lens[i]
            if c.rep_q:
                sl = slice(c.n, None) if c.mode == "suffix" else slice(0, c.rep_q)
                tot[:, sl] += rr
                rep_u[:, sl] = u * u
        G = c.Hq // c.Hkv
        kk, vv = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
        tr = tot.abs() * (1 + 0 * rep_u)
        dp = torch.einsum("bnhd,bmhd->bhnm", tot, vv)
        delta = (o * tot).sum(-1).transpose(1, 2)[..., None]
        ds = p * (dp - delta)
        mag_v = torch.einsum("bnhd,bmhd->bhnm", tr, vv.abs())
        mag_o = (o.abs() * tr).sum(-1).transpose(1, 2)[..., None]
        ru = rep_u[:, :, 0, 0][:, None, :, None]
        e_ds = (u + r) * ds.abs() + p * ((ru + r) * mag_v + (u + ru + r) * mag_o)
        e_p = (u + r) * p
        fold = lambda x: x.view(c.B, c.nk, c.Hkv, G, c.D).sum(3)  # noqa: E731
        e_dq = scale * torch.einsum("bhnm,bmhd->bnhd", e_ds, kk.abs())
        e_dk = fold(scale * torch.einsum("bhnm,bnhd->bmhd", e_ds, q.abs()))
        e_dv = fold(torch.einsum("bhnm,bnhd->bmhd", e_p, tr) + torch.einsum("bhnm,bnhd->bmhd", p, tr * rep_u))
        # gradients and statistics of the head-sharded layout, where do is given per gathered row
        ref["h"] = {"o": o.detach().to(torch.bfloat16), "lse": lse.detach().float(), "do": tot.to(torch.bfloat16)}
        for n, e, is_kv in (("dq", e_dq, False), ("dk", e_dk, True), ("dv", e_dv, True)):
            ref["e_" + n] = [(1 + u) * (x + r) for x in to_shards(c, e, is_kv)]
            ref["e_" + n] = [x + u * y.abs() + 1e-6 for x, y in zip(ref["e_" + n], ref[n])]
    return ref


def check(got, want, bound, what):
    """Every element within its bound, and the whole within 2^-7 in the 2-norm:
    the output's rounding is at most 2^-8 of it, and the operands' roundings,
    independent of each other, add up to no more in the norm."""
    for i, (x, y, e) in enumerate(zip(got, want, bound)):
        x = x.double()
        assert torch.isfinite(x).all(), "%s[%d]: not finite or not written" % (what, i)
        bad = (x - y).abs() > e
        assert not bad.any(), "%s[%d]: %d elements, worst %.3g over its bound at %s" % (
            what, i, int(bad.sum()), float(((x - y).abs() / e).max()), bad.nonzero()[0].tolist())
    num = math.sqrt(sum(float((x.double() - y).square().sum()) for x, y in zip(got, want)))
    den = math.sqrt(sum(float(y.square().sum()) for y in want))
    slack = math.sqrt(sum(float(e.square().sum()) for e in bound))
    assert num <= 2.0 ** -7 * den + 1e-3 * slack, "%s: off by %.3g of its norm" % (what, num / max(den, 1e-300))


# ---------------------------------------------------- norm and rotation --
def table_rows(c, p, is_kv):
    """Table row of each row of shard p's tensor (global key order)."""
    a = sum(c.lens[:p])
    R = c.R if is_kv else c.rep_q
    if c.mode == "suffix":
        return torch.cat([torch.arange(a, a + c.lens[p]), torch.arange(c.n, c.n + R)])
    return torch.cat([torch.arange(R), torch.arange(c.R + a, c.R + a + c.lens[p])])


def norm_rope(c, x, w, cos, sin, p, is_kv, pairs, eps):
    """64-bit norm and rotation of shard p's tensor by complex products."""
    D = c.D
    y = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    if w is not None:
        y = y * w
    if cos is None:
        return y
    rows = table_rows(c, p, is_kv).to(x.device)
    turn = torch.complex(cos.double(), sin.double())[..., rows, :].unsqueeze(-2)
    if pairs == "interleaved":
        z = torch.complex(y[..., 0::2], y[..., 1::2]) * turn
        return torch.stack((z.real, z.imag), -1).flatten(-2)
    z = torch.complex(y[..., :D // 2], y[..., D // 2:]) * turn
    return torch.cat((z.real, z.imag), -1)
