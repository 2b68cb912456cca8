"""Norm and rotation of q and k heads and its gradient on the GPU
(uly_norm_rope, uly_norm_rope_backward) against 64-bit complex arithmetic and
autograd, and the training step around the attention that they belong to."""
import math

import pytest

from tests import _grad as R

pytestmark = pytest.mark.gpu

# (case, pairs, packed, table batches, weights, tables)
CASES = [
    (R.Case("token", 8, (1,), 0, "none", 40, 8, 128), "half", False, 1, True, True),
    (R.Case("one-head", 1, (1,), 0, "none", 1, 1, 64), "interleaved", False, 1, True, True),
    (R.Case("prefix", 2, (37, 37), 11, "prefix", 6, 2, 128), "interleaved", False, 1, True, True),
    (R.Case("suffix-uneven", 2, (5, 61, 1), 9, "suffix", 6, 3, 64), "half", False, 2, True, True),
    (R.Case("kv-prefix", 1, (33, 20), 7, "kv_prefix", 10, 2, 128), "half", False, 1, True, True),
    (R.Case("packed", 3, (29, 12), 0, "none", 6, 2, 64), "interleaved", True, 3, True, True),
    (R.Case("packed-rep", 1, (19, 19), 4, "prefix", 4, 4, 128), "half", True, 1, False, True),
    (R.Case("no-tables", 1, (50,), 0, "none", 5, 5, 128), "interleaved", False, 1, True, False),
    (R.Case("many-rows", 1, (6000, 1), 3, "suffix", 2, 2, 64), "interleaved", False, 1, True, True),
    (R.Case("odd-heads", 1, (70,), 0, "none", 33, 11, 128), "half", False, 1, False, True),
]
ids = lambda x: x[0].name  # noqa: E731
EPS = 1e-6


def make(case, seed=1, std=1.0):
    import torch
    c, pairs, packed, tb, weights, tables = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = [(R.shard_rows(c, p, False), R.shard_rows(c, p, True)) for p in range(c.P)]
    rnd = lambda *s: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    if packed:
        qkv = [rnd(c.B, a, c.Hq + 2 * c.Hkv, c.D) for a, _ in rows]
        q, k = [x[:, :, :c.Hq] for x in qkv], [x[:, :, c.Hq:c.Hq + c.Hkv] for x in qkv]
    else:
        q, k = [rnd(c.B, a, c.Hq, c.D) for a, _ in rows], [rnd(c.B, b, c.Hkv, c.D) for _, b in rows]
    d = {"q": q, "k": k, "pairs": pairs}
    d["gq"], d["gk"] = [rnd(*x.shape) for x in q], [rnd(*x.shape) for x in k]
    d["wq"], d["wk"] = ((1 + 0.3 * torch.randn(c.D, generator=g, device="cuda")) if weights else None for _ in "qk")
    d["cos"] = d["sin"] = None
    if tables:
        shape = (tb, c.nk, c.D // 2) if tb > 1 else (c.nk, c.D // 2)
        ang = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64) * 50 - 25
        d["cos"], d["sin"] = ang.cos().float(), ang.sin().float()
    return d


def dense(ts, fill=float("nan")):
    import torch
    return [torch.full(tuple(t.shape), fill, dtype=torch.bfloat16, device="cuda") for t in ts]


def reference(c, d, t, p, grad):
    """64-bit value (or gradients) of shard p's tensor and elementwise bounds:
    u = 2^-8 for the one rounding to bf16, r = 2^-17 of the terms' magnitudes
    for the 32-bit arithmetic (a sum of 128 squares, a reciprocal root, five
    products)."""
    import torch
    u, r = 2.0 ** -8, 2.0 ** -17
    is_kv = t == "k"
    x = d[t][p].double().requires_grad_()
    w = None if d["w" + t] is None else d["w" + t].double().requires_grad_()
    y = R.norm_rope(c, x, w, d["cos"], d["sin"], p, is_kv, d["pairs"], EPS)
    with torch.no_grad():
        z = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        n = z if w is None else z * w
        # |cos|, |sin| <= 1: a pair's terms are at most its two magnitudes
        a, b = (n[..., 0::2], n[..., 1::2]) if d["pairs"] == "interleaved" else n.chunk(2, -1)
        m = a.abs() + b.abs()
        m = torch.stack((m, m), -1).flatten(-2) if d["pairs"] == "interleaved" else torch.cat((m, m), -1)
    if not grad:
        return y.detach(), u * y.detach().abs() * (1 + u) + r * m + 1e-30
    g = d["g" + t][p].double()
    gx, = torch.autograd.grad(y, x, g, retain_graph=True)
    with torch.no_grad():
        a, b = (g[..., 0::2], g[..., 1::2]) if d["pairs"] == "interleaved" else g.chunk(2, -1)
        m = a.abs() + b.abs()
        dn = torch.stack((m, m), -1).flatten(-2) if d["pairs"] == "interleaved" else torch.cat((m, m), -1)
        ww = 1.0 if w is None else w.abs()
        rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        e = r * rstd * (dn * ww + z.abs() * (dn * ww * z.abs()).mean(-1, keepdim=True))
        e_w = r * (dn * z.abs()).sum((0, 1, 2))
    gw = torch.zeros(c.D, dtype=torch.float64, device="cuda") if w is None else torch.autograd.grad(y, w, g)[0]
    return gx, u * gx.abs() * (1 + u) + e + 1e-30, gw, e_w


def within(got, want, bound, what):
    import torch
    assert torch.isfinite(got.double()).all(), what + ": not finite or not written"
    err = (got.double() - want).abs()
    assert (err <= bound).all(), "%s: worst %.3g over its bound" % (what, float((err / bound).max()))


def run(plan, d, **kw):
    qo, ko = dense(d["q"]), dense(d["k"])
    plan.norm_rope(d["q"], d["k"], qo, ko, d["wq"], d["wk"], d["cos"], d["sin"], pairs=d["pairs"], eps=EPS, **kw)
    return qo, ko


def run_backward(plan, d, **kw):
    import torch
    dq, dk = dense(d["q"]), dense(d["k"])
    dw = [torch.full((d["q"][0].shape[-1],), float("nan"), device="cuda") for _ in "qk"]
    plan.norm_rope_backward(d["q"], d["k"], d["gq"], d["gk"], dq, dk, d["wq"], d["wk"], d["cos"], d["sin"], *dw,
                            pairs=d["pairs"], eps=EPS, **kw)
    return dq, dk, dw


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case):
    c, d = case[0], make(case)
    qo, ko = run(R.plan_of(c), d)
    for t, out in (("q", qo), ("k", ko)):
        for p in range(c.P):
            within(out[p], *reference(c, d, t, p, False), "%s[%d]" % (t, p))


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case):
    c, d = case[0], make(case, 2)
    dq, dk, dw = run_backward(R.plan_of(c), d)
    for t, out, w in (("q", dq, dw[0]), ("k", dk, dw[1])):
        total = bound = 0
        for p in range(c.P):
            gx, e, gw, e_w = reference(c, d, t, p, True)
            within(out[p], gx, e, "d%s[%d]" % (t, p))
            total, bound = total + gw, bound + e_w
        if d["w" + t] is not None:
            within(w, total, bound, "dw" + t)


@pytest.mark.parametrize("std", [1e-6, 1e-3, 100.0])
def test_small_and_large_values(std):
    case = CASES[2]
    c, d = case[0], make(case, 3, std)
    qo, ko = run(R.plan_of(c), d)
    dq, dk, _ = run_backward(R.plan_of(c), d)
    for t, out, grad in (("q", qo, dq), ("k", ko, dk)):
        for p in range(c.P):
            within(out[p], *reference(c, d, t, p, False), t)
            within(grad[p], *reference(c, d, t, p, True)[:2], "d" + t)


def test_zero_head():
    """A head of zeros: zeros out, and a finite gradient."""
    case = CASES[2]
    c, d = case[0], make(case, 4)
    d["q"][0][0, 0, 0] = 0
    qo, _ = run(R.plan_of(c), d)
    assert (qo[0][0, 0, 0] == 0).all()
    dq, _, _ = run_backward(R.plan_of(c), d)
    within(dq[0], *reference(c, d, "q", 0, True)[:2], "dq")


def test_against_differences():
    """<gradient, direction> against the 64-bit difference quotient."""
    import torch
    case = CASES[2]
    c, d = case[0], make(case, 5)
    dq, dk, dw = run_backward(R.plan_of(c), d)
    gen = torch.Generator(device="cuda").manual_seed(6)
    for t, gx, gw in (("q", dq, dw[0]), ("k", dk, dw[1])):
        dirs = [torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64) for x in gx]
        dirw = torch.randn(c.D, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        loss = lambda s: sum(float((R.norm_rope(c, d[t][p].double() + s * dirs[p], d["w" + t].double() + s * dirw,  # noqa: E731
                                                d["cos"], d["sin"], p, t == "k", d["pairs"], EPS)
                                    * d["g" + t][p].double()).sum()) for p in range(c.P))
        want = (loss(h) - loss(-h)) / (2 * h)
        got = sum(float((x.double() * y).sum()) for x, y in zip(gx, dirs)) + float((gw.double() * dirw).sum())
        norm = math.sqrt(sum(float(x.double().square().sum()) for x in gx))
        assert abs(got - want) <= 5 * 2.0 ** -8 * norm + 1e-6 * abs(want), (t, got, want)


def test_in_place_and_one_tensor():
    """Outputs over dense inputs, gradients over the output's, q alone and k
    alone: the same bits."""
    import torch
    case = CASES[3]
    c, d = case[0], make(case, 7)
    plan = R.plan_of(c)
    qo, ko = run(plan, d)
    dq, dk, dw = run_backward(plan, d)
    q2, k2 = [x.clone() for x in d["q"]], [x.clone() for x in d["k"]]
    plan.norm_rope(q2, k2, q2, k2, d["wq"], d["wk"], d["cos"], d["sin"], pairs=d["pairs"], eps=EPS)
    only = dense(d["k"])
    plan.norm_rope(None, d["k"], None, only, None, d["wk"], d["cos"], d["sin"], pairs=d["pairs"], eps=EPS)
    for a, b in zip(qo + ko + ko, q2 + k2 + only):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    g2 = [x.clone() for x in d["gq"]]
    w2 = torch.empty(c.D, device="cuda")
    plan.norm_rope_backward(d["q"], None, g2, None, g2, None, d["wq"], None, d["cos"], d["sin"], w2, None,
                            pairs=d["pairs"], eps=EPS)
    for a, b in zip(dq, g2):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # (q alone has other CTAs, so another order of the sum)
    torch.testing.assert_close(w2, dw[0], rtol=1e-4, atol=1e-3)


def test_same_bits_streams_and_graph():
    """The weights' gradient has the same bits on every call, on another stream,
    in a graph and with any workspace."""
    import torch
    case = CASES[8]
    c, d = case[0], make(case, 8)
    plan = R.plan_of(c)
    want = run_backward(plan, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = run_backward(plan, d, stream=s)
    s.synchronize()
    n = plan.norm_rope_backward_workspace()
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    dq, dk = dense(d["q"]), dense(d["k"])
    dw = [torch.empty(c.D, device="cuda") for _ in "qk"]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan.norm_rope_backward(d["q"], d["k"], d["gq"], d["gk"], dq, dk, d["wq"], d["wk"], d["cos"], d["sin"], *dw,
                                pairs=d["pairs"], eps=EPS, workspace=ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got in (other, (dq, dk, dw)):
        for a, b in zip(want, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_writes_nothing_else():
    import torch
    case = CASES[5]
    c, d = case[0], make(case, 9)
    plan = R.plan_of(c)
    want, _ = run(plan, d)
    bufs = [torch.full((x.numel() + 1024,), 7.0, dtype=torch.bfloat16, device="cuda") for x in d["q"]]
    out = [b[512:512 + x.numel()].view(x.shape) for b, x in zip(bufs, d["q"])]
    plan.norm_rope(d["q"], None, out, None, d["wq"], None, d["cos"], d["sin"], pairs=d["pairs"], eps=EPS)
    for b, x, y in zip(bufs, out, want):
        assert torch.equal(x, y)
        assert (b[:512] == 7).all() and (b[512 + x.numel():] == 7).all()


def test_offsets_past_32_bits():
    """A q shard of more than 2^31 elements: its last rows have the bits of a
    call of their own."""
    import torch
    from ulysses_sequence_attention_uly_gb300 import Plan
    H, D, n = 64, 128, 5
    B = 2 ** 31 // (n * H * D) + 2
    g = torch.Generator(device="cuda").manual_seed(1)
    ang = torch.rand((n, D // 2), generator=g, device="cuda") * 6
    small = [torch.randn((1, n, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    x, gr = (torch.zeros((B, n, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[B - 1], gr[B - 1] = small[0][0], small[1][0]
    out, dx = torch.empty_like(x), torch.empty_like(x)
    for plan, a, b, y, dy in ((Plan(B, 1, n, 0, "none", H, H, D), x, gr, out, dx),
                              (Plan(1, 1, n, 0, "none", H, H, D), small[0], small[1], torch.empty_like(small[0]),
                               torch.empty_like(small[0]))):
        plan.norm_rope([a], None, [y], None, None, None, ang.cos(), ang.sin())
        plan.norm_rope_backward([a], None, [b], None, [dy], None, None, None, ang.cos(), ang.sin())
    for big, one in ((out, y), (dx, dy)):
        assert torch.equal(big[B - 1], one[0])
        assert (big[0] == 0).all()


def test_refusals():
    import torch
    import ulysses_sequence_attention_uly_gb300 as uly
    case = CASES[2]
    c, d = case[0], make(case, 10)
    plan = R.plan_of(c)
    qo, ko = dense(d["q"]), dense(d["k"])
    base = dict(q=d["q"], k=d["k"], q_out=qo, k_out=ko, q_weight=d["wq"], k_weight=d["wk"], cos=d["cos"], sin=d["sin"])

    def refuse(exc, status=None, **kw):
        with pytest.raises(exc) as e:
            plan.norm_rope(**{**base, **kw})
        if status is not None:
            assert e.value.status == status

    refuse(ValueError, q=d["q"][:1])
    refuse(ValueError, q=[x.float() for x in d["q"]])
    refuse(ValueError, q=[x.transpose(2, 3).contiguous().transpose(2, 3) for x in d["q"]])
    refuse(ValueError, q=[torch.empty(x.shape[:3] + (c.D + 4,), dtype=torch.bfloat16, device="cuda")[..., :c.D]
                          for x in d["q"]])
    refuse(ValueError, q_out=None)
    refuse(ValueError, cos=None)
    refuse(ValueError, cos=d["cos"][1:])
    refuse(ValueError, sin=d["sin"].double())
    refuse(ValueError, q_weight=d["wq"][1:])
    refuse(ValueError, q_weight=d["wq"].to(torch.bfloat16))
    refuse(ValueError, pairs="neox")
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, eps=0.0)
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, eps=float("nan"))
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, q=None, k=None, q_out=None, k_out=None)
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, q_out=[qo[0], qo[0]])
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, q_out=[d["q"][1], d["q"][0]])
    with pytest.raises(ValueError):
        plan.norm_rope_backward(d["q"], d["k"], d["gq"], d["gk"], qo, ko, workspace=torch.empty(8, device="cuda"))
    p8 = R.plan_of(R.Case("e4m3", 1, (64,), 0, "none", 1, 1, 128), dtype="e4m3")
    x = [torch.zeros((1, 64, 1, 128), dtype=torch.bfloat16, device="cuda")]
    with pytest.raises(uly.UlyError) as e:
        p8.norm_rope(x, None, [torch.empty_like(x[0])], None)
    assert e.value.status == uly.ULY_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert all(torch.isnan(t).all() for t in qo + ko)


@pytest.mark.parametrize("c", [R.Case("prefix", 2, (150, 131), 40, "prefix", 4, 2, 128, mask="ranges"),
                               R.Case("kv-prefix", 1, (140, 140), 12, "kv_prefix", 4, 4, 64, rows="zero",
                                      mask="ranges")], ids=lambda c: c.name)
def test_training_step(c):
    """norm_rope -> sp_attention (with its log-sum-exp) -> sp_attention_backward
    -> norm_rope_backward, as one layer's training step, against 64-bit autograd
    of the whole chain.  Each of the step's intermediate tensors is rounded to
    bf16 (q, k, o, their gradients): six independent roundings of at most 2^-8
    on the way, so the gradients agree to 6 * 2^-8 in the norm."""
    import torch
    case = (c, "interleaved", False, 1, True, True)
    d = make(case, 20)
    plan = R.plan_of(c)
    att = R.inputs(c, 21)
    v, do, mask = att["v"], att["do"], att["mask"]
    qo, ko = run(plan, d)
    o = dense(d["q"])
    lse = [torch.empty(x.shape[:3], device="cuda") for x in d["q"]]
    plan.sp_attention(qo, ko, v, o, key_mask=mask, lse=lse)
    dqo, dko, dv = dense(d["q"]), dense(d["k"]), dense(d["k"])
    plan.sp_attention_backward(qo, ko, v, o, lse, do, dqo, dko, dv, key_mask=mask)
    d["gq"], d["gk"] = dqo, dko
    dq, dk, dw = run_backward(plan, d)
    assert plan.sync_status() == 0
    x = {n: [t.double().requires_grad_() for t in (d[n] if n != "v" else v)] for n in "qkv"}
    w = {n: d["w" + n].double().requires_grad_() for n in "qk"}
    n = {t: [R.norm_rope(c, x[t][p], w[t], d["cos"], d["sin"], p, t == "k", "interleaved", EPS) for p in range(c.P)]
         for t in "qk"}
    out, _, _ = R.attention(c, R.to_global(c, n["q"], False), R.to_global(c, n["k"], True),
                            R.to_global(c, x["v"], True), mask, 1 / math.sqrt(c.D))
    want = torch.autograd.grad(R.to_shards(c, out, False), x["q"] + x["k"] + x["v"] + [w["q"], w["k"]],
                               [t.double() for t in do])
    got = dq + dk + dv + dw
    for i in range(0, 3 * c.P, c.P):
        num = sum(float((a.double() - b).square().sum()) for a, b in zip(got[i:i + c.P], want[i:i + c.P]))
        den = sum(float(b.square().sum()) for b in want[i:i + c.P])
        assert math.sqrt(num / den) <= 6 * 2.0 ** -8, (i, math.sqrt(num / den))
    for a, b in zip(got[3 * c.P:], want[3 * c.P:]):
        assert float((a.double() - b).norm() / b.norm()) <= 6 * 2.0 ** -8


# rows enough for a warp to take a whole row: several turns of its loop over the heads, the last one partly filled
WHOLE_ROWS = [
    (R.Case("33-11-heads", 2, (1300,), 0, "none", 33, 11, 128), "interleaved", False, 2, True, True),
    (R.Case("18-6-heads-half", 1, (1400, 1300), 33, "suffix", 18, 6, 128), "half", False, 1, True, True),
    (R.Case("9-3-heads", 1, (2500,), 7, "kv_prefix", 9, 3, 128), "half", False, 1, True, True),
    (R.Case("21-7-heads-64", 1, (2600,), 0, "none", 21, 7, 64), "interleaved", False, 1, True, True),
    (R.Case("39-13-heads-64-packed", 3, (900,), 0, "none", 39, 13, 64), "half", True, 3, True, True),
    (R.Case("20-20-heads-64", 1, (1200, 1301), 50, "prefix", 20, 20, 64), "interleaved", False, 1, True, True),
]


@pytest.mark.parametrize("case", WHOLE_ROWS, ids=ids)
def test_whole_rows(case):
    """Outputs, gradients and the weights' gradients where tasks are whole rows;
    in place, the same bits."""
    import torch
    c, d = case[0], make(case, 11)
    plan = R.plan_of(c)
    rows = c.B * sum(R.shard_rows(c, p, kv) for p in range(c.P) for kv in (False, True))
    assert rows >= 32 * torch.cuda.get_device_properties(0).multi_processor_count
    qo, ko = run(plan, d)
    dq, dk, dw = run_backward(plan, d)
    for t, out, grad, w in (("q", qo, dq, dw[0]), ("k", ko, dk, dw[1])):
        total = bound = 0
        for p in range(c.P):
            within(out[p], *reference(c, d, t, p, False), "%s[%d]" % (t, p))
            gx, e, gw, e_w = reference(c, d, t, p, True)
            within(grad[p], gx, e, "d%s[%d]" % (t, p))
            total, bound = total + gw, bound + e_w
        within(w, total, bound, "dw" + t)
    x2, g2 = ({t: [x.clone() for x in d[n + t]] for t in "qk"} for n in ("", "g"))
    x2 = {t: [x.contiguous() for x in x2[t]] for t in "qk"}
    w2 = [torch.empty(c.D, device="cuda") for _ in "qk"]
    plan.norm_rope_backward(x2["q"], x2["k"], g2["q"], g2["k"], g2["q"], g2["k"], d["wq"], d["wk"], d["cos"], d["sin"],
                            *w2, pairs=d["pairs"], eps=EPS)
    plan.norm_rope(x2["q"], x2["k"], x2["q"], x2["k"], d["wq"], d["wk"], d["cos"], d["sin"], pairs=d["pairs"], eps=EPS)
    for a, b in zip(dq + dk + dw + qo + ko, g2["q"] + g2["k"] + w2 + x2["q"] + x2["k"]):
        assert torch.equal(a, b)
