"""The gradient of the attention on the GPU (uly_attention_backward,
uly_sp_attention_backward) against 64-bit autograd of the whole call as a
function of the shards, against differences of it, and where masks, short and
uneven shards, replicated rows, streams and graphs can make it go wrong."""
import math

import pytest

from tests import _grad as R

pytestmark = pytest.mark.gpu

CASES = [
    R.Case("plain", 1, (256,), 0, "none", 2, 2, 128),
    R.Case("plain-d64", 2, (128, 128), 0, "none", 2, 2, 64),
    R.Case("one-row", 1, (1,), 0, "none", 1, 1, 128),
    R.Case("two-rows", 2, (1, 1), 0, "none", 4, 2, 64),
    R.Case("tile-edges", 1, (127, 129), 0, "none", 2, 2, 128),
    R.Case("long", 1, (1300,), 0, "none", 1, 1, 128, mask="ranges"),
    R.Case("prefix", 2, (300, 300), 200, "prefix", 4, 2, 128, mask="ranges"),
    R.Case("prefix-tiny", 1, (56, 56), 16, "prefix", 4, 4, 64, mask="ranges"),
    R.Case("suffix-uneven", 1, (45, 257, 130), 33, "suffix", 6, 3, 128, mask="random"),
    R.Case("suffix-zero", 2, (300, 77), 140, "suffix", 4, 2, 64, rows="zero", mask="ranges"),
    R.Case("prefix-zero", 1, (200, 200), 129, "prefix", 4, 4, 128, rows="zero", mask="random"),
    R.Case("kv-prefix", 2, (256, 100), 70, "kv_prefix", 8, 2, 128, mask="ranges"),
    R.Case("kv-prefix-self", 1, (150, 150), 30, "kv_prefix", 4, 2, 64, rows="self", mask="random"),
    R.Case("self", 2, (260, 131), 64, "suffix", 4, 2, 128, rows="self", mask="ranges"),
    R.Case("self-none", 1, (130, 130), 0, "none", 2, 2, 128, rows="self", mask="none"),
    R.Case("self-all", 1, (130, 130), 0, "none", 2, 2, 128, rows="self"),
    R.Case("no-key", 2, (140, 20), 5, "prefix", 2, 2, 128, mask="none"),
    R.Case("no-key-zero", 1, (140,), 0, "none", 2, 2, 64, rows="zero", mask="none"),
    R.Case("three-keys", 1, (700,), 0, "none", 4, 1, 128, mask="tail"),
    R.Case("ranks16", 1, (20,) * 16, 7, "prefix", 16, 16, 128, mask="ranges"),
    R.Case("gqa8", 1, (400,), 0, "none", 8, 1, 64),
    R.Case("large-scores", 1, (300,), 0, "none", 2, 2, 128, std=2.5),
]
ids = lambda c: c.name  # noqa: E731


def mask_args(c, mask, form):
    import torch
    if mask is None:
        return {}
    if form == "mask":
        return {"key_mask": mask}
    # the mask's runs as ranges, padded with empty ones
    runs = []
    for b in range(c.B):
        m = [0] + mask[b].int().tolist() + [0]
        at = [i for i in range(1, len(m)) if m[i] != m[i - 1]]
        runs.append([(a - 1, e - 1) for a, e in zip(at[::2], at[1::2])])
    n = max(1, max(len(r) for r in runs))
    t = torch.tensor([r + [(0, 0)] * (n - len(r)) for r in runs], dtype=torch.int32, device=mask.device)
    return {"key_ranges": t}


def outputs(ts, fill=float("nan")):
    import torch
    return [torch.full_like(t, fill) for t in ts]


def run_fused(c, plan, d, ref, form="mask", **kw):
    g = [outputs(d[n]) for n in "qkv"]
    plan.sp_attention_backward(d["q"], d["k"], d["v"], kw.pop("o", ref["o"]), kw.pop("lse", ref["lse"]), d["do"], *g,
                               scale=ref["scale"], **mask_args(c, d["mask"], form), **kw)
    return g


def heads(c, x):
    """Global [B, N, H, ...] -> one contiguous tensor per rank."""
    return [y.contiguous() for y in x.chunk(c.P, 2)]


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_fused(c):
    d = R.inputs(c, 1)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    g = run_fused(c, plan, d, ref, "ranges" if c.mask == "ranges" else "mask")
    assert plan.sync_status() == 0
    for n, x in zip(("dq", "dk", "dv"), g):
        R.check(x, ref[n], ref["e_" + n], n)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_staged(c):
    """The head-sharded call.  The shards' gradients are split by head here
    (owner's copies), which is what to_heads gathers."""
    d = R.inputs(c, 2)
    for p in range(1, c.P):  # one gradient for the gathered replicated rows
        rep, _ = R._parts(c, d["do"][p], p, c.rep_q)
        rep.zero_()
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    q, k, v = (heads(c, R.to_global(c, d[n], i)) for n, i in zip("qkv", (False, True, True)))
    o, lse, do = (heads(c, ref["h"][n]) for n in ("o", "lse", "do"))
    g = [outputs(x) for x in (q, k, v)]
    plan.attention_backward(q, k, v, o, lse, do, *g, scale=ref["scale"], **mask_args(c, d["mask"], "mask"))
    assert plan.sync_status() == 0
    for n, x, is_kv in zip(("dq", "dk", "dv"), g, (False, True, True)):
        want, bound = (heads(c, R.to_global(c, t, is_kv)) for t in (ref[n], ref["e_" + n]))
        R.check(x, want, bound, n)


# few tiles, of long loops: shared by two or four CTAs each
SPLIT = [
    R.Case("one-head", 1, (2000,), 0, "none", 1, 1, 128),
    R.Case("one-head-ranges", 1, (1100,), 0, "none", 1, 1, 64, mask="ranges"),
    R.Case("shared-kv", 1, (1025,), 0, "none", 4, 1, 128, mask="random"),
    R.Case("shared-kv-prefix", 1, (700, 260), 140, "prefix", 8, 2, 128, mask="ranges"),
    R.Case("suffix-zero", 2, (1000,), 200, "suffix", 2, 1, 64, rows="zero", mask="random"),
    R.Case("self", 1, (900,), 129, "prefix", 4, 1, 128, rows="self", mask="random"),
    R.Case("kv-prefix-self", 1, (600, 600), 70, "kv_prefix", 4, 2, 64, rows="self", mask="ranges"),
    R.Case("few-keys", 1, (1500,), 0, "none", 4, 1, 128, mask="tail"),
    R.Case("no-key", 1, (1500,), 0, "none", 2, 1, 128, mask="none"),
    R.Case("two-parts", 1, (2048,), 0, "none", 8, 2, 128),
]


@pytest.mark.parametrize("c", SPLIT, ids=ids)
def test_few_tiles(c):
    """Right, and the same bits on every call; nothing behind the rows written."""
    import torch
    d = R.inputs(c, 21)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    g = run_fused(c, plan, d, ref)
    assert plan.sync_status() == 0
    for n, x in zip(("dq", "dk", "dv"), g):
        R.check(x, ref[n], ref["e_" + n], n)
    for _ in range(3):
        again = run_fused(c, plan, d, ref)
        for x, y in zip(sum(g, []), sum(again, [])):
            assert torch.equal(x, y)


@pytest.mark.parametrize("c", [R.Case("rounds", 2, (900,), 0, "none", 24, 8, 64, rows="zero", mask="random"),
                               R.Case("rounds-text", 1, (800, 801), 150, "prefix", 16, 16, 128, mask="ranges")], ids=ids)
def test_more_ctas_than_sms(c):
    d = R.inputs(c, 22)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    g = run_fused(c, plan, d, ref)
    assert plan.sync_status() == 0
    for n, x in zip(("dq", "dk", "dv"), g):
        R.check(x, ref[n], ref["e_" + n], n)


@pytest.mark.parametrize("mode", ["prefix", "kv_prefix"])
def test_conventions_are_one_without_a_mask(mode):
    """No mask, no masked row: every convention gives the same bits, right ones."""
    import torch
    got = []
    for rows in ("sdpa", "zero", "self"):
        c = R.Case("no-mask", 1, (300, 211), 140, mode, 4, 2, 64, rows=rows)
        d = R.inputs(c, 24)
        ref = R.reference(c, d)
        plan = R.plan_of(c)
        got.append(sum(run_fused(c, plan, d, ref), []))
        assert plan.sync_status() == 0
        for n, x in zip(("dq", "dk", "dv"), (got[-1][:2], got[-1][2:4], got[-1][4:])):
            R.check(x, ref[n], ref["e_" + n], n)
    for other in got[1:]:
        for x, y in zip(got[0], other):
            assert torch.equal(x, y)


def test_few_tiles_at_once_and_in_graphs():
    """Calls whose CTAs work in clusters, several under way at once on streams of
    their own and replayed from graphs: the bits of a call alone."""
    import torch
    live = []
    for i, c in enumerate((SPLIT[0], SPLIT[3], SPLIT[5], SPLIT[9])):
        d = R.inputs(c, 30 + i)
        ref = R.reference(c, d)
        plan = R.plan_of(c)
        want = run_fused(c, plan, d, ref)
        torch.cuda.synchronize()
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        ws = torch.empty(plan.attention_backward_workspace(), dtype=torch.uint8, device="cuda")
        got = [outputs(d[n]) for n in "qkv"]
        with torch.cuda.graph(graph, stream=s):
            plan.sp_attention_backward(d["q"], d["k"], d["v"], ref["o"], ref["lse"], d["do"], *got, scale=ref["scale"],
                                       workspace=ws, **mask_args(c, d["mask"], "mask"))
        live.append((c, plan, d, ref, want, s, graph, got, torch.cuda.Stream()))
    eager = []
    for _ in range(4):
        for c, plan, d, ref, want, s, graph, got, s2 in live:
            with torch.cuda.stream(s):
                graph.replay()
            with torch.cuda.stream(s2):
                eager.append((want, run_fused(c, plan, d, ref)))
    torch.cuda.synchronize()
    for c, plan, *_ in live:
        assert plan.sync_status() == 0
    for want, got in eager + [(x[4], x[7]) for x in live]:
        for x, y in zip(sum(want, []), sum(got, [])):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("c", [CASES[6], CASES[13]], ids=ids)
def test_against_differences(c):
    """<gradient, direction> against the difference quotient of <o, do> in 64
    bits, one direction for each of q, k, v."""
    import torch
    d = R.inputs(c, 3)
    ref = R.reference(c, d)
    g = run_fused(c, R.plan_of(c), d, ref)
    gen = torch.Generator(device="cuda").manual_seed(5)

    def loss(t):
        o, _, _ = R.attention(c, *(R.to_global(c, t[n], i) for n, i in zip("qkv", (False, True, True))), d["mask"],
                              ref["scale"])
        return sum(float((x * y.double()).sum()) for x, y in zip(R.to_shards(c, o, False), d["do"]))

    base = {n: [x.double() for x in d[n]] for n in "qkv"}
    for i, n in enumerate("qkv"):
        dirs = [torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64) for x in base[n]]
        h = 1e-4
        up, down = (loss({**base, n: [x + s * y for x, y in zip(base[n], dirs)]}) for s in (h, -h))
        want = (up - down) / (2 * h)
        got = sum(float((x.double() * y).sum()) for x, y in zip(g[i], dirs))
        # a random direction: the elements' errors (2^-7 of the norm) enter with random signs, 5 deviations
        norm = math.sqrt(sum(float(x.double().square().sum()) for x in g[i]))
        assert abs(got - want) <= 5 * 2.0 ** -7 * norm + 1e-5 * abs(want), (n, got, want, norm)


def test_same_bits_any_workspace():
    """Every call gives the same bits, whatever the workspace held."""
    import torch
    c = CASES[6]
    d = R.inputs(c, 4)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    first = run_fused(c, plan, d, ref)
    n = plan.attention_backward_workspace()
    for fill in (0x00, 0xFF, 0x7F):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        again = run_fused(c, plan, d, ref, workspace=ws)
        for a, b in zip(first, again):
            for x, y in zip(a, b):
                assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3.0e38])
@pytest.mark.parametrize("c", [R.Case("zero", 2, (300, 77), 140, "suffix", 4, 2, 128, rows="zero", mask="ranges"),
                               R.Case("zero-d64", 1, (200, 200), 129, "prefix", 4, 4, 64, rows="zero", mask="random"),
                               R.Case("sdpa", 1, (300, 300), 60, "kv_prefix", 4, 2, 128, mask="ranges"),
                               R.Case("sdpa-d64", 2, (700,), 0, "none", 2, 2, 64, mask="tail")], ids=ids)
def test_masked_places_hold_anything(c, fill):
    """Masked keys' k and v, and what a zeroed query row's q, o, do hold, change
    no bit of the result."""
    import torch
    d = R.inputs(c, 6)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    want = run_fused(c, plan, d, ref)
    own = R.to_shards(c, (d["mask"][:, c.R:] if c.mode == "kv_prefix" else d["mask"]), False)
    key = R.to_shards(c, d["mask"], True)
    for p in range(c.P):
        for n in "kv":
            d[n][p][~key[p]] = fill
        if c.rows == "zero":
            for t in (d["q"][p], d["do"][p], ref["o"][p]):
                t[~own[p]] = fill
    got = run_fused(c, plan, d, ref)
    assert plan.sync_status() == 0
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))


# the last tile of a shard's image rows ends inside the tile (and, in suffix mode, before the shard's text rows)
COPIES = [
    R.Case("suffix", 1, (300, 77), 140, "suffix", 4, 2, 128, mask="ranges"),
    R.Case("suffix-d64", 2, (45, 257, 130), 33, "suffix", 6, 3, 64),
    R.Case("suffix-zero", 1, (300, 77), 140, "suffix", 4, 4, 64, rows="zero", mask="random"),
    R.Case("suffix-self", 2, (300, 77), 140, "suffix", 4, 2, 128, rows="self", mask="random"),
    R.Case("suffix-self-d64", 1, (200, 333), 70, "suffix", 4, 4, 64, rows="self", mask="ranges"),
    R.Case("suffix-few-tiles", 1, (900, 701), 129, "suffix", 2, 2, 128, rows="self", mask="random"),
    R.Case("suffix-many-tiles", 2, (500, 631), 60, "suffix", 16, 16, 64),
    R.Case("prefix", 1, (300, 77), 140, "prefix", 4, 2, 128, rows="self", mask="random"),
    R.Case("kv-prefix", 2, (300, 77), 140, "kv_prefix", 4, 2, 64, mask="ranges"),
]


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3.0e38])
@pytest.mark.parametrize("c", COPIES, ids=ids)
def test_copies_that_are_not_read_hold_anything(c, fill):
    """A shard's copies of the replicated rows of heads that another rank owns
    are not read (do's apart): they change no bit of the result."""
    import torch
    d = R.inputs(c, 25)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    want = run_fused(c, plan, d, ref)
    for n, x in zip(("dq", "dk", "dv"), want):
        R.check(x, ref[n], ref["e_" + n], n)
    for ts, rep_rows in ((d["q"], c.rep_q), (d["k"], c.R), (d["v"], c.R), (ref["o"], c.rep_q), (ref["lse"], c.rep_q)):
        per = ts[0].shape[2] // c.P
        for p, t in enumerate(ts):
            rep, _ = R._parts(c, t, p, rep_rows)
            rep[:, :, :p * per] = fill
            rep[:, :, (p + 1) * per:] = fill
    got = run_fused(c, plan, d, ref)
    assert plan.sync_status() == 0
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_writes_nothing_else():
    """Outputs inside larger buffers: the memory around them stays as it was."""
    import torch
    c = CASES[8]
    d = R.inputs(c, 7)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    bufs, g = [], []
    for n in "qkv":
        ts = []
        for x in d[n]:
            b = torch.full((x.numel() + 2048,), 7.0, dtype=torch.bfloat16, device="cuda")
            ts.append(b[1024:1024 + x.numel()].view(x.shape))
            bufs.append((b, x.numel()))
        g.append(ts)
    plan.sp_attention_backward(d["q"], d["k"], d["v"], ref["o"], ref["lse"], d["do"], *g, key_mask=d["mask"])
    for n, x in zip(("dq", "dk", "dv"), g):
        R.check(x, ref[n], ref["e_" + n], n)
    for b, n in bufs:
        assert (b[:1024] == 7).all() and (b[1024 + n:] == 7).all()


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last batch has the bits of a call
    of its own."""
    import torch
    c = R.Case("wide", 1, (70,), 0, "none", 64, 64, 128)
    B = 2 ** 31 // (70 * 64 * 128) + 2
    d = R.inputs(c, 8)
    ref = R.reference(c, d)
    one = run_fused(c, R.plan_of(c), d, ref)
    from ulysses_sequence_attention_uly_gb300 import Plan
    plan = Plan(B, 1, 70, 0, "none", 64, 64, 128)
    big = {n: [torch.zeros((B, 70, 64, 128), dtype=torch.bfloat16, device="cuda")] for n in ("q", "k", "v", "o", "do")}
    lse = torch.zeros((B, 70, 64), device="cuda")
    for n, x in (("q", d["q"]), ("k", d["k"]), ("v", d["v"]), ("o", ref["o"]), ("do", d["do"])):
        big[n][0][B - 1] = x[0][0]
    lse[B - 1] = ref["lse"][0][0]
    g = [outputs(big[n]) for n in "qkv"]
    plan.sp_attention_backward(big["q"], big["k"], big["v"], big["o"], [lse], big["do"], *g)
    assert plan.sync_status() == 0
    for x, y in zip(g, one):
        assert torch.equal(x[0][B - 1].view(torch.int16), y[0][0].view(torch.int16))
        assert (x[0][0] == 0).all()


def test_forward_then_backward_of_every_form():
    """o and lse of the fused call and of the one-launch ring: the gradient of
    either is that of the attention."""
    import torch
    c = R.Case("forms", 1, (200, 130), 50, "prefix", 4, 2, 128, mask="ranges")
    d = R.inputs(c, 9)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    o = outputs(d["q"])
    lse = [torch.empty(x.shape[:3], device="cuda") for x in d["q"]]
    plan.sp_attention(d["q"], d["k"], d["v"], o, key_mask=d["mask"], lse=lse)
    g = run_fused(c, plan, d, ref, o=o, lse=lse)
    for n, x in zip(("dq", "dk", "dv"), g):
        R.check(x, ref[n], ref["e_" + n], n)
    for p in range(1, c.P):
        d["do"][p][:, :c.R] = 0
    ref = R.reference(c, d)
    q, k, v = (heads(c, R.to_global(c, d[n], i)) for n, i in zip("qkv", (False, True, True)))
    oh, lh = outputs(q), [torch.empty(x.shape[:3], device="cuda") for x in q]
    plan.ring_attention(q, k, v, oh, [0, 170, c.nk], key_mask=d["mask"], lse=lh)
    g = [outputs(x) for x in (q, k, v)]
    plan.attention_backward(q, k, v, oh, lh, heads(c, ref["h"]["do"]), *g, key_mask=d["mask"])
    for n, x, is_kv in zip(("dq", "dk", "dv"), g, (False, True, True)):
        want, bound = (heads(c, R.to_global(c, t, is_kv)) for t in (ref[n], ref["e_" + n]))
        R.check(x, want, bound, n)


def test_streams_and_graphs():
    """Two captured calls of one plan with their own workspaces, replayed at the
    same time on two streams, after their inputs changed in place, beside a
    forward call; each gives the bits of an eager call."""
    import torch
    c = CASES[6]
    plan = R.plan_of(c)
    sets = []
    for seed in (10, 11):
        d = R.inputs(c, seed)
        ref = R.reference(c, d)
        sets.append([d, ref, run_fused(c, plan, d, ref)])  # warm-up and one of the two wanted results
    n = plan.attention_backward_workspace()
    live = []
    for d, ref, _ in sets:
        s = torch.cuda.Stream()
        state = {n_: [torch.zeros_like(x) for x in d[n_]] for n_ in ("q", "k", "v", "do")}
        o, lse = [torch.zeros_like(x) for x in ref["o"]], [torch.zeros_like(x) for x in ref["lse"]]
        g = [outputs(d[n_]) for n_ in "qkv"]
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        mask = torch.ones_like(d["mask"])
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan.sp_attention_backward(state["q"], state["k"], state["v"], o, lse, state["do"], *g, key_mask=mask,
                                       scale=ref["scale"], workspace=ws)
        live.append((s, graph, state, o, lse, g, mask))
    for (d, ref, _), (_, _, state, o, lse, g, mask) in zip(sets, live):
        for n_ in ("q", "k", "v", "do"):
            for x, y in zip(state[n_], d[n_]):
                x.copy_(y)
        for x, y in zip(o + lse, ref["o"] + ref["lse"]):
            x.copy_(y)
        mask.copy_(d["mask"])
    torch.cuda.synchronize()
    fo = outputs(sets[0][0]["q"])
    for _ in range(5):
        for s, graph, *_ in live:
            with torch.cuda.stream(s):
                graph.replay()
        plan.sp_attention(sets[0][0]["q"], sets[0][0]["k"], sets[0][0]["v"], fo, key_mask=sets[0][0]["mask"])
    torch.cuda.synchronize()
    assert plan.sync_status() == 0
    for (_, _, want), (_, _, _, _, _, g, _) in zip(sets, live):
        for a, b in zip(g, want):
            for x, y in zip(a, b):
                assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_withheld_load_times_out():
    """A tile that never arrives ends in ULY_ERR_TIMEOUT in each kernel, and the
    next call is right."""
    import torch
    import ulysses_sequence_attention_uly_gb300 as uly
    c = CASES[5]
    d = R.inputs(c, 12)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    plan.set_wait_limit(20_000_000)
    plan.test_withhold_fill(2)
    run_fused(c, plan, d, ref)
    assert plan.sync_status() == uly.ULY_ERR_TIMEOUT
    plan.test_withhold_fill(-1)
    plan.set_wait_limit(4_000_000_000)
    g = run_fused(c, plan, d, ref)
    torch.cuda.synchronize()
    assert plan.sync_status() == 0
    for n, x in zip(("dq", "dk", "dv"), g):
        R.check(x, ref[n], ref["e_" + n], n)


def test_withheld_load_of_unsplit_tiles_times_out():
    """The same where every tile has a CTA of its own, with masks by the queries'
    own tokens and replicated rows."""
    import torch
    import ulysses_sequence_attention_uly_gb300 as uly
    c = R.Case("withheld", 2, (500, 431), 140, "suffix", 16, 8, 64, rows="zero", mask="random")
    d = R.inputs(c, 14)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    for fill in (0, 1, 3):
        plan.set_wait_limit(20_000_000)
        plan.test_withhold_fill(fill)
        run_fused(c, plan, d, ref)
        assert plan.sync_status() == uly.ULY_ERR_TIMEOUT
    plan.test_withhold_fill(-1)
    plan.set_wait_limit(4_000_000_000)
    g = run_fused(c, plan, d, ref)
    torch.cuda.synchronize()
    assert plan.sync_status() == 0
    for n, x in zip(("dq", "dk", "dv"), g):
        R.check(x, ref[n], ref["e_" + n], n)


def test_refusals():
    import torch
    import ulysses_sequence_attention_uly_gb300 as uly
    c = CASES[6]
    d = R.inputs(c, 13)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    g = [outputs(d[n]) for n in "qkv"]
    args = [d["q"], d["k"], d["v"], ref["o"], ref["lse"], d["do"]] + g

    def refuse(exc, status=None, change=None, **kw):
        a = list(args)
        for i, x in (change or {}).items():
            a[i] = x
        with pytest.raises(exc) as e:
            plan.sp_attention_backward(*a, **kw)
        if status is not None:
            assert e.value.status == status

    refuse(ValueError, change={4: None})
    refuse(ValueError, change={0: d["q"][:1]})
    refuse(ValueError, change={5: [x.float() for x in d["do"]]})
    refuse(ValueError, change={3: [x[:, :-1] for x in ref["o"]]})
    refuse(ValueError, change={7: [x.transpose(2, 3).contiguous().transpose(2, 3) for x in g[1]]})
    refuse(ValueError, change={4: [x.double() for x in ref["lse"]]})
    refuse(ValueError, key_mask=d["mask"][:, 1:])
    n = plan.attention_backward_workspace()
    refuse(ValueError, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    big = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, workspace=big[16:])
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, scale=0.0)
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, scale=float("nan"))
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, key_mask=d["mask"],
           key_ranges=torch.zeros((c.B, 1, 2), dtype=torch.int32, device="cuda"))
    # an output that is an input, twice the same output
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, change={6: d["q"]})
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, change={8: g[1]})
    refuse(uly.UlyError, uly.ULY_ERR_INVALID, change={7: [g[1][0], g[1][0]]})
    c8 = R.Case("e4m3", 1, (64,), 0, "none", 1, 1, 128)
    p8 = R.plan_of(c8, dtype="e4m3")
    x8 = [torch.zeros((1, 64, 1, 128), dtype=torch.uint8, device="cuda")]
    xb = [torch.zeros((1, 64, 1, 128), dtype=torch.bfloat16, device="cuda")]
    with pytest.raises(uly.UlyError):
        p8.sp_attention_backward(x8, x8, x8, xb, [torch.zeros((1, 64, 1), device="cuda")], xb, xb, xb, xb)
    # nothing was written
    torch.cuda.synchronize()
    assert all(torch.isnan(x).all() for t in g for x in t)


@pytest.mark.parametrize("fused", [True, False])
def test_masks_inside_written_memory_are_refused(fused):
    """A mask or ranges inside the workspace or an output would be overwritten
    while the call still reads them."""
    import torch
    import ulysses_sequence_attention_uly_gb300 as uly
    c = CASES[6]
    d = R.inputs(c, 15)
    plan = R.plan_of(c)
    shape = (lambda n: d[n]) if fused else (lambda n: heads(c, R.to_global(c, d[n], n in "kv")))  # noqa: E731
    q, k, v, do = (shape(n) for n in ("q", "k", "v", "do"))
    lse = [torch.zeros(x.shape[:3], device="cuda") for x in q]
    g = [outputs(x) for x in (q, k, v)]
    n = plan.attention_backward_workspace()
    ws = torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
    call = plan.sp_attention_backward if fused else plan.attention_backward
    for t in (ws, g[0][0], g[1][1], g[2][0]):
        b = t.view(-1).view(torch.uint8)
        for kw in ({"key_mask": b[:c.B * c.nk].view(c.B, c.nk)},
                   {"key_mask": b[-c.B * c.nk:].view(c.B, c.nk)},
                   {"key_ranges": b[256:256 + c.B * 24].view(torch.int32).view(c.B, 3, 2)}):
            with pytest.raises(uly.UlyError) as e:
                call(q, k, v, q, lse, do, *g, workspace=ws, **kw)
            assert e.value.status == uly.ULY_ERR_INVALID
    torch.cuda.synchronize()
    assert (ws == 0x55).all() and all(torch.isnan(x).all() for t in g for x in t)


@pytest.mark.parametrize("fused", [True, False])
def test_misaligned_ranges_are_refused(fused):
    """Through the C ABI (the binding's tensors are aligned): ranges that are not
    on a 4-byte boundary would fault when they are read."""
    import torch
    import ulysses_sequence_attention_uly_gb300 as uly
    c = CASES[0]
    plan = R.plan_of(c)
    x = [torch.zeros((c.B, c.n, c.Hq, c.D), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    lse = torch.zeros((c.B, c.n, c.Hq), device="cuda")
    rg = torch.zeros(6, dtype=torch.int32, device="cuda")
    n = plan.attention_backward_workspace()
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    fn = uly.lib().uly_sp_attention_backward if fused else uly.lib().uly_attention_backward
    q, k, v, o, do, dq, dk, dv, l = (uly._ptr_array([t]) for t in x + [lse])
    for off in (1, 2, 3):
        assert fn(plan._h, q, k, v, o, l, do, None, rg.data_ptr() + off, 2, 0.1, dq, dk, dv, ws.data_ptr(), n,
                  None) == uly.ULY_ERR_INVALID


@pytest.mark.parametrize("c", [R.Case("plain", 1, (1500,), 0, "none", 8, 8, 128),
                               R.Case("suffix", 1, (700, 461), 140, "suffix", 8, 4, 128, mask="random"),
                               R.Case("zero-d64", 1, (700, 500), 0, "none", 8, 8, 64, rows="zero", mask="random"),
                               R.Case("plain-d64", 1, (1500,), 0, "none", 12, 4, 64),
                               R.Case("shared", 1, (1500,), 0, "none", 4, 1, 128),
                               R.Case("shared-self", 1, (700, 700), 60, "prefix", 2, 2, 64, rows="self", mask="random")],
                         ids=ids)
def test_any_wait_limit(c):
    """However short the limit of a wait is (the hardware waits a while of its own
    before the clock is read), the call ends with ULY_ERR_TIMEOUT or is right, and
    the next one is right."""
    import torch
    import ulysses_sequence_attention_uly_gb300 as uly
    d = R.inputs(c, 16)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    want = run_fused(c, plan, d, ref)
    assert plan.sync_status() == 0
    same = lambda g: all(torch.equal(x, y) for a, b in zip(g, want) for x, y in zip(a, b))  # noqa: E731
    for ns in (1, 1500, 4000, 8000, 12000, 16000, 24000):
        plan.set_wait_limit(ns)
        got = run_fused(c, plan, d, ref)
        status = plan.sync_status()
        assert status in (uly.ULY_ERR_TIMEOUT, uly.ULY_OK), (ns, status)
        assert status == uly.ULY_ERR_TIMEOUT or same(got)
        plan.set_wait_limit(4_000_000_000)
        assert same(run_fused(c, plan, d, ref)) and plan.sync_status() == 0


# one tile of queries and many of keys: only a dQ CTA has a load of that number; one tile with admitted keys and many of
# queries: only a dK/dV CTA has.  With 16 heads every tile has a CTA of its own, with one head four share it.
WITHHELD = [
    (R.Case("dq", 1, (20,), 1500, "kv_prefix", 16, 16, 128), (1, 5, 12), "dq"),
    (R.Case("dq-d64", 2, (30,), 1400, "kv_prefix", 16, 16, 64, mask="random"), (1, 2, 10), "dq"),
    (R.Case("dq-twice", 1, (7, 7), 100, "suffix", 64, 64, 128), (4, 5), "dq"),
    (R.Case("dq-split", 1, (20,), 1500, "kv_prefix", 1, 1, 128), (1, 2), "dq"),
    (R.Case("dq-split-d64", 1, (20,), 2100, "kv_prefix", 1, 1, 64, rows="self", mask="random"), (1, 3), "dq"),
    (R.Case("dkdv", 1, (1500,), 0, "none", 16, 16, 128, mask="tail"), (1, 2, 11), "dkdv"),
    (R.Case("dkdv-own", 1, (1500,), 0, "none", 16, 16, 64, rows="zero", mask="tail"), (1, 3, 10), "dkdv"),
    (R.Case("dkdv-split", 1, (1500,), 0, "none", 1, 1, 128, mask="tail"), (1, 2), "dkdv"),
    (R.Case("dkdv-split-d64", 1, (2000,), 0, "none", 1, 1, 64, mask="tail"), (1, 2, 3), "dkdv"),
]


@pytest.mark.parametrize("c, fills, kind", WITHHELD, ids=[x[0].name for x in WITHHELD])
def test_withheld_load_of_one_kind_times_out(c, fills, kind):
    """A tile that never arrives in dQ's CTAs alone, and in dK's and dV's alone,
    ends in ULY_ERR_TIMEOUT; the other kind's outputs and the next call are right."""
    import torch
    import ulysses_sequence_attention_uly_gb300 as uly
    d = R.inputs(c, 17)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    want = run_fused(c, plan, d, ref)
    assert plan.sync_status() == 0
    for n, x in zip(("dq", "dk", "dv"), want):
        R.check(x, ref[n], ref["e_" + n], n)
    for fill in fills:
        plan.set_wait_limit(20_000_000)
        plan.test_withhold_fill(fill)
        got = run_fused(c, plan, d, ref)
        assert plan.sync_status() == uly.ULY_ERR_TIMEOUT
        for a, b in zip(got[1:], want[1:]) if kind == "dq" else zip(got[:1], want[:1]):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
        plan.test_withhold_fill(-1)
        plan.set_wait_limit(4_000_000_000)
        again = run_fused(c, plan, d, ref)
        assert plan.sync_status() == 0
        for a, b in zip(again, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


# more key tiles than one turn of the tile tables' loop takes (256), few queries
LONG_KEYS = [
    R.Case("sdpa-ranges", 2, (70,), 40000, "kv_prefix", 4, 2, 64, mask="ranges"),
    R.Case("zero-random", 1, (130, 20), 70000, "kv_prefix", 2, 2, 128, rows="zero", mask="random"),
    R.Case("self-random", 1, (200,), 33000, "kv_prefix", 2, 1, 128, rows="self", mask="random"),
    R.Case("self-ranges", 1, (90, 61), 66001, "kv_prefix", 2, 2, 64, rows="self", mask="ranges"),
    R.Case("all", 1, (50,), 33100, "kv_prefix", 2, 2, 128),
    R.Case("tail", 1, (300,), 99000, "kv_prefix", 1, 1, 64, mask="tail"),
    R.Case("none", 1, (20,), 40000, "kv_prefix", 1, 1, 128, mask="none"),
]


@pytest.mark.parametrize("c", LONG_KEYS, ids=ids)
def test_long_key_lists(c):
    d = R.inputs(c, 18)
    ref = R.reference(c, d)
    plan = R.plan_of(c)
    g = run_fused(c, plan, d, ref, "ranges" if c.mask == "ranges" else "mask")
    assert plan.sync_status() == 0
    for n, x in zip(("dq", "dk", "dv"), g):
        R.check(x, ref[n], ref["e_" + n], n)


def test_two_threads_one_plan():
    """Gradient calls of one plan from two threads at once, each on a stream and
    with tensors of its own, beside norm_rope calls: the bits of calls alone."""
    import threading

    import torch
    c = R.Case("threads", 2, (300, 77), 140, "suffix", 4, 2, 128, rows="zero", mask="random")
    plan = R.plan_of(c)
    jobs = []
    for seed in (40, 41):
        d = R.inputs(c, seed)
        ref = R.reference(c, d)
        nq, nk = outputs(d["q"]), outputs(d["k"])
        plan.norm_rope(d["q"], d["k"], nq, nk)
        jobs.append((d, ref, run_fused(c, plan, d, ref), nq + nk))
    torch.cuda.synchronize()
    wrong = []

    def work(d, ref, want, norm):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(50):
                    g = run_fused(c, plan, d, ref)
                    nq, nk = outputs(d["q"]), outputs(d["k"])
                    plan.norm_rope(d["q"], d["k"], nq, nk)
                    s.synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(sum(g, []) + nq + nk, sum(want, []) + norm)):
                        wrong.append("other bits")
        except Exception as e:  # noqa: BLE001 - reported below
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
    assert plan.sync_status() == 0
