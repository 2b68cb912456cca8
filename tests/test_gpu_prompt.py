"""Causal attention over packed prompts on the shards (uly_sp_prompt_attention)
against 64 bits: lengths around the tiles' ends, sequences across shards, empty
and single-row ones, rows of no sequence, every kind of head group."""
import pytest
import torch

from tests import _serve as R

pytestmark = pytest.mark.gpu

CASES = [
    R.Prompt("one row", (1,), (1,), 1, 1, 64),
    R.Prompt("short", (17,), (17,), 4, 2, 64),
    R.Prompt("a tile", (128,), (128,), 2, 1, 128),
    R.Prompt("past a tile", (129,), (129,), 2, 2, 128),
    R.Prompt("two tiles", (256,), (256,), 3, 1, 128),
    R.Prompt("past two tiles", (257,), (257,), 1, 1, 128),
    R.Prompt("tile ends", (1500,), (127, 128, 129, 255, 256, 257, 1), 4, 2, 128, first=100),
    R.Prompt("single rows", (700,), (1,) * 300 + (0,) * 7 + (1,) * 200, 4, 1, 64, first=3),
    R.Prompt("four shards", (300,) * 4, (1000, 0, 1, 199), 8, 4, 128),
    R.Prompt("uneven shards", (333, 1, 77, 500), (410, 2, 400), 4, 4, 64, first=50),
    R.Prompt("shards of a row", (1,) * 16, (5, 9), 16, 16, 64, first=1),
    R.Prompt("tiny shards", (3, 200, 5, 130), (330,), 4, 4, 128, first=2),
    R.Prompt("odd group", (600,), (77, 300, 223), 6, 2, 128),
    R.Prompt("group of five", (400,), (399,), 5, 1, 64),
    R.Prompt("group of eight", (520,), (130, 390), 16, 2, 128),
    R.Prompt("long rows", (2000, 1300), (3200,), 4, 2, 128, first=7, std=0.7),
    R.Prompt("long rows, odd group", (2000, 1300), (3200,), 6, 2, 64, first=7),
    R.Prompt("peaked", (512,), (512,), 4, 2, 128, std=4.0),
    # (more items than SMs, and more than two an SM: the ones above mostly have fewer)
    R.Prompt("tile ends, some heads", (800, 700), (127, 128, 129, 255, 256, 257, 1), 28, 14, 128, first=100),
    R.Prompt("tile ends, some odd groups", (800, 700), (127, 128, 129, 255, 256, 257, 1), 20, 20, 64, first=100),
    R.Prompt("long rows, some heads", (2100,), (2100,), 16, 8, 64),
    R.Prompt("tile ends, many heads", (1500,), (127, 128, 129, 255, 256, 257, 1), 48, 8, 128, first=100),
    R.Prompt("tile ends, many odd groups", (1500,), (127, 128, 129, 255, 256, 257, 1), 24, 8, 64, first=100),
    R.Prompt("long rows, many heads", (2000, 1300, 9, 700), (3200, 0, 77, 700), 32, 8, 128, first=7, std=0.7),
    R.Prompt("long rows, many odd groups", (2000, 1300), (3200, 50), 20, 20, 128, first=7),
    R.Prompt("no rows", (64,), (0, 0), 2, 2, 64, first=9),
]


def run(c, d, plan=None, **kw):
    plan = plan or R.plan_of(c)
    plan.prompt_attention(d["q"], d["k"], d["v"], d["o"], d["starts"], lse=d["lse"], **kw)
    torch.cuda.synchronize()
    assert plan.sync_status() == 0
    return plan


@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_against_64_bits(c):
    d = R.prompt_inputs(c, 1)
    run(c, d)
    R.check_prompt(c, d, d["o"], d["lse"])


@pytest.mark.parametrize("c", CASES[6:12:2], ids=lambda c: c.name)
def test_scale_and_no_lse(c):
    d = R.prompt_inputs(c, 2)
    plan = R.plan_of(c)
    plan.prompt_attention(d["q"], d["k"], d["v"], d["o"], d["starts"], scale=0.031)
    torch.cuda.synchronize()
    R.check_prompt(c, d, d["o"], None, scale=0.031)


def _mixed(n, most, empty=()):
    return tuple(0 if i in empty else 1 + (i * 29) % most for i in range(n))


# more sequences than a warp has lanes, and yet so little work that the CTAs find their items by themselves
FOUND = [
    R.Prompt("33", (700,), _mixed(33, 40), 2, 1, 128),
    R.Prompt("64, empty ones at a turn's end", (950,), _mixed(64, 30, (30, 31, 32, 33, 63)), 2, 1, 64, first=3),
    R.Prompt("65, the last alone", (300,), (0,) * 64 + (300,), 2, 1, 128),
    R.Prompt("33, the first 32 empty", (270, 20), (0,) * 32 + (290,), 4, 2, 64),
    R.Prompt("a long one over a turn's end", (500, 600), _mixed(31, 9) + (700,) + _mixed(12, 9), 4, 2, 128, first=5),
    R.Prompt("100 over shards", (400, 350), _mixed(100, 13, (31, 32)), 4, 2, 128, first=7),
    R.Prompt("40 over shards, odd groups", (333, 400), _mixed(32, 9) + (300, 0, 5, 4, 3, 2, 1, 1), 6, 2, 64, first=2),
    R.Prompt("90, odd group", (2000,), _mixed(90, 20, (32, 64)), 3, 1, 128, first=1),
    R.Prompt("220, two items a CTA", (700,), _mixed(220, 4, (31, 95, 96)), 2, 1, 64),
]


@pytest.mark.parametrize("c", FOUND, ids=lambda c: c.name)
def test_more_sequences_than_lanes(c):
    d = R.prompt_inputs(c, 15)
    plan = R.plan_of(c)
    assert plan.prompt_attention_workspace(len(c.seqs)) == 0
    run(c, d, plan)
    R.check_prompt(c, d, d["o"], d["lse"])


def test_starts_that_fall_at_a_turn_of_lanes():
    c = R.Prompt("falling", (500, 300), (800,), 4, 2, 64)
    starts = [8 * i for i in range(31)] + [400, 30, 20, 10] + [250 + 5 * i for i in range(29)] + [0, 0, 640, 90] + [700]
    d = R.prompt_inputs(c, 16)
    d["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    plan = R.plan_of(c)
    assert plan.prompt_attention_workspace(len(starts) - 1) == 0
    run(c, d, plan)
    top = torch.tensor(starts).cummax(0).values.tolist()
    as_is = R.Prompt("falling", c.shards, tuple(b - a for a, b in zip(top, top[1:])), 4, 2, 64, first=top[0])
    R.check_prompt(as_is, d, d["o"], d["lse"])


def test_the_most_sequences():
    """65536 sequences of two rows: the second row's weights in closed form."""
    import ulysses_sequence_attention_uly_gb300 as uly
    n, D = 65536, 64
    plan = uly.Plan(1, 2, n, 0, "none", 4, 2, D)
    g = torch.Generator(device="cuda").manual_seed(19)
    q, k, v = ([torch.randn((1, n, h, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
               for h in (4, 2, 2))
    o, lse = [torch.full_like(x, 7.0) for x in q], [torch.full((1, n, 4), 7.0, device="cuda") for _ in range(2)]
    starts = torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda")
    plan.prompt_attention(q, k, v, o, starts, scale=0.125, lse=lse)
    assert plan.sync_status() == 0
    qq, kk, vv = (torch.cat(x, 1)[0].double().view(n, 2, -1, D) for x in (q, k, v))
    kk, vv = (x.repeat_interleave(2, 2) for x in (kk, vv))
    s = (qq[:, 1, None] * kk).sum(-1) * 0.125  # [n, 2 keys, heads]
    p = s.softmax(1)[..., None]
    want = torch.stack((vv[:, 0], (p * vv).sum(1)), 1)
    u, r = 2.0 ** -8, 2.0 ** -13  # as in the reference of the other cases
    err = torch.stack((vv[:, 0].abs(), (p * vv.abs()).sum(1)), 1) * (u + r) * (1 + u) + u * want.abs() + 1e-30
    R.check_rows(torch.cat(o, 1)[0].view(n, 2, 4, D), want, err, "o")
    wl = torch.stack(((qq[:, 0] * kk[:, 0]).sum(-1) * 0.125, s.logsumexp(1)), 1)
    R.check_rows(torch.cat(lse, 1)[0].view(n, 2, 4), wl, 2.0 ** -13 + 2.0 ** -22 * wl.abs(), "lse")
    too_many = torch.zeros(n + 2, dtype=torch.int32, device="cuda")
    with pytest.raises(uly.UlyError) as e:
        plan.prompt_attention(q, k, v, o, too_many)
    assert e.value.status == uly.ULY_ERR_UNSUPPORTED


def test_offsets_past_32_bits():
    """A sequence at the end of tensors of more than 2^32 bytes."""
    from ulysses_sequence_attention_uly_gb300 import Plan
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    n, H, D, tail = 450000, 40, 128, 1000
    plan = Plan(1, 1, n, 0, "none", H, H, D)
    c = R.Prompt("tail", (tail,), (300, 77), H, H, D, first=500)
    small = R.prompt_inputs(c, 20)
    big = {}
    for t in ("q", "k", "v", "o", "lse"):
        x = small[t][0]
        big[t] = torch.zeros((1, n) + x.shape[2:], dtype=x.dtype, device="cuda")
        big[t][:, n - tail:] = x
    starts = (small["starts"] + (n - tail)).int()
    plan.prompt_attention([big["q"]], [big["k"]], [big["v"]], [big["o"]], starts, lse=[big["lse"]])
    assert plan.sync_status() == 0
    R.check_prompt(c, small, [big["o"][:, n - tail:]], [big["lse"][:, n - tail:]])
    assert not big["o"][:, :n - tail].any() and not big["lse"][:, :n - tail].any()


def test_more_sequences_than_threads():
    lens = tuple((i * 7) % 4 for i in range(2500))
    c = R.Prompt("many", (2200, 2000), lens, 2, 2, 64, first=11)
    d = R.prompt_inputs(c, 3)
    run(c, d)
    R.check_prompt(c, d, d["o"], d["lse"])


MANY = [
    # more runs than shared memory holds the first units of (2048), with longer ones at both ends and in the middle
    R.Prompt("runs", (3500, 3000, 2500), (700,) + tuple(1 + i % 3 for i in range(1500)) + (900, 0, 257) +
             tuple(1 + i % 2 for i in range(1700)) + (600,), 6, 3, 64, first=13),
    R.Prompt("runs, odd groups", (6000, 2500), (700,) + tuple(1 + i % 3 for i in range(1500)) + (900, 0, 257) +
             tuple(1 + i % 2 for i in range(1000)) + (600,), 2, 2, 128, first=13),
    # so many rows that units of like length share a place in the order
    R.Prompt("rows", (140000, 130000), (9000,) + tuple(300 + (i * 797) % 2400 for i in range(150)) + (5000, 1, 128),
             4, 2, 64, first=129),
]


@pytest.mark.parametrize("c", MANY, ids=lambda c: c.name)
def test_tables_of_many_runs_and_many_rows(c):
    runs = sum(1 for a, b in zip(c.bounds, c.bounds[1:]) if b > a)
    assert c.bounds[-1] <= c.n and (runs > 2048 or c.n // 128 + len(c.shards) >= 2048)
    d = R.prompt_inputs(c, 17)
    plan = R.plan_of(c)
    assert plan.prompt_attention_workspace(len(c.seqs)) > 0
    run(c, d, plan)
    R.check_prompt(c, d, d["o"], d["lse"])


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 4, 128), (4, 4, 64)])
def test_the_same_rows_in_one_two_and_four_shards(Hq, Hkv, D):
    """Key tiles begin anew where a shard does, so that bits differ between the
    numbers of shards; each is within the bound of the same 64-bit result."""
    seqs = (300, 256, 1, 467)
    whole = R.prompt_inputs(R.Prompt("whole", (1024,), seqs, Hq, Hkv, D), 18)
    for shards in ((1024,), (512, 512), (700, 324), (256,) * 4, (130, 500, 1, 393)):
        c = R.Prompt("split", shards, seqs, Hq, Hkv, D)
        d = {n: [y.contiguous() for y in whole[n][0].split(list(shards), 1)] for n in ("q", "k", "v")}
        d["o"] = [torch.full_like(x, 7.0) for x in d["q"]]
        d["lse"] = [torch.full(x.shape[:3], 7.0, device="cuda") for x in d["q"]]
        d["starts"] = whole["starts"]
        run(c, d)
        R.check_prompt(c, d, d["o"], d["lse"])


@pytest.mark.parametrize("Hq", [96, 4])  # with tables, and without
def test_two_threads_one_plan(Hq):
    """Calls of one plan from two threads at once, each on a stream and with tensors
    of its own: the bits of calls alone."""
    import threading
    c = R.Prompt("threads", (500, 400), (123, 456, 200), Hq, Hq // 2, 128, first=30)
    plan = R.plan_of(c)
    assert (plan.prompt_attention_workspace(3) > 0) == (Hq == 96)
    jobs, wrong = [], []
    for seed in (50, 51):
        d = R.prompt_inputs(c, seed)
        run(c, d, plan)
        jobs.append((d, [x.clone() for x in d["o"] + d["lse"]]))

    def work(d, want):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(50):
                    for x in d["o"] + d["lse"]:
                        x.fill_(7.0)
                    plan.prompt_attention(d["q"], d["k"], d["v"], d["o"], d["starts"], lse=d["lse"])
                    s.synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(d["o"] + d["lse"], want)):
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


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 3)])
def test_what_other_rows_hold_does_not_matter(Hq, Hkv):
    """Rows of no sequence, and of a neighbour, may hold NaN and infinities."""
    c = R.Prompt("neighbours", (200, 300), (100, 90, 230), Hq, Hkv, 128, first=20) if Hkv % 2 == 0 else \
        R.Prompt("neighbours", (500,), (100, 90, 230), Hq, Hkv, 128, first=20)
    clean = R.prompt_inputs(c, 4)
    want, _, _, _ = R.prompt_reference(c, clean)
    run(c, clean)
    d = R.prompt_inputs(c, 4)
    flat = {n: torch.cat(d[n], 1) for n in "qkv"}
    for n, bad in zip("qkv", (float("nan"), float("inf"), float("nan"))):
        flat[n][:, :20] = bad
        flat[n][:, 120:210] = bad  # the middle sequence
        flat[n][:, 440:] = -bad
        d[n] = [x.contiguous() for x in flat[n].split(list(c.shards), 1)]
    run(c, d)
    a, b = (torch.cat(x["o"], 1)[0] for x in (clean, d))
    for lo, hi in ((0, 120), (210, 500)):
        assert torch.equal(a[lo:hi].view(torch.int16), b[lo:hi].view(torch.int16))


def test_the_same_bits_every_time_and_between_shard_counts():
    c = R.Prompt("again", (256,) * 4, (300, 256, 1, 467), 8, 4, 128)
    d = R.prompt_inputs(c, 5)
    plan = run(c, d)
    first = [x.clone() for x in d["o"]]
    for _ in range(5):
        run(c, d, plan)
        for x, y in zip(first, d["o"]):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_plain_attention_of_the_last_row():
    """A sequence's last row sees what the framework's attention without a mask sees."""
    c = R.Prompt("last", (300,), (300,), 4, 2, 128)
    d = R.prompt_inputs(c, 6)
    plan = run(c, d)
    o = [torch.empty_like(x) for x in d["q"]]
    plan.sp_attention(d["q"], d["k"], d["v"], o)
    torch.cuda.synchronize()
    diff = (o[0][0, -1].double() - d["o"][0][0, -1].double()).abs()
    # each is off by a rounding of the probabilities and one of the output
    assert float(diff.max()) <= 4 * 2.0 ** -8 * float(d["v"][0].abs().max())


@pytest.mark.parametrize("Hq", [64, 4])  # more items than two an SM, and so few that no workspace is needed
def test_streams_workspaces_and_graph(Hq):
    c = R.Prompt("graph", (500, 400), (123, 456, 200), Hq, 4 if Hq > 4 else 2, 128, first=30)
    d = R.prompt_inputs(c, 7)
    plan = run(c, d)  # outside a capture
    side = torch.cuda.Stream()
    # two calls at once on two streams, their workspaces their own
    e = R.prompt_inputs(c, 8)
    assert (plan.prompt_attention_workspace(3) > 0) == (Hq == 64)
    ws = [torch.empty(plan.prompt_attention_workspace(3), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        plan.prompt_attention(d["q"], d["k"], d["v"], d["o"], d["starts"], lse=d["lse"], workspace=ws[0])
        plan.prompt_attention(e["q"], e["k"], e["v"], e["o"], e["starts"], lse=e["lse"], workspace=ws[1], stream=side)
    torch.cuda.synchronize()
    R.check_prompt(c, d, d["o"], d["lse"])
    R.check_prompt(c, e, e["o"], e["lse"])
    # replayed with other sequences in the same tensor
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.prompt_attention(d["q"], d["k"], d["v"], d["o"], d["starts"], lse=d["lse"], workspace=ws[0])
    for seqs, first in (((1, 799, 2), 0), ((0, 300, 0), 128)):
        other = R.Prompt("other", c.shards, seqs, c.Hq, c.Hkv, c.D, first=first)
        for n in ("o", "lse"):
            for x in d[n]:
                x.fill_(7.0)
        d["starts"].copy_(torch.tensor(other.bounds, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        R.check_prompt(other, d, d["o"], d["lse"])


def test_sequence_bounds_are_clamped():
    c = R.Prompt("clamped", (200, 100), (300,), 4, 2, 64)
    d = R.prompt_inputs(c, 9)
    d["starts"] = torch.tensor([-5, 120, 1 << 30], dtype=torch.int32, device="cuda")
    run(c, d)
    as_is = R.Prompt("clamped", (200, 100), (120, 180), 4, 2, 64)
    R.check_prompt(as_is, d, d["o"], d["lse"])


def test_a_start_below_an_earlier_one_counts_as_that_one():
    c = R.Prompt("falling", (200, 100), (300,), 4, 2, 64)
    d = R.prompt_inputs(c, 11)
    d["starts"] = torch.tensor([10, 150, 50, 40, 290, 0, 7], dtype=torch.int32, device="cuda")
    run(c, d)
    as_is = R.Prompt("falling", (200, 100), (140, 0, 0, 140, 0, 0), 4, 2, 64, first=10)
    R.check_prompt(as_is, d, d["o"], d["lse"])
    # past a thousand sequences, too
    starts = [(i * 37) % 200 for i in range(2500)] + [250]
    d = R.prompt_inputs(c, 12)
    d["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    run(c, d)
    top = torch.tensor(starts).cummax(0).values.tolist()
    as_is = R.Prompt("falling", (200, 100), tuple(b - a for a, b in zip(top, top[1:])), 4, 2, 64, first=top[0])
    R.check_prompt(as_is, d, d["o"], d["lse"])


@pytest.mark.parametrize("fill", [0, 1, 3, 4])
def test_a_withheld_load_times_out_and_the_next_call_is_right(fill):
    from ulysses_sequence_attention_uly_gb300 import ULY_ERR_TIMEOUT
    c = R.Prompt("withheld", (700, 500), (900, 300), 4, 2, 128)
    d = R.prompt_inputs(c, 13)
    plan = R.plan_of(c)
    plan.set_wait_limit(20_000_000)
    plan.test_withhold_fill(fill)
    plan.prompt_attention(d["q"], d["k"], d["v"], d["o"], d["starts"], lse=d["lse"])
    assert plan.sync_status() == ULY_ERR_TIMEOUT
    plan.test_withhold_fill(-1)
    for n in ("o", "lse"):
        for x in d[n]:
            x.fill_(7.0)
    run(c, d, plan)
    R.check_prompt(c, d, d["o"], d["lse"])


def test_refusals():
    import ulysses_sequence_attention_uly_gb300 as uly
    c = R.Prompt("refused", (64, 64), (100,), 256, 2, 64)
    d = R.prompt_inputs(c, 10)
    plan = R.plan_of(c)
    ok = dict(q=d["q"], k=d["k"], v=d["v"], o=d["o"], seq_starts=d["starts"], lse=d["lse"])
    need = plan.prompt_attention_workspace(1)
    assert need > 0
    for change in (dict(q=d["q"][:1]), dict(k=d["q"]), dict(o=[x.float() for x in d["o"]]), dict(lse=d["lse"][:1]),
                   dict(seq_starts=d["starts"].long()), dict(seq_starts=d["starts"].cpu()), dict(seq_starts=[0, 1]),
                   dict(seq_starts=d["starts"][:0]), dict(v=[x.transpose(1, 2) for x in d["v"]]),
                   dict(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            plan.prompt_attention(**{**ok, **change})
    for change in (dict(o=d["q"]), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
                   dict(workspace=torch.empty(need + 256, dtype=torch.uint8, device="cuda")[1:])):
        with pytest.raises(uly.UlyError) as e:
            plan.prompt_attention(**{**ok, **change})
        assert e.value.status == uly.ULY_ERR_INVALID
    for other in (uly.Plan(2, 2, 64, 0, "none", 4, 2, 64), uly.Plan(1, 2, 64, 8, "prefix", 4, 2, 64)):
        q, k = ([torch.zeros((other.B, other.shard_rows(p, kv), h, 64), dtype=torch.bfloat16, device="cuda")
                 for p in range(2)] for kv, h in ((False, 4), (True, 2)))
        with pytest.raises(uly.UlyError) as e:
            other.prompt_attention(q, k, k, [torch.empty_like(x) for x in q], d["starts"])
        assert e.value.status == uly.ULY_ERR_UNSUPPORTED
    with pytest.raises(uly.UlyError) as e:
        uly.Plan(1, 2, 64, 0, "none", 4, 2, 128, dtype="e4m3").prompt_attention(**ok)
    assert e.value.status == uly.ULY_ERR_UNSUPPORTED
    plan.prompt_attention(**{**ok, "seq_starts": d["starts"][:1]})  # no sequence: nothing happens
    torch.cuda.synchronize()
    assert all((x == 7.0).all() for x in d["o"])


def test_the_wait_limit_is_a_waits_and_not_the_calls():
    """A call that takes longer than the limit in all (about 1.3 ms), no wait of it
    does (a CTA's item: at most 128 steps of 2 us)."""
    from ulysses_sequence_attention_uly_gb300 import Plan
    plan = Plan(1, 1, 16384, 0, "none", 32, 8, 128)
    q, k, v = (torch.randn((1, 16384, h, 128), device="cuda").to(torch.bfloat16) for h in (32, 8, 8))
    o, again = torch.empty_like(q), torch.empty_like(q)
    starts = torch.tensor([0, 16384], dtype=torch.int32, device="cuda")
    plan.prompt_attention([q], [k], [v], [o], starts)
    torch.cuda.synchronize()
    plan.set_wait_limit(700_000)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    plan.prompt_attention([q], [k], [v], [again], starts)
    b.record()
    assert plan.sync_status() == 0
    assert a.elapsed_time(b) > 0.7
    assert torch.equal(o.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("heads", [2, 400])  # items that CTAs find by themselves, and from the tables
@pytest.mark.parametrize("D", [64, 128])
def test_a_withheld_v_of_a_short_tile(heads, D):
    """V of a sequence's only tile, which is short, does not come: the warps that
    would zero its rows behind the end give up with their P just stored.  The call
    ends with a timeout, TMEM is free again, and the next calls are right."""
    from ulysses_sequence_attention_uly_gb300 import ULY_ERR_TIMEOUT
    c = R.Prompt("short v", (100,), (100,), heads, heads // 2, D)
    d = R.prompt_inputs(c, 14)
    plan = R.plan_of(c)
    for _ in range(3):
        plan.set_wait_limit(5_000_000)
        plan.test_withhold_fill(1)  # K of step 0 is copy 0, its V copy 1
        plan.prompt_attention(d["q"], d["k"], d["v"], d["o"], d["starts"], lse=d["lse"])
        assert plan.sync_status() == ULY_ERR_TIMEOUT
        plan.test_withhold_fill(-1)
        plan.set_wait_limit(4_000_000_000)
        run(c, d, plan)
        R.check_prompt(c, d, d["o"], d["lse"])


def test_a_wait_for_a_tile_of_the_other_warps_is_no_timeout():
    """One head of its own k and v and an odd number of tiles: a unit has a single
    tile, through which (2049 steps, 1.4 ms and more) the other four warps have
    nothing to do.  No wait of the roles at work comes near the limit."""
    from ulysses_sequence_attention_uly_gb300 import Plan
    n = 2049 * 128
    plan = Plan(1, 1, n, 0, "none", 1, 1, 64)
    q, k, v = (torch.randn((1, n, 1, 64), device="cuda").to(torch.bfloat16) for _ in range(3))
    o, again = torch.empty_like(q), torch.empty_like(q)
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    plan.prompt_attention([q], [k], [v], [o], starts)
    assert plan.sync_status() == 0
    plan.set_wait_limit(400_000)
    plan.prompt_attention([q], [k], [v], [again], starts)
    assert plan.sync_status() == 0
    assert torch.equal(o.view(torch.int16), again.view(torch.int16))
