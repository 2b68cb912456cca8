"""The 8-bit paged cache: rows into pages (uly_cache_append), attention of the
newest tokens over them (uly_cache_attention), and both together with the
prompt's attention, against 64 bits."""
import math

import pytest
import torch

from tests import _serve as R

pytestmark = pytest.mark.gpu

APPENDS = [
    R.Cached("one token", (0,), (1,), 1, 64, 16),
    R.Cached("tokens", (700, 64, 63, 5, 1023, 130, 127, 0), (1,) * 8, 4, 128, 64),
    R.Cached("page ends", (15, 16, 17, 0, 31), (1, 16, 15, 33, 2), 2, 64, 16),
    R.Cached("none of some", (9, 0, 40), (0, 0, 7), 3, 128, 32),
    R.Cached("prompts", (0, 5, 0), (700, 1, 333), 3, 128, 128),
    R.Cached("many rows", (0, 100, 7), (1500, 900, 31), 2, 64, 32),
    R.Cached("wide page", (100, 0), (200, 129), 2, 64, 128),
    R.Cached("small page", (3, 0), (50, 17), 2, 128, 16),
    # (few rows a sequence on average)
    R.Cached("a long one among tokens", (5,) * 12 + (3,), (1,) * 12 + (75,), 5, 128, 64),
    R.Cached("long ones among tokens", (0, 100) + (126, 127, 0) * 10, (90, 30) + (1, 2, 3) * 10, 3, 64, 128),
]


def same_codes(got, want, what):
    got = got.to(torch.float64).cpu()
    assert torch.equal(got.isnan(), want.isnan()), what + ": NaN codes"
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0)), "%s: %d codes differ" % (
        what, int((got.nan_to_num(0.0) != want.nan_to_num(0.0)).sum()))


def check_append(c, d, call=None):
    want = R.appended(c, d)
    (call or (lambda: R.cache_of(d).append(d["k"], d["v"], d["starts"], d["lens"], d["table"])))()
    torch.cuda.synchronize()
    for t in "kv":
        assert torch.equal(d[t + "_scale"].double().cpu(), want[t + "_scale"]), t + "_scale"
        same_codes(d[t + "_pages"], want[t + "_pages"], t)


@pytest.mark.parametrize("c", APPENDS, ids=lambda c: c.name)
@pytest.mark.parametrize("big", [0.01, 1.0, 300.0])
def test_append(c, big):
    """Codes and scales to the bit; small and large new values against the pages'
    older scales (kept, or raised with the older codes brought along)."""
    d = R.cache_inputs(c, 1)
    for t in "kv":
        d[t] = (d[t].float() * big).to(torch.bfloat16)
    check_append(c, d)


@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 64)])
def test_append_a_token_that_raises_every_scale(D, page):
    """A token to every sequence, larger than all before it, again and again: the
    page's scale is read by all lanes of a warp and written by one, and the older
    codes are brought along each time."""
    n, old = 60, page // 2
    c = R.Cached("raised", (old,) * n, (1,) * n, 7, D, page)
    d = R.cache_inputs(c, 9)
    lens = list(c.lens)
    for step in range(8):
        before = {t: d[t + "_scale"].clone() for t in "kv"}
        for t in "kv":
            d[t] = (torch.randn((n, 7, D), device="cuda").clamp(-4, 4) + 20).to(torch.bfloat16) * 4.0 ** step
        d["lens"] = R.ints([x + step for x in lens])
        check_append(c, d)
        pages = d["table"][:, 0].long()
        for t in "kv":
            assert (d[t + "_scale"][pages] > before[t][pages]).all() or step == 0


def test_append_from_a_packed_projection():
    c = R.Cached("packed", (17, 0, 250, 16), (3, 40, 1, 16), 3, 64, 16)
    d = R.cache_inputs(c, 2)
    qkv = torch.randn((c.rows, 3 * c.H, c.D), device="cuda").to(torch.bfloat16)
    d["k"], d["v"] = qkv[:, c.H:2 * c.H], qkv[:, 2 * c.H:]
    check_append(c, d)


def test_append_extreme_values():
    c = R.Cached("extreme", (0, 20, 0, 3), (40, 5, 16, 2), 2, 64, 16)
    d = R.cache_inputs(c, 3)
    for t in "kv":
        x = d[t]
        x[:16] = 0.0                                   # a page of zeros: the least scale
        x[16:32] *= 1e-30                              # below it
        x[32:40] = 3e38
        x[3, 1] = float("nan")                         # stays in its page, head and row
        x[45, 0, 5] = float("nan")
        x[46:62, 1] = 448.0 * 2.0 ** -4                # exactly a power's largest value
        x[46, 0, 0] = -448.0 * 2.0 ** 5
    check_append(c, d)


def test_append_an_infinity_takes_its_page_and_head_alone():
    c = R.Cached("infinity", (0, 0), (20, 16), 2, 64, 16)
    d = R.cache_inputs(c, 4)
    d["k"][18, 1, 3] = float("inf")
    R.cache_of(d).append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    torch.cuda.synchronize()
    page = int(d["table"][0, 1])
    assert float(d["k_scale"][page, 1]) == 2.0 ** 120 and float(d["k_pages"][page, 1, 2, 3].float()) == 448.0
    other = R.cache_inputs(c, 4)
    R.cache_of(other).append(other["k"], other["v"], other["starts"], other["lens"], other["table"])
    for t in "kv":
        a, b = (x[t + "_pages"].view(torch.uint8).clone() for x in (d, other))
        if t == "k":
            a[page, 1], b[page, 1] = 0, 0
        assert torch.equal(a, b)


def test_append_shard_by_shard():
    """The rows of sequences that lie across shards, a call for each shard in order:
    its starts clamped to its rows, the lengths those up to its end.  Pages that a
    shard's end cuts are taken up again, also where the later rows raise their scale."""
    shards, first, old, new = (70, 1, 129, 100), 9, (20, 0, 5, 33), (40, 130, 0, 111)
    c = R.Cached("shards", old, new, 2, 64, 32)
    d = R.cache_inputs(c, 28)
    rows = sum(shards)
    assert first + c.rows <= rows
    at = [first]
    for n in new:
        at.append(at[-1] + n)
    whole = {t: (torch.randn((rows, 2, 64), device="cuda") * torch.arange(1, rows + 1, device="cuda")[:, None, None])
             .to(torch.bfloat16) for t in "kv"}  # (larger and larger: every cut page's scale is raised)
    lo, cache = 0, R.cache_of(d)
    for n in shards:
        part = R.Cached("shard", old, new, 2, 64, 32)
        x = {**d, "k": whole["k"][lo:lo + n], "v": whole["v"][lo:lo + n],
             "starts": R.ints([min(max(a - lo, 0), n) for a in at]),
             "lens": R.ints([o + min(max(lo + n - a, 0), m) for o, a, m in zip(old, at, new)])}
        check_append(part, x, lambda: cache.append(x["k"], x["v"], x["starts"], x["lens"], x["table"]))
        lo += n
    for s, (a, m) in enumerate(zip(at, new)):  # every row is there
        for i in range(m):
            pos = old[s] + i
            page, slot = int(d["table"][s, pos // 32]), pos % 32
            for t in "kv":
                scale = d[t + "_scale"][page].double()[:, None]
                was, got = whole[t][a + i].double(), d[t + "_pages"][page, :, slot].double() * scale
                # rounded once for its call's scale and, where that is subnormal in a later one, once more
                assert ((got - was).abs() <= 2.0 ** -4 * was.abs() + 2.0 ** -9 * scale).all()


def test_append_drops_rows_without_a_place():
    """Positions below zero or past the table, bad pages: nothing else is written."""
    c = R.Cached("dropped", (10, 0, 40), (20, 5, 30), 2, 64, 16)
    d = R.cache_inputs(c, 5)
    d["lens"] = R.ints([13, 5, 16 * d["table"].shape[1] + 3])      # seven rows below zero; three past the end
    d["table"][2] = torch.randperm(d["table"].shape[1], device="cuda").int() + 1  # all entries real,
    d["table"][2, -2] = -3                                          # but one
    d["table"][0], d["table"][1] = 0, -1
    check_append(c, d)


def test_append_scales_that_are_no_powers():
    """Pages that another program filled: the scale is kept, or raised to a power;
    older codes within a rounding of it."""
    c = R.Cached("foreign", (7, 20), (2, 3), 2, 64, 16)
    d = R.cache_inputs(c, 6, powers=False)
    had = {t: d[t + "_scale"].clone() for t in "kv"}
    was = {t: d[t + "_pages"].double() * had[t].double()[..., None, None] for t in "kv"}
    for t in "kv":
        d[t] = (d[t].float() * 20).to(torch.bfloat16)
    R.cache_of(d).append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    torch.cuda.synchronize()
    for t in "kv":
        now = d[t + "_scale"].double()[..., None, None]
        got = d[t + "_pages"].double() * now
        for s in range(2):
            at, slot = int(d["table"][s, c.old[s] // 16]), c.old[s] % 16
            assert (now[at].flatten() >= had[t][at].double()).all()
            x, y = got[at, :, :slot], was[t][at, :, :slot]
            # half a step of e4m3, 2^-4 of the value or 2^-10 of the scale, and the f32 factor
            assert ((x - y).abs() <= (2.0 ** -4 + 1e-6) * y.abs() + 2.0 ** -10 * now[at]).all()


ATTENTION = [
    R.Cached("one key", (0,), (1,), 1, 64, 16),
    R.Cached("few keys", (4,), (1,), 2, 128, 16, G=4),
    R.Cached("lengths", (0, 1, 14, 15, 16, 17, 62, 63, 64, 65, 127, 128, 300), (1,) * 13, 2, 128, 64, G=4),
    R.Cached("small pages", (0, 1, 14, 15, 16, 17, 31, 32, 200), (1,) * 9, 3, 64, 16, G=3),
    R.Cached("wide pages", (5, 127, 128, 400, 900), (1,) * 5, 1, 64, 128, G=8),
    R.Cached("single heads", (77, 500, 3), (1,) * 3, 6, 128, 32),
    R.Cached("guesses", (0, 1, 15, 300, 777), (3, 3, 1, 3, 5), 2, 128, 32, G=4),
    R.Cached("no new token", (40, 0, 9, 70), (0, 0, 2, 0), 2, 64, 16, G=2),
    R.Cached("end of a prompt", (100, 0, 30), (40, 33, 1), 2, 128, 64, G=2),
    R.Cached("large group", (50, 333), (1, 2), 1, 128, 64, G=12),
    R.Cached("larger group", (50, 333), (2, 1), 2, 64, 32, G=20),
    R.Cached("long", (20000,), (1,), 2, 128, 64, G=4, std=0.7),
    R.Cached("long and short", (9000, 3, 70, 2500), (1, 2, 1, 1), 2, 64, 128, G=2),
    R.Cached("many", tuple((i * 37) % 150 for i in range(300)), tuple(i % 3 for i in range(300)), 1, 64, 16, G=2),
    R.Cached("many, some long", tuple(2500 if i % 70 == 3 else (i * 37) % 150 for i in range(200)),
             tuple(i % 3 for i in range(200)), 2, 64, 32, G=2),
    R.Cached("one long among many", (12, 9, 130) * 16 + (20000, 3), (1,) * 50, 2, 64, 64, G=2),
    R.Cached("two long among many, wide", (12, 9, 130) * 16 + (5000, 7000), (1,) * 48 + (3, 5), 2, 128, 128, G=4),
    R.Cached("peaked", (700,), (2,), 2, 128, 64, G=4, std=6.0),
]


@pytest.mark.parametrize("c", ATTENTION, ids=lambda c: c.name)
def test_attention_against_64_bits(c):
    d = R.cache_inputs(c, 11)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    o, lse = R.attend(cache, c, d)
    torch.cuda.synchronize()
    R.check_cached(c, d, o, lse)


def _ragged(n, lo, hi):
    """n lengths between lo and hi, even over the logarithm, in no order."""
    return tuple(int(lo * (hi / lo) ** ((i * 37 % n) / (n - 1))) for i in range(n))


# so many long units that their parts are half as long as what a CTA's share would be
FULL = [
    R.Cached("batch", _ragged(64, 400, 12000), (1,) * 64, 8, 128, 64, G=4),
    R.Cached("batch, 64 wide", _ragged(64, 1000, 16000), (1,) * 64, 8, 64, 32, G=4),
    R.Cached("more sequences than a CTA has threads", _ragged(200, 100, 6000), (1,) * 200, 8, 128, 128, G=2),
    R.Cached("two tiles of queries", _ragged(64, 400, 9000), (3,) * 64, 8, 128, 64, G=4, std=0.7),
    R.Cached("three tiles, 64 wide", _ragged(64, 400, 9000), (9,) * 40 + (0, 11) * 12, 8, 64, 16, G=4),
    R.Cached("more sequences, two tiles, 64 wide", _ragged(150, 300, 6000), (4, 2, 5) * 50, 8, 64, 64, G=3),
]


@pytest.mark.parametrize("c", FULL, ids=lambda c: c.name)
def test_attention_full_batches(c):
    # the case does reach that way: blocks of 64 keys, and what a CTA slot has of them (320 KB of codes and more)
    tiles = 2 if c.rows * c.G > 8 * len(c.new) else 1
    slots = min(torch.cuda.get_device_properties(0).multi_processor_count, 160) * (4, 3)[tiles - 1]
    blocks = sum(-(-t * c.G // (8 * tiles)) * -(-n // 64) for n, t in zip(c.lens, c.new)) * c.H
    assert blocks > slots * ((320 << 10) // (64 * 2 * c.D))
    assert max(c.lens) > 1024 and len(c.lens) * c.H * 8 > slots  # neither whole units nor few of them
    d = R.cache_inputs(c, 26)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    o, lse = R.attend(cache, c, d)
    torch.cuda.synchronize()
    R.check_cached(c, d, o, lse)


@pytest.mark.parametrize("c", ATTENTION[2:9:3], ids=lambda c: c.name)
def test_attention_other_scales(c):
    """Scales of any value, far apart between pages, and another softmax scale."""
    d = R.cache_inputs(c, 12, powers=False)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    d["v_scale"] *= torch.exp2(torch.randint(-5, 6, d["v_scale"].shape, device="cuda").float())
    o, lse = R.attend(cache, c, d, scale=0.05)
    torch.cuda.synchronize()
    R.check_cached(c, d, o, lse, scale=0.05)


@pytest.mark.parametrize("D,T", [(64, 1), (128, 1), (128, 5)])  # (five tokens of two heads: two tiles of queries)
def test_attention_a_page_of_a_far_larger_scale(D, T):
    """The first page's v scale 2^20 times the others', its codes zero in every second
    element (a warp has 16 of every 64 keys, so that all of them see it first):
    there the output is made of weights 2^-20 of the largest, which f16 has to hold
    to 2^-11.  The reference exponent leaves seven binary orders above the largest
    weight, so that half a step of the smallest is 2^-32 of it."""
    c = R.Cached("far", (100,), (T,), 2, D, 64, G=2, std=0.3)
    d = R.cache_inputs(c, 23)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    page = int(d["table"][0, 0])
    d["v_scale"].fill_(1.0)
    d["v_scale"][page] = 2.0 ** 20
    d["v_pages"].view(torch.uint8)[page, :, :, ::2] = 0
    o, lse = R.attend(cache, c, d)
    torch.cuda.synchronize()
    want, wl, _, _ = R.cached_reference(c, d)
    n, page = c.lens[0], c.page
    at = d["table"][0, torch.arange(n, device="cuda") // page].long()
    k, v = (d[t + "_pages"].double()[at, :, torch.arange(n, device="cuda") % page].repeat_interleave(2, 1) for t in "kv")
    ks, vs = (d[t + "_scale"].double()[at].repeat_interleave(2, 1) for t in "kv")  # [keys, heads]
    z = torch.einsum("ihd,jhd->ihj", d["q"].double(), k * ks[..., None]) / math.sqrt(D)
    ok = torch.arange(n, device="cuda") <= n - T + torch.arange(T, device="cuda")[:, None]
    w = z.masked_fill(~ok[:, None], -math.inf).softmax(-1) * vs.T  # weights of the codes
    # an f16 rounding of each weight (2^-11, or 2^-32 of the largest), 32-bit sums, and bf16 once
    err = torch.einsum("ihj,jhd->ihd", w * (2.0 ** -11 + 2.0 ** -13) + 2.0 ** -32 * w.amax(-1, keepdim=True) * ok[:, None],
                       v.abs())
    R.check_rows(o, want, err * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 1e-30, "o")
    R.check_rows(lse, wl, 2.0 ** -13 + 2.0 ** -22 * wl.abs(), "lse")


@pytest.mark.parametrize("e", [-60, -20, 60, 100])
def test_attention_scales_at_their_ends(e):
    """All of v's scales at an end of their range, and one page at the least one."""
    c = R.Cached("ends", (200, 90), (1, 2), 2, 128, 16, G=4)
    d = R.cache_inputs(c, 13)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    d["v_scale"].fill_(2.0 ** e)
    for lone in (False, True):
        if lone:
            d["v_scale"][int(d["table"][0, 3])] = 2.0 ** -60
        o, lse = R.attend(cache, c, d)
        torch.cuda.synchronize()
        R.check_cached(c, d, o, lse)


def test_large_and_small_queries():
    """q of any magnitude: a power of two is taken out of each row."""
    c = R.Cached("magnitudes", (200,), (4,), 2, 64, 32, G=2)
    d = R.cache_inputs(c, 14)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    q = d["q"]
    q[0] *= 2.0 ** 20
    q[1] *= 2.0 ** -100
    q[2] = 0.0
    q[3, :, 1:] *= 2.0 ** -12
    for scale, rows in ((2.0 ** -23, [0]), (2.0 ** 97, [1]), (0.125, [2, 3])):
        o, lse = R.attend(cache, c, d, scale=scale)
        torch.cuda.synchronize()
        want, wl, err, _ = R.cached_reference(c, d, scale)
        R.check_rows(o[rows], want[rows], err[rows], "o")
        R.check_rows(lse[rows], wl[rows], 2.0 ** -13 + 2.0 ** -22 * wl[rows].abs(), "lse")


@pytest.mark.parametrize("D,T", [(64, 1), (128, 5)])
def test_one_large_element_of_q(D, T):
    """An element of q 2^20 times the others meets codes of zero: the scores are made
    of the small ones, which f16 holds exactly down to 2^-31 of the largest.  (The
    bound: q, 8 bits wide, is exact, so that the reference's stands as it is.)"""
    c = R.Cached("outlier", (200,), (T,), 2, D, 32, G=2)
    d = R.cache_inputs(c, 24)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    d["k_pages"].view(torch.uint8)[..., 5] = 0
    d["q"][..., 5] = 2.0 ** 20
    o, lse = R.attend(cache, c, d, scale=0.125)
    torch.cuda.synchronize()
    R.check_cached(c, d, o, lse, scale=0.125)


@pytest.mark.parametrize("e", [127, 126, -112, -120, -126])
def test_queries_at_the_ends_of_bf16(e):
    """Largest elements of q at both ends of bf16's exponents."""
    c = R.Cached("ends of q", (60,), (2,), 1, 64, 32, G=2)
    d = R.cache_inputs(c, 25)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    d["k_scale"].fill_(2.0 ** -20 if e > 0 else 2.0 ** 30)
    d["q"].clamp_(-1.99, 1.99)
    d["q"][..., 0] = 1.9921875
    d["q"] = (d["q"].float() * 2.0 ** e).to(torch.bfloat16)
    assert torch.isfinite(d["q"]).all()
    scale = 2.0 ** (20 - e - 9) if e > 0 else 2.0 ** (-e - 30 - 9)  # scores of about one
    o, lse = R.attend(cache, c, d, scale=scale)
    torch.cuda.synchronize()
    R.check_cached(c, d, o, lse, scale=scale)


def test_bad_pages_and_lengths():
    """Tokens in bad pages take no part; a length past the table ends with it; a
    row before the first position has no key."""
    c = R.Cached("bad", (60, 100, 5, 200, 0), (2, 1, 1, 3, 4), 2, 128, 16, G=4)
    d = R.cache_inputs(c, 15)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    n = d["k_pages"].shape[0]
    d["table"][0, 1] = -1
    d["table"][1, 0], d["table"][1, 6] = n, 2 ** 31 - 1
    d["table"][2, 0] = -2 ** 31
    d["table"][3, -1] = d["table"][3, 0]
    d["lens"] = R.ints([62, 101, 6, 16 * d["table"].shape[1] + 40, 2])
    d["table"][4, 0] = d["table"][0, 0]
    for t in "kv":  # (slots behind the last tokens become tokens)
        d[t + "_pages"].view(torch.uint8)[d[t + "_pages"].view(torch.uint8) == 0x7F] = 0x31
    o, lse = R.attend(cache, c, d)
    torch.cuda.synchronize()
    R.check_cached(c, d, o, lse)
    d["lens"] = R.ints([0, -7, 0, -2 ** 31, 1])
    o, lse = R.attend(cache, c, d)
    torch.cuda.synchronize()
    R.check_cached(c, d, o, lse)


def test_rows_of_no_sequence_stay_and_starts_are_clamped():
    c = R.Cached("stay", (60, 30), (3, 2), 2, 64, 16, G=2)
    d = R.cache_inputs(c, 16)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    for starts in ([1, 3, 4], [-4, 2, 1 << 30], [5, 5, 5]):
        d["starts"] = R.ints(starts)
        o, lse = R.attend(cache, c, d)
        torch.cuda.synchronize()
        d["starts"] = d["starts"].clamp(0, 5)
        R.check_cached(c, d, o, lse)


@pytest.mark.parametrize("width", [2, 70])  # units whole, and in parts that the table's width asks for
def test_the_most_sequences(width):
    """65536 sequences of 20 tokens, one of them new, against 64 bits in one piece."""
    import ulysses_sequence_attention_uly_gb300 as uly
    n, D, page, L = 65536, 64, 16, 20
    g = torch.Generator(device="cuda").manual_seed(27)
    x = {t: torch.zeros((2 * n, 1, page, D), dtype=torch.float8_e4m3fn, device="cuda") for t in ("k_pages", "v_pages")}
    x |= {t: torch.zeros((2 * n, 1), device="cuda") for t in ("k_scale", "v_scale")}
    cache = R.cache_of(x)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[:, :2] = torch.randperm(2 * n, generator=g, device="cuda").int().view(n, 2)
    k, v = (torch.randn((n, L, 1, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for a, b in ((0, L - 1), (L - 1, L)):  # the first tokens, then the newest one
        cache.append(k[:, a:b].reshape(-1, 1, D), v[:, a:b].reshape(-1, 1, D),
                     torch.arange(0, n * (b - a) + 1, b - a, dtype=torch.int32, device="cuda"),
                     torch.full((n,), b, dtype=torch.int32, device="cuda"), table)
    kk, vv = ((x[t + "_pages"].double() * x[t + "_scale"].double()[..., None, None])[table[:, :2].long()]
              .reshape(n, 2 * page, D)[:, :L] for t in "kv")
    for got, was in ((kk, k), (vv, v)):  # what the cache holds: within an e4m3 rounding of what came
        was = was[:, :, 0].double()
        # a scale s is at most twice top / 448, half a step of the smallest codes 2^-10 s: 2^-9 top / 448 for a
        # page that was written once.  The second page's first tokens were rounded for a scale s' <= s / 2 before
        # they came to s: small ones by 2^-10 s' + 2^-10 s at most, which is 1.5 times that
        top = was.abs().amax((1, 2))[:, None, None] / 448
        off = (got - was).abs() - 2.0 ** -4 * was.abs()
        assert (off[:, :page] <= 2.0 ** -9 * top).all() and (off[:, page:] <= 1.5 * 2.0 ** -9 * top).all()
    q = torch.randn((n, 2, D), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = torch.full_like(q, 7.0), torch.full((n, 2), 7.0, device="cuda")
    starts, lens = torch.arange(n + 1, dtype=torch.int32, device="cuda"), torch.full((n,), L, dtype=torch.int32, device="cuda")
    cache.attention(q, o, starts, lens, table, scale=0.125, lse=lse)
    torch.cuda.synchronize()
    s = torch.einsum("nhd,njd->nhj", q.double(), kk) * 0.125
    p = s.softmax(-1)
    want = torch.einsum("nhj,njd->nhd", p, vv)
    err = torch.einsum("nhj,njd->nhd", p, vv.abs()) * (2.0 ** -11 + 2.0 ** -13) + 2.0 ** -8 * want.abs()
    # (weights below f16's normal range: 2^-32 of the largest, for values of 448 scales at most)
    err = err * (1 + 2.0 ** -8) + L * 2.0 ** -32 * 448 * x["v_scale"].amax().double() + 1e-30
    R.check_rows(o, want, err, "o")
    R.check_rows(lse, s.logsumexp(-1), 2.0 ** -13 + 2.0 ** -22 * s.logsumexp(-1).abs(), "lse")
    with pytest.raises(uly.UlyError) as e:
        cache.attention(q, o, R.ints([0] * (n + 2)), R.ints([0] * (n + 1)), torch.zeros((n + 1, 1), dtype=torch.int32,
                                                                                      device="cuda"))
    assert e.value.status == uly.ULY_ERR_UNSUPPORTED


@pytest.mark.parametrize("seqs", [100, 150])
def test_starts_that_fall(seqs):
    """Rows that two sequences claim may get anything, but the call ends, writes to
    no other row and leaves the next one right."""
    c = R.Cached("falling", (3000,) * seqs, (1,) * seqs, 2, 64, 64, G=4)
    d = R.cache_inputs(c, 18)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    right = d["starts"]
    d["starts"] = R.ints([2, c.rows - 2] * (seqs // 2) + [2])
    o, lse = R.attend(cache, c, d)
    torch.cuda.synchronize()
    for got in (o, lse):
        assert (got[:2] == 7.0).all() and (got[-2:] == 7.0).all()
    d["starts"] = right
    o, lse = R.attend(cache, c, d)
    torch.cuda.synchronize()
    R.check_cached(c, d, o, lse)


def test_strided_queries_and_no_lse():
    c = R.Cached("strided", (60, 300), (3, 2), 2, 128, 32, G=3)
    d = R.cache_inputs(c, 17)
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    wide = torch.full((c.rows, 10, c.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8] = d["q"]
    d["q"] = wide[:, 2:8]
    o = torch.full((c.rows, 6, c.D), 7.0, dtype=torch.bfloat16, device="cuda")
    cache.attention(d["q"], o, d["starts"], d["lens"], d["table"])
    torch.cuda.synchronize()
    R.check_cached(c, d, o, None)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: pages at its end."""
    n, H, page, D = 70000, 4, 128, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    d = {t: torch.zeros((n, H, page, D), dtype=torch.uint8, device="cuda") for t in ("k_pages", "v_pages")}
    c = R.Cached("far", (100, 300), (2, 150), H, D, page, G=2)
    for t in "kv":
        d[t + "_scale"] = torch.ones((n, H), device="cuda")
        d[t] = torch.randn((c.rows, H, D), device="cuda").to(torch.bfloat16)
    d["q"] = torch.randn((c.rows, H * 2, D), device="cuda").to(torch.bfloat16)
    d["starts"], d["lens"] = R.starts_of(c.new), R.ints(c.lens)
    d["table"] = R.ints([[n - 1, 65600, 3, 3], [n - 2, 69990, 65537, n - 7]])
    cache = R.cache_of(d)
    cache.append(d["k"], d["v"], d["starts"], d["lens"], d["table"])
    o, lse = R.attend(cache, c, d)
    torch.cuda.synchronize()
    pages = d["table"].flatten().unique().long()
    small = {t: d[t][pages] for t in ("k_scale", "v_scale")}
    small |= {t: d[t][pages].view(torch.float8_e4m3fn) for t in ("k_pages", "v_pages")}
    small["table"] = torch.searchsorted(pages, d["table"].long()).int()
    R.check_cached(c, {**d, **small}, o, lse)


def test_the_same_bits_every_time_streams_and_graph():
    c = R.Cached("again", (3000, 20, 700, 0), (1, 3, 1, 2), 2, 128, 64, G=4)
    d, e = R.cache_inputs(c, 18), R.cache_inputs(c, 19)
    for x in (d, e):
        R.cache_of(x).append(x["k"], x["v"], x["starts"], x["lens"], x["table"])
    first, _ = R.attend(R.cache_of(d), c, d)
    cache, other, side = R.cache_of(d), R.cache_of(e), torch.cuda.Stream()
    o, p = torch.empty_like(first), torch.empty_like(first)
    torch.cuda.synchronize()
    for _ in range(10):
        cache.attention(d["q"], o, d["starts"], d["lens"], d["table"])
        other.attention(e["q"], p, e["starts"], e["lens"], e["table"], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), first.view(torch.int16))
    R.check_cached(c, e, p, None)
    # two graphs that share a workspace, replayed one after the other, with lengths that change
    ws = torch.empty(cache.attention_workspace(8, c.rows, 4, d["table"].shape[1]), dtype=torch.uint8, device="cuda")
    graphs = []
    for x, y in ((d, o), (e, p)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ca = R.cache_of(x)
            ca.append(x["k"], x["v"], x["starts"], x["lens"], x["table"])
            ca.attention(x["q"], y, x["starts"], x["lens"], x["table"], workspace=ws)
        graphs.append(g)
    for lens in ((2990, 23, 701, 2), (1, 3, 64, 2), (2049, 16, 1, 2)):
        for x, y, g in ((d, o, graphs[0]), (e, p, graphs[1])):
            x["lens"].copy_(R.ints(lens))
            fresh = {n: t.clone() for n, t in x.items()}
            g.replay()
            torch.cuda.synchronize()
            want = R.appended(c, fresh)
            for t in "kv":
                same_codes(x[t + "_pages"], want[t + "_pages"], t)
            R.check_cached(c, x, y, None)


@pytest.mark.parametrize("old", [(3000, 20, 700, 0), (300, 20, 70, 0)])  # in parts, and whole without a workspace
def test_two_threads(old):
    """Appends and attention from two threads at once, each with a stream and a cache
    of its own: the bits of calls alone."""
    import threading
    c = R.Cached("threads", old, (1, 3, 1, 2), 2, 128, 64, G=4)
    jobs, wrong = [], []

    def step(x):
        o, lse = torch.full_like(x["q"], 7.0), torch.full(x["q"].shape[:2], 7.0, device="cuda")
        cache = R.cache_of(x)
        cache.append(x["k"], x["v"], x["starts"], x["lens"], x["table"])
        cache.attention(x["q"], o, x["starts"], x["lens"], x["table"], lse=lse)
        return [o, lse] + [x[n].view(torch.uint8) for n in ("k_pages", "v_pages")]

    for seed in (60, 61):
        x = R.cache_inputs(c, seed)
        jobs.append((x, [t.clone() for t in step(x)]))
    torch.cuda.synchronize()

    def work(x, want):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(50):
                    got = step(x)  # (the same rows again: the same codes)
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        wrong.append("other bits")
        except Exception as e:  # noqa: BLE001 - reported below
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]


def test_prompt_cache_and_generation_together():
    """Prompts through the causal attention and into the cache, then tokens one by
    one (and three at once): each step's output against attention over all keys
    as the cache holds them; the first step's against the prompt's own, whose
    keys and values are not quantised."""
    lens, H, G, D, page = [130, 1, 65], 2, 2, 128, 32
    c = R.Prompt("prompt", (100, 96), tuple(lens), H * G, H, D)
    d = R.prompt_inputs(c, 20)
    plan = R.plan_of(c)
    plan.prompt_attention(d["q"], d["k"], d["v"], d["o"], d["starts"], lse=d["lse"])
    n_pages = 40
    x = {t: torch.zeros((n_pages, H, page, D), dtype=torch.float8_e4m3fn, device="cuda") for t in ("k_pages", "v_pages")}
    x |= {t: torch.zeros((n_pages, H), device="cuda") for t in ("k_scale", "v_scale")}
    x["table"] = torch.randperm(n_pages, device="cuda").int()[:36].view(3, 12).contiguous()
    cache = R.cache_of(x)
    x["lens"], x["starts"] = R.ints(lens), d["starts"]
    for t in "kv":
        x[t] = torch.cat(d[t], 1)[0]
    cache.append(x["k"], x["v"], x["starts"], x["lens"], x["table"])
    # the prompts' rows over the cache: off by the 8-bit rounding, 2^-4 of v in the output and, with scores of
    # about one, 2^-4 of the weights through k
    x["q"] = torch.cat(d["q"], 1)[0]
    whole = R.Cached("whole", (0, 0, 0), tuple(lens), H, D, page, G=G)
    o, lse = R.attend(cache, whole, x)
    torch.cuda.synchronize()
    R.check_cached(whole, x, o, lse)
    exact = torch.cat(d["o"], 1)[0].double()
    assert float((o.double() - exact).norm() / exact.norm()) < 2.0 ** -3
    R.check_prompt(c, d, d["o"], d["lse"])
    g = torch.Generator(device="cuda").manual_seed(21)
    for new in ((1, 1, 1),) * 3 + ((3, 0, 1), (1, 1, 1)):
        lens = [a + n for a, n in zip(lens, new)]
        step = R.Cached("step", (0, 0, 0), new, H, D, page, G=G)
        x["lens"], x["starts"] = R.ints(lens), R.starts_of(new)
        for t, h in (("q", H * G), ("k", H), ("v", H)):
            x[t] = (torch.randn((sum(new), h, D), generator=g, device="cuda") * 2).to(torch.bfloat16)
        cache.append(x["k"], x["v"], x["starts"], x["lens"], x["table"])
        o, lse = R.attend(cache, step, x)
        torch.cuda.synchronize()
        R.check_cached(step, x, o, lse)
        # the newest keys as the cache holds them
        s = 2
        at, slot = int(x["table"][s, (lens[s] - 1) // page]), (lens[s] - 1) % page
        for t in "kv":
            scale = x[t + "_scale"][at].double()[:, None]
            got = x[t + "_pages"][at, :, slot].double() * scale
            was = x[t][-1].double()
            assert ((got - was).abs() <= 2.0 ** -4 * was.abs() + 2.0 ** -10 * scale).all()


def test_refusals():
    import ulysses_sequence_attention_uly_gb300 as uly
    c = R.Cached("refused", (1030, 3), (2, 1), 2, 64, 16, G=2)
    d = R.cache_inputs(c, 22)
    cache = R.cache_of(d)
    o = torch.empty_like(d["q"])
    a = dict(k=d["k"], v=d["v"], starts=d["starts"], lens=d["lens"], table=d["table"])
    b = dict(q=d["q"], o=o, starts=d["starts"], lens=d["lens"], table=d["table"])
    for change in (dict(k=d["k"].float()), dict(k=d["k"][:, :1]), dict(v=d["v"][:2]), dict(k=d["k"].cpu()),
                   dict(starts=d["starts"].long()), dict(lens=d["lens"][:1]), dict(table=d["table"][:1]),
                   dict(table=d["table"].t()), dict(table=None), dict(lens=None), dict(starts=3),
                   dict(k=torch.zeros((3, 2, 70), dtype=torch.bfloat16, device="cuda")[:, :, :64]),
                   dict(k=torch.zeros((3 * 132,), dtype=torch.bfloat16, device="cuda").as_strided((3, 2, 64), (132, 64, 1)))):
        with pytest.raises(ValueError):
            cache.append(**{**a, **change})
    need = cache.attention_workspace(4, 3, 2, d["table"].shape[1])
    assert need > 0
    for change in (dict(q=d["q"][:, :3]), dict(o=o[:2]), dict(o=o.float()), dict(lse=torch.zeros((3, 3), device="cuda")),
                   dict(q=d["q"][0]), dict(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            cache.attention(**{**b, **change})
    for change in (dict(o=d["q"]), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
                   dict(workspace=torch.empty(need + 256, dtype=torch.uint8, device="cuda")[1:])):
        with pytest.raises(uly.UlyError) as e:
            cache.attention(**{**b, **change})
        assert e.value.status == uly.ULY_ERR_INVALID
    for shape in ((4, 2, 24, 64), (4, 2, 16, 96), (4, 2, 8, 128)):
        p = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        s = torch.ones(shape[:2], device="cuda")
        x = torch.zeros((3, 2, shape[3]), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(uly.UlyError) as e:
            uly.Cache(p, p.clone(), s, s.clone()).append(x, x, d["starts"], d["lens"], d["table"])
        assert e.value.status == uly.ULY_ERR_UNSUPPORTED
    with pytest.raises(uly.UlyError) as e:  # one pool for both
        uly.Cache(d["k_pages"], d["k_pages"], d["k_scale"], d["v_scale"]).append(**a)
    assert e.value.status == uly.ULY_ERR_INVALID
    for bad in (dict(k_pages=d["k_pages"].float()), dict(v_pages=d["v_pages"][:1]), dict(k_scale=d["k_scale"].half()),
                dict(v_scale=d["v_scale"][:, :1]), dict(k_pages=d["k_pages"].cpu())):
        with pytest.raises(ValueError):
            uly.Cache(**{**{n: d[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")}, **bad})
    # nothing to do
    cache.append(d["k"][:0], d["v"][:0], R.ints([0]), R.ints([]), d["table"][:0])
    cache.attention(d["q"][:0], o[:0], R.ints([0]), R.ints([]), d["table"][:0])
