"""The prompt and cache calls on the CPU: refusals that need no GPU, and the
64-bit references of the GPU tests against direct sums."""
import ctypes
import math

import pytest
import torch

import ulysses_sequence_attention_uly_gb300 as uly
from tests import _serve as R

A = 1 << 24  # an address that is never followed: every call below returns before it would be


def cache(**change):
    d = dict(k_pages=A, v_pages=2 * A, k_scale=3 * A, v_scale=4 * A, n_pages=4, page_rows=16, H=2, D=64)
    d.update(change)
    return uly._CacheDesc(**d)


def append(c=None, **change):
    a = dict(k=5 * A, v=6 * A, ks=0, vs=0, rows=3, starts=7 * A, lens=8 * A, table=9 * A, n=2, width=4)
    a.update(change)
    return uly.lib().uly_cache_append(c or cache(), *a.values(), None)


def attention(c=None, **change):
    a = dict(q=5 * A, qs=0, Hq=4, rows=3, starts=7 * A, lens=8 * A, table=9 * A, n=2, width=400, scale=0.125, o=10 * A,
             lse=11 * A, ws=12 * A, ws_bytes=1 << 40)  # (a width of more than 1024 tokens: with a workspace)
    a.update(change)
    return uly.lib().uly_cache_attention(c or cache(), *a.values(), None)


BAD_CACHE = [(dict(n_pages=0), 1), (dict(page_rows=0), 1), (dict(H=0), 1), (dict(D=0), 1), (dict(page_rows=24), 2),
             (dict(page_rows=256), 2), (dict(D=96), 2), (dict(H=65536), 2), (dict(k_pages=A + 8), 1),
             (dict(v_pages=0), 1), (dict(k_scale=3 * A + 2), 1), (dict(v_scale=0), 1)]
BAD_SEQS = [(dict(rows=-1), 1), (dict(n=-1), 1), (dict(width=0), 1), (dict(starts=0), 1), (dict(lens=0), 1),
            (dict(table=0), 1), (dict(starts=7 * A + 1), 1), (dict(lens=8 * A + 2), 1), (dict(n=65537), 2),
            (dict(rows=(1 << 27) + 1), 2)]


@pytest.mark.parametrize("change,want", BAD_CACHE, ids=str)
def test_caches_that_are_refused(change, want):
    assert append(cache(**change)) == want
    assert attention(cache(**change), Hq=4 if change.get("H", 2) else 0) == want


@pytest.mark.parametrize("change,want", BAD_SEQS, ids=str)
def test_sequences_that_are_refused(change, want):
    assert append(**change) == want
    assert attention(**change) == want


@pytest.mark.parametrize("change", [dict(k=0), dict(v=6 * A + 8), dict(ks=127), dict(vs=132), dict(ks=-8),
                                    dict(vs=(1 << 41)), dict(k=A), dict(v=2 * A + 64), dict(k=3 * A), dict(k=4 * A)],
                         ids=str)
def test_append_refuses(change):
    assert append(**change) == uly.ULY_ERR_INVALID


def test_append_refuses_pools_that_overlap_each_other_or_the_tables():
    for change in (dict(v_pages=A), dict(v_pages=A + 64), dict(v_scale=3 * A), dict(k_scale=A + 128)):
        assert append(cache(**change)) == uly.ULY_ERR_INVALID
    for n in ("starts", "lens", "table"):
        assert append(**{n: 3 * A}) == uly.ULY_ERR_INVALID
    assert append(k=5 * A, v=5 * A + 128, ks=512, vs=512, rows=0) == uly.ULY_OK  # (no row: nothing to do)


@pytest.mark.parametrize("change", [dict(q=0), dict(o=0), dict(ws=0), dict(q=5 * A + 8), dict(lse=11 * A + 1),
                                    dict(qs=255), dict(qs=260), dict(Hq=3), dict(Hq=0), dict(scale=0.0),
                                    dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(ws=12 * A + 16),
                                    dict(ws_bytes=8), dict(o=5 * A), dict(lse=10 * A), dict(o=A), dict(o=8 * A),
                                    dict(ws=10 * A), dict(ws=5 * A)], ids=str)
def test_attention_refuses(change):
    a = dict(ws_bytes=1 << 23)
    need = uly.lib().uly_cache_attention_workspace(cache(), 4, 3, 2, 400)
    assert 0 < need <= 1 << 23
    assert attention(**{**a, **change}) == uly.ULY_ERR_INVALID


def test_nothing_to_do():
    assert append(rows=0) == append(n=0) == uly.ULY_OK
    assert attention(rows=0, ws_bytes=1 << 23) == attention(n=0, ws_bytes=1 << 23) == uly.ULY_OK


def test_null_arguments_and_workspaces():
    L = uly.lib()
    assert L.uly_sp_prompt_attention(None, None, None, None, None, 1, 0.1, None, None, None, 0, None) == \
        uly.ULY_ERR_INVALID
    assert L.uly_sp_prompt_attention_workspace(None, 1) == -1
    assert L.uly_cache_append(None, A, A, 0, 0, 1, A, A, A, 1, 1, None) == uly.ULY_ERR_INVALID
    assert L.uly_cache_attention(None, A, 0, 4, 1, A, A, A, 1, 1, 0.1, A, A, A, 1, None) == uly.ULY_ERR_INVALID
    assert L.uly_cache_attention_workspace(cache(), 4, 3, 2, 64) == 0 < L.uly_cache_attention_workspace(cache(), 4, 3, 2, 65)
    for a in ((None, 4, 3, 2, 1), (cache(H=0), 4, 3, 2, 1), (cache(), 3, 3, 2, 1), (cache(), 0, 3, 2, 1),
              (cache(), 4, -1, 2, 1), (cache(), 4, 3, -1, 1), (cache(), 4, 3, 2, 0), (cache(page_rows=0), 4, 3, 2, 1),
              (cache(), 4, 1 << 62, 2, 100)):
        assert L.uly_cache_attention_workspace(*a) == -1


def test_workspace_of_what_the_call_refuses():
    """-1 where uly_cache_attention refuses the sizes, and no wrapped product of them."""
    L = uly.lib()
    for a in ((cache(H=1), (1 << 31) - 1, 1 << 27, 2, 400), (cache(), 65536, 1 << 27, 2, 400),
              (cache(D=(1 << 31) - 4), 4, 1 << 27, 2, 400), (cache(D=96), 4, 3, 2, 400),
              (cache(page_rows=24), 4, 3, 2, 400), (cache(H=65536), 65536, 3, 2, 400), (cache(), 4, 3, 65537, 400)):
        assert L.uly_cache_attention_workspace(*a) == -1, a[1:]
    # the largest that is taken: units of 16 rows, their notes and sums
    most = L.uly_cache_attention_workspace(cache(H=65535, D=128, page_rows=128), 65535, 1 << 27, 65536, (1 << 31) - 1)
    parts = 2 * 160 * 3 + 65535 * ((1 << 27) // 16 + 65536)
    assert abs(most - (65538 * 8 + parts * (32 + 16 * 132 * 4))) < 1024


class _Shape(uly.Plan):
    """A plan's shape without the library's plan: the binding's own checks."""

    def __init__(self, dtype="bf16"):
        self.B, self.P, self.Hq, self.Hkv, self.D, self.dtype, self.device = 1, 2, 4, 2, 64, dtype, 0
        self._h = None

    def shard_rows(self, shard, is_kv=False):
        return 8

    heads_rows_q = heads_rows_kv = 16


def test_binding_refuses_tensors_that_are_on_no_gpu():
    q, k = [torch.zeros((1, 8, 4, 64), dtype=torch.bfloat16)] * 2, [torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)] * 2
    with pytest.raises(ValueError):
        _Shape().prompt_attention(q, k, k, q, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(uly.UlyError) as e:
        _Shape("e4m3").prompt_attention(q, k, k, q, torch.zeros(2, dtype=torch.int32))
    assert e.value.status == uly.ULY_ERR_UNSUPPORTED
    p, s = torch.zeros((4, 2, 16, 64), dtype=torch.uint8), torch.zeros((4, 2))
    for bad in (p, None, [p]):
        with pytest.raises(ValueError):
            uly.Cache(bad, p, s, s)


# ------------------------------------------------------------ references --
def test_prompt_reference_by_hand():
    c = R.Prompt("hand", (3, 4), (2, 0, 3), 2, 1, 4, first=1)
    d = R.prompt_inputs(c, 1, "cpu")
    o, lse, err, inside = R.prompt_reference(c, d, 0.5)
    q, k, v = (torch.cat(d[n], 1)[0].double() for n in "qkv")
    assert inside.tolist() == [False, True, True, True, True, True, False]
    for i, first in ((1, 1), (2, 1), (3, 3), (4, 3), (5, 3)):
        for h in range(2):
            w = [math.exp(0.5 * float(q[i, h] @ k[j, 0])) for j in range(first, i + 1)]
            want = sum(x * v[j, 0] for x, j in zip(w, range(first, i + 1))) / sum(w)
            assert torch.allclose(o[i, h], want, rtol=1e-12)
            assert math.isclose(float(lse[i, h]), math.log(sum(w)), rel_tol=1e-12, abs_tol=1e-12)


def test_cache_reference_by_hand():
    c = R.Cached("hand", (14, 0), (3, 1), 1, 64, 16, G=2)
    d = R.cache_inputs(c, 2, "cpu")
    w = R.appended(c, d)
    for t in "kv":
        # every new value within half a step of what it was, and the scale the least that holds the page
        for s, a, n, first in ((0, 14, 3, 0), (1, 0, 1, 3)):
            for i in range(n):
                at, slot = int(d["table"][s, (a + i) // 16]), (a + i) % 16
                scale = float(w[t + "_scale"][at, 0])
                x, y = d[t][first + i, 0].double(), w[t + "_pages"][at, 0, slot] * scale
                assert ((x - y).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * scale).all()
        at = int(d["table"][0, 1])  # slot 0 on: positions 16
        top = float(d[t][2, 0].abs().max())
        scale = float(w[t + "_scale"][at, 0])
        assert top <= 448 * scale and top > 224 * scale
        d[t + "_pages"] = w[t + "_pages"].float().to(torch.float8_e4m3fn)
        d[t + "_scale"] = w[t + "_scale"].float()
    o, lse, _, _ = R.cached_reference(c, d, 0.3)
    pages = {t: (w[t + "_pages"] * w[t + "_scale"][..., None, None])[:, 0] for t in "kv"}
    for row, (s, limit) in enumerate(((0, 15), (0, 16), (0, 17), (1, 1))):
        keys = [(int(d["table"][s, j // 16]), j % 16) for j in range(limit)]
        e = [math.exp(0.3 * float(d["q"][row, 1].double() @ pages["k"][p, t])) for p, t in keys]
        want = sum(x * pages["v"][p, t] for x, (p, t) in zip(e, keys)) / sum(e)
        assert torch.allclose(o[row, 1], want, rtol=1e-10)
        assert math.isclose(float(lse[row, 1]), math.log(sum(e)), rel_tol=1e-10)


def test_e4m3_grid():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = codes[~codes.isnan()]
    assert torch.equal(R.to_e4m3(codes), codes)
    x = torch.randn(20000, dtype=torch.float64) * 60
    assert torch.equal(R.to_e4m3(x), x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double())
    x = torch.randn(20000, dtype=torch.float64) * 2.0 ** -8
    assert torch.equal(R.to_e4m3(x.float().double()), x.float().to(torch.float8_e4m3fn).double())


@pytest.mark.parametrize("amax,want", [(0.0, -60), (448.0, 0), (449.0, 1), (7.0, -6), (7.5, -5), (1e-30, -60)])
def test_least_power(amax, want):
    assert R.least_power(amax) == 2.0 ** want


def test_struct_layout():
    assert ctypes.sizeof(uly._CacheDesc) == 48
