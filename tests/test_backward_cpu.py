"""The gradient calls and uly_norm_rope on the CPU: refusals that need no GPU,
and the 64-bit reference of the GPU tests against difference quotients."""
import ctypes
import math

import pytest
import torch

import ulysses_sequence_attention_uly_gb300 as uly
from tests import _grad as R


def test_null_plans_are_refused():
    L = uly.lib()
    one = ctypes.c_float(0.125)
    for fn in (L.uly_attention_backward, L.uly_sp_attention_backward):
        assert fn(None, None, None, None, None, None, None, None, None, 0, one, None, None, None, None, 0,
                  None) == uly.ULY_ERR_INVALID
    assert L.uly_norm_rope(None, None, None, 0, 0, None, None, None, None, 1, 0, one, None, None,
                           None) == uly.ULY_ERR_INVALID
    assert L.uly_norm_rope_backward(None, None, None, 0, 0, None, None, None, None, None, None, 1, 0, one, None, None,
                                    None, None, None, 0, None) == uly.ULY_ERR_INVALID
    assert L.uly_attention_backward_workspace(None) == -1
    assert L.uly_norm_rope_backward_workspace(None) == -1


class _Shape(uly.Plan):
    """A plan's shape without the library's plan: the binding's own checks."""

    def __init__(self):
        self.B, self.P, self.Hq, self.Hkv, self.D, self.dtype, self.device = 1, 2, 4, 2, 64, "bf16", 0
        self._h = None

    def shard_rows(self, shard, is_kv=False):
        return 8

    heads_rows_q = heads_rows_kv = 16


def test_binding_refuses_before_any_call():
    p = _Shape()
    q, k = [torch.zeros((1, 8, 4, 64), dtype=torch.bfloat16)] * 2, [torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)] * 2
    lse = [torch.zeros((1, 8, 4))] * 2
    for call in (p.sp_attention_backward, p.attention_backward):
        with pytest.raises(ValueError):  # not on a GPU
            call(q, k, k, q, lse, q, q, k, k)
        with pytest.raises(ValueError):
            call(q, k, k, q, None, q, q, k, k)
        for bad in ([1], q[0]):  # neither is a mask or ranges on a GPU
            with pytest.raises(ValueError):
                call(q, k, k, q, lse, q, q, k, k, key_mask=bad)
            with pytest.raises(ValueError):
                call(q, k, k, q, lse, q, q, k, k, key_ranges=bad)
    with pytest.raises(ValueError):
        p.norm_rope(q, k, q, k)
    with pytest.raises(ValueError):
        p.norm_rope_backward(q, k, q, k, q, k)


@pytest.mark.parametrize("bad", [[1.0], 1.0, "cos"])
def test_tables_that_are_no_tensors_are_refused(bad):
    p = _Shape()
    good = torch.zeros((16, 32))
    for cos, sin in ((bad, good), (bad, bad), (good, bad)):
        with pytest.raises(ValueError):
            p.norm_rope(None, None, None, None, cos=cos, sin=sin)
        with pytest.raises(ValueError):
            p.norm_rope_backward(None, None, None, None, None, None, cos=cos, sin=sin)


@pytest.mark.parametrize("c", [R.Case("prefix", 1, (5, 4), 3, "prefix", 4, 2, 8, mask="ranges"),
                               R.Case("suffix-self", 2, (6, 3), 2, "suffix", 2, 2, 8, rows="self", mask="random"),
                               R.Case("kv-zero", 1, (7, 5), 4, "kv_prefix", 4, 2, 8, rows="zero", mask="random")],
                         ids=lambda c: c.name)
def test_reference_gradient_is_the_difference_quotient(c):
    """The reference's dq, dk, dv against central differences of <o, do>, and its
    own forward's o against softmax by hand for one row."""
    d = R.inputs(c, 1, "cpu")
    ref = R.reference(c, d)
    gen = torch.Generator().manual_seed(2)

    def loss(t):
        o, _, _ = R.attention(c, *(R.to_global(c, t[n], i) for n, i in zip("qkv", (False, True, True))), d["mask"],
                              ref["scale"])
        return sum(float((x * y.double()).sum()) for x, y in zip(R.to_shards(c, o, False), d["do"]))

    base = {n: [x.double() for x in d[n]] for n in "qkv"}
    for n in "qkv":
        dirs = [torch.randn(x.shape, generator=gen, dtype=torch.float64) for x in base[n]]
        h = 1e-5
        up, down = (loss({**base, n: [x + s * y for x, y in zip(base[n], dirs)]}) for s in (h, -h))
        got = sum(float((x * y).sum()) for x, y in zip(ref["d" + n], dirs))
        # central differences: h^2 times the third derivative, and 2^-52 / h of the loss
        assert abs((up - down) / (2 * h) - got) <= 1e-6 * (1 + abs(got))


def test_reference_rotation_is_a_rotation():
    c = R.Case("rot", 1, (4,), 2, "prefix", 2, 2, 8)
    g = torch.Generator().manual_seed(3)
    x = torch.randn((1, 6, 2, 8), generator=g, dtype=torch.float64)
    ang = torch.randn((c.nk, 4), generator=g, dtype=torch.float64)
    for pairs in ("interleaved", "half"):
        y = R.norm_rope(c, x, None, ang.cos(), ang.sin(), 0, False, pairs, 1e-12)
        # unit mean square, and pair 1 of row 3 turned by its angle
        torch.testing.assert_close(y.square().mean(-1), torch.ones((1, 6, 2), dtype=torch.float64), rtol=1e-6, atol=0)
        z = x[0, 3, 0] / x[0, 3, 0].square().mean().sqrt()
        a, b = (2, 3) if pairs == "interleaved" else (1, 5)
        t = float(ang[3, 1])
        assert math.isclose(float(y[0, 3, 0, a]), float(z[a]) * math.cos(t) - float(z[b]) * math.sin(t), rel_tol=1e-5)
        assert math.isclose(float(y[0, 3, 0, b]), float(z[a]) * math.sin(t) + float(z[b]) * math.cos(t), rel_tol=1e-5)
