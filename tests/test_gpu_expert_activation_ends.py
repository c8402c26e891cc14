"""The activations where the exponential leaves fp32's normal numbers but the result does not: gates whose
logistic lies below 2^-126. Every BF16 gate there, alone and under factors that bring the result back up."""
import pytest
import torch

import expert_ref as R
from test_gpu_expert import BF16, _check, _fill, _operands, _place, _rows, _stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _gates(kind):
    """Every BF16 value whose y (of the logistic's exponential) lies between -80 and -104, 2^-115 to 2^-150."""
    x = -torch.arange(0x4000, 0x4400, dtype=torch.int32).to(torch.int16).view(BF16).double()
    y = x if kind == R.SILU else 2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)
    return x[(y < -80) & (y > -104)].to(BF16)


# As where the exponential is normal (expert_ref.ACT, here |y| up to 104, and two last places more for its square); what
# fp32 holds of a value, 2^-150 beside it, comes with the factor; BF16's results have a step of 2^-133 at the least.
TOL = (4 * 104 + 12) * 2.0 ** -24 + R.half_step(BF16)


def _bound(want, factor):
    return TOL * want.abs() + factor * 2.0 ** -149 + 2.0 ** -134


@pytest.mark.parametrize("kind", [R.SILU, R.GELU])
@pytest.mark.parametrize("exponent", [0, 20, 100])
def test_forward(wt, kind, exponent):
    g = _gates(kind)
    assert len(g) > 10
    n, f = len(g), 2.0 ** exponent
    rows = torch.stack([g, torch.full_like(g, f)], 1)
    w = torch.tensor([[[1.0, 0.0], [0.0, 1.0]]], dtype=BF16)
    h, gx, gw, d, keep = _fill((n, 1), BF16), _place(rows), _place(w), wt.wt_product_desc_init(), []
    _rows(d, R.Layout([n]), keep, dense=True)
    d.form, d.n, d.k, d.act = R.NT, 1, 2, kind
    _operands(d, gx, gw, h, None, keep)
    wt.wt_gated_forward(d, 0, 0, _stream())
    torch.cuda.synchronize()
    want = f * R.act(kind, g.double())[:, None]
    _check("h", h, want, _bound(want, f))


@pytest.mark.parametrize("kind", [R.SILU, R.GELU])
@pytest.mark.parametrize("exponent", [0, 20, 100])
def test_backward(wt, kind, exponent):
    g = _gates(kind)
    n, f = len(g), 2.0 ** exponent
    p = torch.stack([g, torch.ones_like(g)], 1)  # up = 1, dh = f
    out, gy, gd, gp = _fill((n, 2), BF16), _place(torch.full((n, 1), f, dtype=BF16)), _place(torch.ones(1, 1, 1, dtype=BF16)), _place(p)
    d, keep = wt.wt_product_desc_init(), []
    _rows(d, R.Layout([n]), keep, dense=True)
    d.form, d.n, d.k, d.act = R.NN, 1, 1, kind
    _operands(d, gy, gd, out, None, keep)
    wt.wt_gated_backward(d, gp.data_ptr(), 2, _stream())
    torch.cuda.synchronize()
    x = g.double()
    slope, value = f * R.slope(kind, x)[:, None], f * R.act(kind, x)[:, None]
    # the slope is s (1 + (1 - s) x y'), a difference of 1 and a number between 80 and 300: two roundings more
    _check("slope", out[:, :1], slope, _bound(slope, f) + 2.0 ** -22 * slope.abs())
    _check("value", out[:, 1:], value, _bound(value, f))
