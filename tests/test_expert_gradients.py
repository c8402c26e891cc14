"""The gated block's gradients (forward, backward through the gate, both products) against 64-bit
gradients of the block and against its differences, element by element, within what BF16 does to the
values kept between the calls. On the CPU: the bounds hold for these calls done in 64 bits with the same
roundings, and exclude gradients that are wrong."""
import pytest
import torch

import expert_ref as R
from test_gpu_expert import _fill, _gen, _normal, _operands, _place, _rows, _stream

BF16, F32 = torch.bfloat16, torch.float32
LAY, N, K = R.Layout([9, 0, 21], align=8), 24, 40
KINDS = [R.SILU, R.GELU]
# |slope'| is at most 0.5 for SiLU and 0.8 for GELU (both at 0), |slope| at most 1.13
CURVE, SLOPE = 0.85, 1.13


def _inputs(kind):
    g = _gen(12 + kind)
    x, w, down = _normal(g, LAY.n_rows, K), _normal(g, 3, 2 * N, K, std=0.3), _normal(g, 3, K, N, std=0.3)
    return x, w, down, _normal(g, LAY.n_rows, K)


def _loss(kind, x, w, down, dy):
    y = R.product(R.NT, LAY, x, w)[0]
    h = torch.where(LAY.owned()[:, None], R.act(kind, y[:, :N]) * y[:, N:], torch.zeros((), dtype=torch.float64))
    z = R.product(R.NT, LAY, h, down.double())[0]
    return (z * dy.double())[LAY.owned()].sum()


def _formula(kind, x, w, down, dy):
    """dx and dw in 64 bits, from the chain rule written out expert by expert."""
    dx, dw = torch.zeros(LAY.n_rows, K, dtype=torch.float64), torch.zeros(3, 2 * N, K, dtype=torch.float64)
    for e, s, t in LAY.spans():
        xe, we, de = x[s:t].double(), w[e].double(), down[e].double()
        y = xe @ we.t()
        gate, up = y[:, :N], y[:, N:]
        dh = dy[s:t].double() @ de
        dpre = torch.cat([dh * up * R.slope(kind, gate), dh * R.act(kind, gate)], 1)
        dx[s:t], dw[e] = dpre @ we, dpre.t() @ xe
    return dx, dw


def _bounds(kind, x, w, down, dy):
    """What dx and dw of the calls may be off by: pre and dpre are BF16 in memory, everything else fp32 sums."""
    y, off = R.gated(LAY, x, w, kind)["pre"]
    own = LAY.owned()
    y, off = y.clone(), off.clone()
    y[~own], off[~own] = 0, 0
    dpre, step = R.gated_back(LAY, dy, down, y, kind)  # the step from pre to dpre, and its rounding
    dh = R.product(R.NN, LAY, dy, down)[0]
    dpre[~own], dh[~own], step[~own] = 0, 0, 0
    g, u, dg, du = y[:, :N], y[:, N:], off[:, :N], off[:, N:]
    moved = torch.cat([dh.abs() * (R.slope(kind, g).abs() * du + (u.abs() + du) * CURVE * dg), dh.abs() * SLOPE * dg], 1)
    # `step` is relative to dpre at y; at y + off it is larger by the same part of `moved`
    err = step + moved * (1 + 2.0 ** -7)
    total = dpre.abs() + err
    bx, bw = torch.zeros(LAY.n_rows, K, dtype=torch.float64), torch.zeros(3, 2 * N, K, dtype=torch.float64)
    for e, s, t in LAY.spans():
        we, xe = w[e].double().abs(), x[s:t].double().abs()
        bx[s:t] = err[s:t] @ we + R.bound(torch.zeros(()), total[s:t] @ we, 2 * N, F32)
        bw[e] = err[s:t].t() @ xe + R.bound(torch.zeros(()), total[s:t].t() @ xe, max(1, t - s), F32)
    # R.bound's rounding of the result itself
    fx, fw = _formula(kind, x, w, down, dy)
    return bx + R.half_step(F32) * fx.abs(), bw + R.half_step(F32) * fw.abs()


def _calls(kind, x, w, down, dy, slope=None, cast=lambda t: t.to(BF16).double()):
    """The calls in 64 bits with the roundings of what they keep; `slope` puts another formula in."""
    slope, dx, dw = slope or R.slope, torch.zeros(LAY.n_rows, K, dtype=torch.float64), torch.zeros(3, 2 * N, K, dtype=torch.float64)
    for e, s, t in LAY.spans():
        xe, we, de = x[s:t].double(), w[e].double(), down[e].double()
        pre = cast(xe @ we.t())
        gate, up, dh = pre[:, :N], pre[:, N:], dy[s:t].double() @ de
        dpre = cast(torch.cat([dh * up * slope(kind, gate), dh * R.act(kind, gate)], 1))
        dx[s:t], dw[e] = dpre @ we, dpre.t() @ xe
    return dx, dw


def _far(got, want, bound):
    """The part of the elements that are beyond the bound."""
    return ((got - want).abs() > bound).double().mean().item()


@pytest.mark.parametrize("kind", KINDS)
def test_the_formula_is_the_blocks_gradient(kind):
    x, w, down, dy = _inputs(kind)
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    _loss(kind, x64, w64, down, dy).backward()
    for got, want in zip(_formula(kind, x, w, down, dy), (x64.grad, w64.grad)):
        assert torch.allclose(got, want, rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("kind", KINDS)
def test_the_bounds_hold_for_bf16_and_exclude_wrong_gradients(kind):
    args = _inputs(kind)
    want, bounds = _formula(kind, *args), _bounds(kind, *args)
    assert [_far(g, t, b) for g, t, b in zip(_calls(kind, *args), want, bounds)] == [0, 0]
    own = LAY.owned()

    def wrong(got):
        return _far(got[0][own], want[0][own], bounds[0][own]), _far(got[1][[0, 2]], want[1][[0, 2]], bounds[1][[0, 2]])

    assert min(wrong((0 * want[0], 0 * want[1]))) > 0.9  # no gradient
    assert min(wrong((-want[0], -want[1]))) > 0.9
    assert min(wrong((1.25 * want[0], 1.25 * want[1]))) > 0.3
    # a slope without its second term
    assert min(wrong(_calls(kind, *args, slope=lambda k, g: torch.sigmoid(g if k == R.SILU else 1.702 * g)))) > 0.2
    # the other activation's slope
    assert min(wrong(_calls(kind, *args, slope=lambda k, g: R.slope(1 - k, g)))) > 0.02
    # gate and up in each other's place
    x, w, down, dy = args
    swapped = torch.cat([w[:, N:], w[:, :N]], 1)
    dx, dw = _calls(kind, x, swapped, down, dy)
    assert min(wrong((dx, torch.cat([dw[:, N:], dw[:, :N]], 1)))) > 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_gradients(kind):
    from bf16_fp8_weight_amd import wt

    x, w, down, dy = _inputs(kind)
    keep = []
    gx, gw, gd, gy = _place(x), _place(w), _place(down), _place(dy)
    h, pre = _fill((LAY.n_rows, N), BF16), _fill((LAY.n_rows, 2 * N), BF16)
    dpre, dx, dw = torch.zeros_like(pre), _fill((LAY.n_rows, K), F32), _fill((3, 2 * N, K), F32)

    def desc(form, m, n, k, a, b, out):
        d = wt.wt_product_desc_init()
        _rows(d, LAY, keep)
        d.form, d.m, d.n, d.k, d.act = form, m, n, k, kind
        d.out_dtype = wt.WT_DT_F32 if out.dtype == F32 else wt.WT_DT_BF16
        _operands(d, a, b, out)
        return d

    wt.wt_gated_forward(desc(R.NT, 0, N, K, gx, gw, h), pre.data_ptr(), pre.stride(0), _stream())
    wt.wt_gated_backward(desc(R.NN, 0, N, K, gy, gd, dpre), pre.data_ptr(), pre.stride(0), _stream())
    wt.wt_expert_product(desc(R.NN, 0, K, 2 * N, dpre, gw, dx), _stream())
    wt.wt_expert_product(desc(R.TN, 2 * N, K, 0, dpre, gx, dw), _stream())
    torch.cuda.synchronize()
    (fx, fw), (bx, bw), own = _formula(kind, x, w, down, dy), _bounds(kind, x, w, down, dy), LAY.owned()
    got_x, got_w = dx.cpu().double(), dw.cpu().double()
    assert _far(got_x[own], fx[own], bx[own]) == 0 and _far(got_w, fw, bw) == 0
    assert bool((got_x[~own] == -7).all()) and bool((got_w[1] == 0).all())
    # differences of the block, whose own error (the third derivative's step^2 / 6, and 64-bit roundings over the step) stays
    # below 1e-5 of the largest gradient
    step, x64, w64 = 1e-4, x.double(), w.double()

    def difference(t, at):
        pair = []
        for sign in (1, -1):
            moved = t.clone()
            moved[at] += sign * step
            pair.append(_loss(kind, moved if t is x64 else x64, moved if t is w64 else w64, down, dy))
        return (pair[0] - pair[1]).item() / (2 * step)

    for at in [(0, 0), (8, 39), (16, 3), (30, 17), (36, 1)]:
        assert abs(got_x[at].item() - difference(x64, at)) <= bx[at].item() + 1e-5 * fx.abs().max().item()
    for at in [(0, 0, 0), (0, 47, 39), (2, 5, 7), (2, 30, 1)]:
        assert abs(got_w[at].item() - difference(w64, at)) <= bw[at].item() + 1e-5 * fw.abs().max().item()
