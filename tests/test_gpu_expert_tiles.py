"""Sizes that reach each of the experts' product kernels: one and several rounds
of 256 x 256 tiles, 128 x 128 tiles of four and of eight waves, and waves that
split the sum, each with ends of rows, columns and sums at odd places. The
reference is the definition in 64 bits, computed on the GPU expert by expert."""
import math

import pytest
import torch

import expert_ref as R
from gpu_util import log
from test_gpu_expert import BF16, F32, _fill, _gen, _operands, _place, _rows, _stream
from test_gpu_mxfp4 import _padded, _random_mx, _small_mx, _type

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF16).cuda()


def _take(x, index):
    if index is None:
        return x
    i = index[0].cuda().long()
    ok = (i >= 0) & (i < x.shape[0])
    return torch.where(ok[:, None], x[i.clamp(0, x.shape[0] - 1)], torch.zeros((), dtype=x.dtype, device="cuda"))


def _near(name, got, want, bound):
    off, got = (got.double() - want).abs(), None
    worst = (off / bound).max().item()
    log(f"  {name}: worst {worst:.3f} of the bound")
    assert worst <= 1.0, f"{name}: {worst} times the bound"  # a NaN fails too


def _outside(name, buf, lay):
    assert bool((buf[~lay.owned().cuda()] == -7.0).all()), f"{name}: rows of no expert written"


EIGHT = R.Layout([900, 0, 300, 257, 128, 1, 700, 515], align=16, lead=3, tail=5)
# rows, columns, sum: (256 x 256) tiles of 1.1 rounds, of many experts, (128) four waves, (128) eight waves, split sums
SHAPES = [
    ("256", R.Layout([4100]), 4104, 134),
    ("256, experts", EIGHT, 4002, 330),
    ("128", R.Layout([1030]), 5640, 96),
    ("128, experts", R.Layout([70] * 30 + [0, 129], align=128), 1100, 72),
    ("128, eight waves", R.Layout([1000]), 2050, 200),
    ("64, split", R.Layout([120]), 1030, 1022),
    ("16, split", R.Layout([9, 0, 5]), 1030, 3070),
]
IDS = [s[0].replace(" ", "") for s in SHAPES]


def _desc(wt, lay, form, m, n, k, a, b, out, keep, index=None, act=R.SILU):
    d = wt.wt_product_desc_init()
    _rows(d, lay, keep, dense=len(lay.counts) == 1)
    d.form, d.m, d.n, d.k, d.act = form, m, n, k, act
    d.out_dtype = wt.WT_DT_F32 if out.dtype == F32 else wt.WT_DT_BF16
    _operands(d, a, b, out, index, keep)
    return d


@pytest.mark.parametrize("name,lay,n,k", SHAPES, ids=IDS)
@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("gathered", [False, True])
def test_products(wt, form, gathered, name, lay, n, k):
    log(f"{name}: {form} {lay.n_rows} rows of {len(lay.counts)}, {k} x {n}")
    f, g, keep, E = {"nt": R.NT, "nn": R.NN}[form], _gen(n), [], len(lay.counts)
    index = (torch.randint(-1, 301, (lay.n_rows,), generator=g, dtype=torch.int32), 300) if gathered else None
    a = _place(_normal(g, 300 if gathered else lay.n_rows, k), pad=2)
    b = _place(_normal(g, E, *((n, k) if f == R.NT else (k, n))), pad=8)
    rows = _take(a, index)
    for dtype in (BF16, F32):
        out = _fill((lay.n_rows, n), dtype)
        wt.wt_expert_product(_desc(wt, lay, f, 0, n, k, a, b, out, keep, index), _stream())
        for e, s, t in lay.spans():
            if t > s:
                w = b[e].double().t().contiguous() if f == R.NT else b[e].double()
                want, mag = rows[s:t].double() @ w, rows[s:t].double().abs() @ w.abs()
                _near(f"expert {e}", out[s:t], want, R.bound(want, mag, k, dtype) + 1e-30)
        _outside(name, out, lay)


@pytest.mark.parametrize("m,n,lay", [(4100, 4106, R.Layout([70])), (1026, 2052, EIGHT), (1030, 1100, R.Layout([1000])),
                                     (640, 520, R.Layout([300, 0, 500, 33, 7] * 3)), (130, 200, R.Layout([3000])),
                                     (66, 2050, R.Layout([1, 2000]))])
@pytest.mark.parametrize("gathered", [False, True])
def test_gradients_of_weights(wt, gathered, m, n, lay):
    log(f"{lay.n_rows} rows of {len(lay.counts)}, {m} x {n}")
    g, keep, E = _gen(m), [], len(lay.counts)
    index = (torch.randint(-1, 301, (lay.n_rows,), generator=g, dtype=torch.int32), 300) if gathered else None
    a, b = _place(_normal(g, lay.n_rows, m), pad=8), _place(_normal(g, 300 if gathered else lay.n_rows, n), pad=2)
    rows = _take(b, index)
    for dtype in (BF16, F32):
        out = _fill((E, m, n), dtype)
        wt.wt_expert_product(_desc(wt, lay, R.TN, m, n, 0, a, b, out, keep, index), _stream())
        for e, s, t in lay.spans():
            at = a[s:t].double().t().contiguous()
            want, mag = at @ rows[s:t].double(), at.abs() @ rows[s:t].double().abs()
            if t > s:
                _near(f"expert {e}", out[e], want, R.bound(want, mag, t - s, dtype) + 1e-30)
            else:
                assert bool((out[e] == 0).all())


@pytest.mark.parametrize("name,lay,n,k", SHAPES, ids=IDS)
@pytest.mark.parametrize("act", [R.SILU, R.GELU])
def test_gated(wt, act, name, lay, n, k):
    n = n // 4 * 2  # half as many columns of h: the gate and up rows make the tiles
    log(f"{name}: {lay.n_rows} rows of {len(lay.counts)}, {k} x {n}")
    g, keep, E = _gen(k), [], len(lay.counts)
    x, w = _place(_normal(g, lay.n_rows, k), pad=8), _place(_normal(g, E, 2 * n, k, std=1.5 * k ** -0.5), pad=2)
    h, pre = _fill((lay.n_rows, n), BF16), _fill((lay.n_rows, 2 * n), BF16)
    wt.wt_gated_forward(_desc(wt, lay, R.NT, 0, n, k, x, w, h, keep, act=act), pre.data_ptr(), pre.stride(0), _stream())
    dy, down = _place(_normal(g, lay.n_rows, k), pad=2), _place(_normal(g, E, k, n, std=k ** -0.5), pad=8)
    dpre = _fill((lay.n_rows, 2 * n), BF16)
    wt.wt_gated_backward(_desc(wt, lay, R.NN, 0, n, k, dy, down, dpre, keep, act=act), pre.data_ptr(), pre.stride(0), _stream())
    for e, s, t in lay.spans():
        if t == s:
            continue
        wt64, x64 = w[e].double().t().contiguous(), x[s:t].double()
        y, off = x64 @ wt64, R.sum_bound(k, x64.abs() @ wt64.abs())
        u, du, a = y[:, n:], off[:, n:], R.act(act, y[:, :n])
        err = 1.2 * off[:, :n] * (u.abs() + du) + a.abs() * du + R.ACT * (a * u).abs()
        hs = R.half_step(BF16)
        _near(f"h {e}", h[s:t], a * u, err + hs * ((a * u).abs() + err) + 1e-30)
        _near(f"pre {e}", pre[s:t], y, off + hs * (y.abs() + off) + 1e-30)
        dh, offd = dy[s:t].double() @ down[e].double(), R.sum_bound(k, dy[s:t].double().abs() @ down[e].double().abs())
        p, q = pre[s:t, :n].double(), pre[s:t, n:].double()
        want = torch.cat([dh * q * R.slope(act, p), dh * R.act(act, p)], 1)
        sl = 2 * R.ACT * (1 + R.slope(act, p).abs()) + 60 * 2.0 ** -23
        err = torch.cat([offd * q.abs() * 1.2 + (dh.abs() + offd) * q.abs() * sl,
                         offd * R.act(act, p).abs() + R.ACT * (dh.abs() + offd) * R.act(act, p).abs()], 1)
        _near(f"dpre {e}", dpre[s:t], want, err + hs * (want.abs() + err) + 1e-30)
    for name, buf in (("h", h), ("pre", pre), ("dpre", dpre)):
        _outside(name, buf, lay)


MX_SHAPES = [("256", R.Layout([4100]), 4104, 1000), ("256, experts", EIGHT, 4002, 330), ("128", R.Layout([1030]), 2600, 200),
             ("128, experts", R.Layout([70] * 30 + [0, 129], align=128), 1100, 1300), ("32, split", R.Layout([60]), 1030, 3000),
             ("32, experts", R.Layout([9, 0, 5]), 1030, 1111)]


@pytest.mark.parametrize("name,lay,n,k", MX_SHAPES, ids=[s[0].replace(" ", "") for s in MX_SHAPES])
@pytest.mark.parametrize("gated", [False, True])
def test_mxfp4_products(wt, gated, name, lay, n, k):
    n = n // 4 * 2 if gated else n
    log(f"{name}: {lay.n_rows} rows of {len(lay.counts)}, {k} x {n}")
    g, keep, E, nb = _gen(k), [], len(lay.counts), -(-k // 32)
    # gates below 10 in magnitude: sums of k products of values below 6, with scales that keep them so
    make = _random_mx if not gated else lambda g, r, k: _gate_mx(g, r, k)
    ac, asc = make(g, lay.n_rows, k)
    bs = [make(g, n * (1 + gated), k) for _ in range(E)]
    spare = -nb % 4 + 4
    ga, gas = _padded(ac, 16, 0x77), _padded(asc, spare, 255)
    gb, gbs = _padded(torch.stack([c for c, _ in bs]), 16, 0x77), _padded(torch.stack([s for _, s in bs]), spare, 255)
    a = R.mx_values(ac, asc).cuda()
    for dtype in ((BF16,) if gated else (BF16, F32)):
        out = _fill((lay.n_rows, n), dtype)
        d = wt.wt_mxfp4_product_desc_init()
        _rows(d, lay, keep, dense=E == 1)
        d.n, d.k, d.gated, d.out_dtype = n, k, int(gated), _type(wt, dtype)
        d.a, d.a_stride, d.a_scales, d.a_scale_stride = ga.data_ptr(), ga.stride(0), gas.data_ptr(), gas.stride(0)
        d.b, d.b_stride, d.b_expert_stride = gb.data_ptr(), gb.stride(1), gb.stride(0)
        d.b_scales, d.b_scale_stride, d.b_scale_expert_stride = gbs.data_ptr(), gbs.stride(1), gbs.stride(0)
        d.out, d.out_stride = out.data_ptr(), out.stride(0)
        wt.wt_mxfp4_product(d, _stream())
        for e, s, t in lay.spans():
            if t == s:
                continue
            w = R.mx_values(*bs[e]).cuda().t().contiguous()
            y, off = a[s:t] @ w, R.sum_bound(k, a[s:t].abs() @ w.abs())
            if gated:
                h = R.act(R.SILU, y[:, :n]) * y[:, n:]
                err = 1.2 * off[:, :n] * (y[:, n:].abs() + off[:, n:]) + R.act(R.SILU, y[:, :n]).abs() * off[:, n:] + R.ACT * h.abs()
                _near(f"h {e}", out[s:t], h, err + R.half_step(BF16) * (h.abs() + err) + 1e-30)
            else:
                _near(f"expert {e}", out[s:t], y, off + R.half_step(dtype) * (y.abs() + off) + 1e-30)
        _outside(name, out, lay)


def _gate_mx(g, rows, k):
    """Codes of random signs with scales of 2^-5: sums of k products of sizes below 36 * 2^-10 and both signs."""
    codes, scales = _small_mx(g, rows, k)
    return codes, torch.full_like(scales, 127 - 5)


@pytest.mark.parametrize("gated", [False, True])
def test_mxfp4_rows_far_apart(wt, gated):
    """Rows of codes 4 MB + 16 bytes apart: beyond what a tile's offsets hold."""
    g, far, n, k, lay = _gen(1), 2 ** 22 + 16, 24, 70, R.Layout([33])
    (ac, asc), (bc, bsc) = _small_mx(g, 33, k), _small_mx(g, n * (1 + gated), k)
    bufs = [torch.zeros(r * far, dtype=torch.uint8, device="cuda") for r in (33, n * (1 + gated))]
    for buf, c in zip(bufs, (ac, bc)):
        torch.as_strided(buf, c.shape, (far, 1)).copy_(c)
    gas, gbs, out = _padded(asc, 1, 255), _padded(bsc, 1, 255), _fill((33, n), BF16)
    d = wt.wt_mxfp4_product_desc_init()
    d.n_rows, d.n, d.k, d.gated = 33, n, k, int(gated)
    d.a, d.a_stride, d.a_scales, d.a_scale_stride = bufs[0].data_ptr(), far, gas.data_ptr(), 4
    d.b, d.b_stride, d.b_scales, d.b_scale_stride = bufs[1].data_ptr(), far, gbs.data_ptr(), 4
    d.out, d.out_stride = out.data_ptr(), n
    wt.wt_mxfp4_product(d, _stream())
    y, mag, terms = R.product(R.NT, lay, R.mx_values(ac, asc), R.mx_values(bc, bsc)[None])
    off = R.sum_bound(terms, mag)
    if gated:
        h = R.act(R.SILU, y[:, :n]) * y[:, n:]
        err = 1.2 * off[:, :n] * (y[:, n:].abs() + off[:, n:]) + R.act(R.SILU, y[:, :n]).abs() * off[:, n:] + R.ACT * h.abs()
        _near("h", out.cpu(), h, err + R.half_step(BF16) * (h.abs() + err) + 1e-30)
    else:
        _near("product", out.cpu(), y, R.bound(y, mag, terms, BF16) + 1e-30)
    assert math.isfinite(out.float().sum().item())
