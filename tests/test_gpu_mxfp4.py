"""MXFP4 on the GPU against its definition (expert_ref): every BF16 value under
every kind of scale, ragged rows, gathered rows, values that are not finite, and
products of such rows."""
import math

import pytest
import torch

import expert_ref as R
from gpu_util import log
from test_gpu_expert import UNEVEN, _check, _fill, _gen, _rows, _stream, _untouched

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _type(wt, dtype):
    return wt.WT_DT_F32 if dtype == F32 else wt.WT_DT_BF16


def _quantize(wt, x, index=None, pad=0, shift=0, code_pad=0, scale_pad=0, scale_shift=0):
    """(packed codes, scales) as views of filled buffers."""
    rows, cols = x.shape
    n_out, nb = rows if index is None else len(index), -(-cols // 32)
    flat = torch.full((rows * (cols + pad) + shift + 8,), math.nan, dtype=x.dtype, device="cuda")
    gx = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    gx.copy_(x)
    gi = None if index is None else index.cuda()
    codes = torch.full((n_out, 16 * nb + code_pad), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((n_out * (nb + scale_pad) + scale_shift,), 0xA5, dtype=torch.uint8, device="cuda")
    wt.wt_mxfp4_quantize(gx.data_ptr(), _type(wt, x.dtype), rows, cols, cols + pad, gi.data_ptr() if gi is not None else 0,
                         n_out, codes.data_ptr(), codes.stride(0), scales.data_ptr() + scale_shift, nb + scale_pad, _stream())
    torch.cuda.synchronize()
    scales = scales[scale_shift:].view(n_out, nb + scale_pad)
    assert bool((codes[:, 16 * nb:] == 0xA5).all()) and bool((scales[:, nb:] == 0xA5).all())
    return codes[:, : 16 * nb], scales[:, :nb]


def _dequantize(wt, codes, scales, cols, dtype, pad=0, shift=0):
    rows = codes.shape[0]
    flat = torch.full((rows * (cols + pad) + shift + 8,), -7.0, dtype=dtype, device="cuda")
    wt.wt_mxfp4_dequantize(codes.data_ptr(), codes.stride(0), scales.data_ptr(), scales.stride(0), rows, cols,
                           flat.data_ptr() + shift * flat.element_size(), _type(wt, dtype), cols + pad, _stream())
    torch.cuda.synchronize()
    v = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)
    assert bool((v[:, cols:] == -7).all()) and bool((flat[:shift] == -7).all())
    return v[:, :cols]


def _same(got, want):
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok]) and torch.equal(torch.signbit(got[ok]), torch.signbit(want[ok]))


def _round_trip(wt, x, **kw):
    codes, scales = _quantize(wt, x, **kw)
    index = kw.get("index")
    src = x if index is None else x[index.long()]
    want_codes, want_scales = R.mx_round(src)
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(codes.cpu(), R.mx_pack(want_codes))
    want = R.mx_values(R.mx_pack(want_codes), want_scales)[:, : x.shape[1]]
    for dtype in (BF16, F32):
        _same(_dequantize(wt, codes, scales, x.shape[1], dtype, pad=kw.get("pad", 0), shift=kw.get("shift", 0)).double().cpu(),
              want)


@pytest.mark.parametrize("top", range(-133, 128, 13))
def test_every_bf16_value_below_a_blocks_largest(wt, top):
    """Blocks whose largest magnitude is 2^top, 1.5 * 2^top or near 2^(top + 1), filled with every BF16 value up to it."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    for largest in (1.0, 1.5, 1.9921875):
        m = torch.tensor(largest * 2.0 ** top, dtype=torch.float64).to(BF16)
        x = every[torch.isfinite(every) & (every.abs() <= m)]
        x = torch.cat([x, torch.zeros(-len(x) % 31, dtype=BF16)]).view(-1, 31)
        x = torch.cat([m.expand(len(x), 1), x], 1).contiguous()
        _round_trip(wt, x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (5, 33), (7, 8), (64, 64), (2, 1000), (300, 7), (17, 7168),
                                       (1000, 96), (9, 2817)])
def test_shapes(wt, dtype, rows, cols):
    x = (torch.randn(rows, cols, generator=_gen(cols)) * torch.exp(2 * torch.randn(rows, cols, generator=_gen(rows)))).to(dtype)
    _round_trip(wt, x)
    for pad, shift, code_pad, scale_pad, scale_shift in [(8, 0, 16, 4, 0), (1, 1, 4, 1, 1), (3, 0, 0, 3, 3), (4, 4, 8, 0, 2)]:
        _round_trip(wt, x, pad=pad, shift=shift, code_pad=code_pad, scale_pad=scale_pad, scale_shift=scale_shift)


def test_fp32_ties_and_neighbours(wt):
    """Values on, just below and just above the points between two codes, under several scales."""
    grid = torch.tensor(R.E2M1, dtype=F32)
    mid = (grid[1:] + grid[:-1]) / 2
    v = torch.cat([mid, torch.nextafter(mid, torch.tensor(0.0)), torch.nextafter(mid, torch.tensor(9.0)), grid,
                   torch.tensor([6.5, 7.0, 7.9999995])])
    v = torch.cat([v, -v])
    v = torch.cat([v, torch.zeros(-len(v) % 31)]).view(-1, 31)
    for e in (-125, -100, -20, 0, 7, 120):
        for first in (4.0, 7.9999995):
            _round_trip(wt, torch.cat([torch.full((len(v), 1), first), v.clamp(-first, first)], 1) * 2.0 ** e)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_that_are_not_finite_and_zeros(wt, dtype):
    x = torch.randn(6, 96, generator=_gen(1)).to(dtype)
    x[0, 3], x[1, 40], x[2, 95], x[3, 64:], x[4, 0] = math.nan, math.inf, -math.inf, 0.0, -0.0
    x[5] = -0.0
    _round_trip(wt, x)
    codes, scales = _quantize(wt, x)
    assert scales[0, 0] == 255 and scales[1, 1] == 255 and scales[2, 2] == 255 and scales[3, 2] == 127


def test_every_scale_of_every_code(wt):
    codes = torch.arange(16, dtype=torch.uint8)
    row = torch.cat([codes | (codes.flip(0) << 4)]).expand(256, 16).contiguous().cuda()
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(256, 1).cuda()
    want = R.mx_values(row.cpu(), scales.cpu())
    for dtype in (BF16, F32):
        top = torch.finfo(dtype).max
        w = torch.where(want.abs() > top, torch.copysign(torch.tensor(math.inf, dtype=torch.float64), want), want)
        _same(_dequantize(wt, row, scales, 32, dtype).double().cpu(), w)


def test_gathered_rows(wt):
    x = torch.randn(40, 200, generator=_gen(2)).to(BF16)
    index = torch.randint(0, 40, (500,), generator=_gen(3), dtype=torch.int32)
    _round_trip(wt, x, index=index)
    index[::7] = -1
    index[3::11] = 40
    nb = 7
    codes = torch.full((500, 16 * nb), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((500, nb), 0xA5, dtype=torch.uint8, device="cuda")
    gx, gi = x.cuda(), index.cuda()
    wt.wt_mxfp4_quantize(gx.data_ptr(), wt.WT_DT_BF16, 40, 200, 200, gi.data_ptr(), 500, codes.data_ptr(), 16 * nb,
                         scales.data_ptr(), nb, _stream())
    torch.cuda.synchronize()
    gone = (index < 0) | (index >= 40)
    assert bool((codes.cpu()[gone] == 0xA5).all()) and bool((scales.cpu()[gone] == 0xA5).all())
    c, s = R.mx_round(x[index[~gone].long()])
    assert torch.equal(codes.cpu()[~gone], R.mx_pack(c)) and torch.equal(scales.cpu()[~gone], s)


# ------------------------------------------------------------------ products
def _random_mx(g, rows, k, wild=False):
    """Packed codes (zero behind k), scales and the values of random rows."""
    nb = -(-k // 32)
    code = torch.randint(0, 16, (rows, nb * 32), generator=g, dtype=torch.int32).to(torch.uint8)
    code[:, k:] = 0
    scales = torch.randint(*((90, 160) if wild else (123, 131)), (rows, nb), generator=g, dtype=torch.int32).to(torch.uint8)
    return R.mx_pack(code), scales


def _padded(x, pad, fill):
    """[..., rows, bytes] on the GPU with `pad` bytes of `fill` behind each row."""
    y = torch.full((*x.shape[:-1], x.shape[-1] + pad), fill, dtype=torch.uint8, device="cuda")
    y[..., : x.shape[-1]] = x.cuda()
    return y


def _product(wt, lay, n, k, seed, gated=False, kind=R.SILU, out_dtype=BF16, dense=False, pad=0, wild=False, share=False, nan=False):
    g, keep, E = _gen(seed), [], len(lay.counts)
    b_rows, nb = n * (2 if gated else 1), -(-k // 32)
    ac, asc = _random_mx(g, lay.n_rows, k, wild)
    bs = [_random_mx(g, b_rows, k, wild) for _ in range(1 if share else E)]
    bc, bsc = torch.stack([c for c, _ in bs]), torch.stack([s for _, s in bs])
    if nan:
        asc[3, 0] = 255
        bsc[0, 5, nb - 1] = 255
        asc[~lay.owned()] = 255
    spare = -nb % 4 + (4 if pad else 0)
    # behind the rows: NaN scales, and codes that would count
    ga, gas = _padded(ac, pad, 0x77), _padded(asc, spare, 255)
    gb, gbs = _padded(bc, pad, 0x77), _padded(bsc, spare, 255)
    out = _fill((lay.n_rows, n), out_dtype, pad=pad // 4)
    d = wt.wt_mxfp4_product_desc_init()
    _rows(d, lay, keep, dense)
    d.n, d.k, d.gated, d.act, d.out_dtype = n, k, int(gated), kind, _type(wt, out_dtype)
    d.a, d.a_stride, d.a_scales, d.a_scale_stride = ga.data_ptr(), ga.stride(0), gas.data_ptr(), gas.stride(0)
    d.b, d.b_stride, d.b_expert_stride = gb.data_ptr(), gb.stride(1), 0 if share else gb.stride(0)
    d.b_scales, d.b_scale_stride, d.b_scale_expert_stride = gbs.data_ptr(), gbs.stride(1), 0 if share else gbs.stride(0)
    d.out, d.out_stride = out.data_ptr(), out.stride(0)
    wt.wt_mxfp4_product(d, _stream())
    torch.cuda.synchronize()
    a = R.mx_values(ac, asc)
    b = torch.stack([R.mx_values(c, s) for c, s in zip(bc, bsc)]).expand(E, -1, -1)
    y, mag, terms = R.product(R.NT, lay, a, b)
    own, off = lay.owned(), R.sum_bound(terms, mag)
    if gated:
        h = R.act(kind, y[:, :n]) * y[:, n:]
        err = 1.2 * off[:, :n] * (y[:, n:].abs() + off[:, n:]) + R.act(kind, y[:, :n]).abs() * off[:, n:] + R.ACT * h.abs()
        _check("h", out, h, err + R.half_step(BF16) * (h.abs() + err) + 2.0 ** -133, own)
    else:
        _check("product", out, y, R.bound(y, mag, terms, out_dtype), own)
    _untouched("rows of no expert", out, ~own)


@pytest.mark.parametrize("n,k", [(128, 256), (64, 128), (1, 1), (5, 33), (40, 31), (131, 300), (264, 1000), (72, 96), (16, 64),
                                 (130, 2817)])
def test_products_of_uneven_experts(wt, n, k):
    log(f"{n} x {k}")
    for dtype in (BF16, F32):
        _product(wt, UNEVEN, n, k, seed=n + k, out_dtype=dtype)
    _product(wt, UNEVEN, n, k, seed=n + k, pad=16)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 255, 257, 400])
def test_products_of_a_dense_layer(wt, rows):
    _product(wt, R.Layout([rows]), 200, 416, seed=rows, dense=True, out_dtype=F32)
    _product(wt, R.Layout([rows]), 200, 416, seed=rows, dense=True, pad=32)


# gates below 10 in magnitude, as the activations' bounds assume
@pytest.mark.parametrize("kind", [R.SILU, R.GELU])
@pytest.mark.parametrize("n,k", [(64, 32), (128, 64), (5, 33), (131, 40), (72, 96)])
def test_gated_products(wt, kind, n, k, monkeypatch):
    monkeypatch.setitem(globals(), "_random_mx", _small_mx)
    _product(wt, UNEVEN, n, k, seed=n + k, gated=True, kind=kind)
    _product(wt, R.Layout([77]), n, k, seed=n + k, gated=True, kind=kind, dense=True, pad=16)


def _small_mx(g, rows, k, wild=False):
    nb = -(-k // 32)
    code = torch.randint(0, 16, (rows, nb * 32), generator=g, dtype=torch.int32).to(torch.uint8)
    code[:, k:] = 0
    scales = torch.randint(123, 126, (rows, nb), generator=g, dtype=torch.int32).to(torch.uint8)
    return R.mx_pack(code), scales


def test_scales_far_apart(wt):
    _product(wt, UNEVEN, 72, 520, seed=5, wild=True, out_dtype=F32)


def test_nan_scales_stay_with_their_rows_and_columns(wt):
    _product(wt, UNEVEN, 72, 520, seed=6, nan=True, out_dtype=F32)
    _product(wt, R.Layout([4, 3, 9], tail=2), 72, 520, seed=6, nan=True)


@pytest.mark.parametrize("experts", [2, 65, 300])
def test_many_experts_and_shared_weights(wt, experts):
    counts = torch.randint(0, 5, (experts,), generator=_gen(experts)).tolist()
    counts[experts // 2] = 140
    lay = R.Layout(counts, align=4, tail=3)
    _product(wt, lay, 40, 64, seed=experts)
    _product(wt, lay, 40, 64, seed=experts, share=True)


def test_from_tokens_to_a_gated_product_replayed(wt):
    """Quantised while gathered, through both products, as an engine serves it; then replayed from a graph with other tokens."""
    T, H, N, E = 30, 96, 64, 5
    g = _gen(9)
    lay = R.Layout([9, 0, 30, 4, 17], align=16)
    x = torch.randn(T, H, generator=g).to(BF16).cuda()
    w1, w2 = (torch.randn(E, n, k, generator=g).mul_(k ** -0.5).to(BF16) for n, k in ((2 * N, H), (H, N)))
    token = torch.where(lay.owned(), torch.randint(0, T, (lay.n_rows,), generator=g, dtype=torch.int32), -1).to(torch.int32)
    tok, off, cnt = token.cuda(), lay.offsets.cuda(), lay.counts_t.cuda()

    def packed(rows, k):
        return (torch.zeros(rows, 16 * -(-k // 32), dtype=torch.uint8, device="cuda"),
                torch.zeros(rows, 4 * -(-k // 128), dtype=torch.uint8, device="cuda"))

    def quantize(src, rows, k, to, index=None):
        wt.wt_mxfp4_quantize(src.data_ptr(), wt.WT_DT_BF16, src.shape[0], k, src.stride(0), index.data_ptr() if index is not None else 0,
                             rows, to[0].data_ptr(), to[0].stride(0), to[1].data_ptr(), to[1].stride(0), _stream())

    mats = []
    for w in (w1, w2):
        gw, to = w.cuda().view(-1, w.shape[2]), packed(E * w.shape[1], w.shape[2])
        quantize(gw, gw.shape[0], w.shape[2], to)
        mats.append(to)
    xa, ha = packed(lay.n_rows, H), packed(lay.n_rows, N)
    h, y = (torch.zeros(lay.n_rows, c, dtype=BF16, device="cuda") for c in (N, H))

    def desc(n, k, a, b, out, gated):
        d = wt.wt_mxfp4_product_desc_init()
        d.n_rows, d.n_experts, d.offsets, d.counts, d.n, d.k, d.gated = lay.n_rows, E, off.data_ptr(), cnt.data_ptr(), n, k, gated
        rows = n * (1 + gated)
        d.a, d.a_stride, d.a_scales, d.a_scale_stride = a[0].data_ptr(), a[0].stride(0), a[1].data_ptr(), a[1].stride(0)
        d.b, d.b_stride, d.b_expert_stride = b[0].data_ptr(), b[0].stride(0), rows * b[0].stride(0)
        d.b_scales, d.b_scale_stride, d.b_scale_expert_stride = b[1].data_ptr(), b[1].stride(0), rows * b[1].stride(0)
        d.out, d.out_stride = out.data_ptr(), out.stride(0)
        return d

    d1, d2 = desc(N, H, xa, mats[0], h, 1), desc(H, N, ha, mats[1], y, 0)

    def step():
        quantize(x, lay.n_rows, H, xa, tok)
        wt.wt_mxfp4_product(d1, _stream())
        quantize(h, lay.n_rows, N, ha)
        wt.wt_mxfp4_product(d2, _stream())

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    own = lay.owned()
    for turn in range(3):
        x.copy_(torch.randn(T, H, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got_h, got_y = h.clone(), y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got_h, h) and torch.equal(got_y, y)
        xs = x.cpu()[token.long().clamp(min=0)]
        q1 = R.mx_round(xs)
        a = R.mx_values(R.mx_pack(q1[0]), q1[1])
        vals = []
        for w in (w1, w2):
            c, s = R.mx_round(w.view(-1, w.shape[2]))
            vals.append(R.mx_values(R.mx_pack(c), s)[:, : w.shape[2]].view(E, w.shape[1], -1))
        p, mag, k = R.product(R.NT, lay, a, vals[0])
        want = R.act(R.SILU, p[:, :N]) * p[:, N:]
        offp = R.sum_bound(k, mag)
        err = 1.2 * offp[:, :N] * (p[:, N:].abs() + offp[:, N:]) + R.act(R.SILU, p[:, :N]).abs() * offp[:, N:] + R.ACT * want.abs()
        _check("h", h, want, err + R.half_step(BF16) * (want.abs() + err) + 2.0 ** -133, own)
        # the second product from the h that the first one gave
        c, s = R.mx_round(h.cpu())
        yy, mag, k = R.product(R.NT, lay, R.mx_values(R.mx_pack(c), s), vals[1])
        _check("y", y, yy, R.bound(yy, mag, k, BF16), own)
