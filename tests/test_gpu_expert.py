"""The experts' products and the gated block on the GPU against their definitions
in 64 bits (expert_ref): every form and type, sizes around the tiles, rows at
odd places, gathered rows, values that are not finite, captured and concurrent
calls, and the run of a whole step."""
import math

import pytest
import torch

import expert_ref as R
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FORMS = {"nt": R.NT, "nn": R.NN, "tn": R.TN}


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF16)


def _place(x, pad=0, shift=0, fill=math.nan):
    """x on the GPU as a view with `pad` elements behind each row and `shift` before the first, all of them `fill`."""
    rows, cols = x.shape[-2:]
    lead = x.shape[:-2]
    n = math.prod(lead) * rows * (cols + pad) + shift
    flat = torch.full((n + 64,), fill, dtype=x.dtype, device="cuda")
    v = flat[shift:n].view(*lead, rows, cols + pad)[..., :cols]
    v.copy_(x)
    return v


def _fill(shape, dtype, pad=0, shift=0):
    return _place(torch.full(shape, -7.0, dtype=dtype), pad, shift, -7.0)


def _rows(d, lay, keep, dense=False):
    d.n_rows, d.n_experts = lay.n_rows, len(lay.counts)
    if not dense:
        off, cnt = lay.offsets.cuda(), lay.counts_t.cuda()
        keep += [off, cnt]
        d.offsets, d.counts = off.data_ptr(), cnt.data_ptr()


def _operands(d, a, b, out, index=None, keep=None):
    d.a, d.a_stride = a.data_ptr(), a.stride(-2)
    d.b, d.b_stride = b.data_ptr(), b.stride(-2)
    d.out, d.out_stride = out.data_ptr(), out.stride(-2)
    if b.dim() == 3:
        d.b_expert_stride = b.stride(0)
    if out.dim() == 3:
        d.out_expert_stride = out.stride(0)
    if index is not None:
        i = index[0].cuda()
        keep.append(i)
        d.row_index, d.n_index_rows = i.data_ptr(), index[1]


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _check(name, got, want, bound, where=None):
    got, want, bound = got.double().cpu(), want.double(), bound.double()
    if where is not None:
        got, want, bound = got[where], want[where], bound[where]
    if got.numel() == 0:
        return
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN elsewhere"
    assert torch.equal(got[~finite & ~torch.isnan(want)], want[~finite & ~torch.isnan(want)]), f"{name}: infinities"
    off = (got - want).abs()[finite]
    allowed = bound[finite]
    if off.numel():
        worst = (off / allowed.clamp(min=1e-300)).max().item()
        log(f"  {name}: worst {worst:.3f} of the bound")
        assert bool((off <= allowed).all()), f"{name}: {worst} times the bound"


def _untouched(name, buf, where):
    assert bool((buf.cpu()[where] == -7.0).all()), f"{name}: written"


def _product(wt, form, lay, m, n, k, out_dtype, seed, pad=0, shift=0, index=None, dense=False, share=False):
    """Runs one product and checks it; index: (row numbers, rows)."""
    g, keep, d, E = _gen(seed), [], wt.wt_product_desc_init(), len(lay.counts)
    gathered = index[1] if index is not None else lay.n_rows
    if form == R.TN:
        a, b = _normal(g, lay.n_rows, m), _normal(g, gathered, n)
        out = _fill((E, m, n), out_dtype, pad, shift)
    else:
        a = _normal(g, gathered, k)
        b = _normal(g, 1 if share else E, *((n, k) if form == R.NT else (k, n)))
        out = _fill((lay.n_rows, n), out_dtype, pad, shift)
    ga, gb = _place(a, pad, shift), _place(b, pad, shift)
    _rows(d, lay, keep, dense)
    d.form, d.m, d.n, d.k = form, m, n, k
    d.out_dtype = wt.WT_DT_F32 if out_dtype == F32 else wt.WT_DT_BF16
    _operands(d, ga, gb, out, index, keep)
    if share:
        d.b_expert_stride = 0
        b = b.expand(E, -1, -1)
    wt.wt_expert_product(d, _stream())
    torch.cuda.synchronize()
    want, mag, terms = R.product(form, lay, a, b, index[0] if index is not None else None)
    where = None if form == R.TN else lay.owned()
    _check("product", out, want, R.bound(want, mag, terms, out_dtype), where)
    if where is not None:
        _untouched("rows of no expert", out, ~where)
    if pad:
        flat = torch.as_strided(out, (*out.shape[:-1], out.shape[-1] + pad), out.stride())
        _untouched("behind the rows", flat[..., out.shape[-1]:], slice(None))
    return out


UNEVEN = R.Layout([0, 1, 37, 0, 130, 16, 255, 3], align=16, lead=5, tail=9)
SIZES = [(128, 128, 64), (256, 256, 128), (8, 8, 8), (136, 264, 72), (40, 24, 200), (1, 1, 1), (3, 5, 7), (129, 131, 65),
         (130, 66, 190), (512, 136, 320)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_products_of_uneven_experts(wt, form, m, n, k):
    log(f"{form} {m}x{n}x{k}")
    for dtype in (BF16, F32):
        _product(wt, FORMS[form], UNEVEN, m, n, k, dtype, seed=m + n + k)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 700])
def test_products_of_a_dense_layer(wt, form, rows):
    log(f"{form} {rows} rows")
    _product(wt, FORMS[form], R.Layout([rows]), 264, 200, 136, BF16, seed=rows, dense=True)
    _product(wt, FORMS[form], R.Layout([rows]), 264, 200, 136, F32, seed=rows, dense=True, pad=8)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("pad,shift", [(8, 0), (2, 0), (1, 0), (0, 1), (8, 8), (3, 5), (8, 4), (4, 2)])
def test_strides_and_alignments(wt, form, pad, shift):
    log(f"{form} pad {pad} shift {shift}")
    # NaN lies behind every row: none of it may reach a sum
    for m, n, k in [(128, 136, 72), (72, 40, 101), (66, 130, 64)]:
        _product(wt, FORMS[form], UNEVEN, m, n, k, BF16, seed=11, pad=pad, shift=shift)
        _product(wt, FORMS[form], UNEVEN, m, n, k, F32, seed=12, pad=pad, shift=shift)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [1, 50])
def test_gathered_rows(wt, form, rows):
    g = _gen(rows)
    index = torch.randint(0, rows, (UNEVEN.n_rows,), generator=g, dtype=torch.int32)
    index[::13] = -1
    index[5::17] = rows
    index[7::19] = 2 ** 31 - 1
    index[3::23] = -2 ** 31
    for m, n, k in [(128, 136, 72), (72, 40, 101)]:
        for pad, shift in [(0, 0), (8, 0), (1, 1)]:
            _product(wt, FORMS[form], UNEVEN, m, n, k, BF16, seed=rows, index=(index, rows), pad=pad, shift=shift)


@pytest.mark.parametrize("form", FORMS)
def test_an_empty_source_of_rows_stands_for_zeros(wt, form):
    index = torch.zeros(UNEVEN.n_rows, dtype=torch.int32)
    _product(wt, FORMS[form], UNEVEN, 64, 72, 64, F32, seed=2, index=(index, 0))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("experts", [2, 63, 64, 65, 300, 1024])
def test_many_experts(wt, form, experts):
    g = _gen(experts)
    counts = torch.randint(0, 5, (experts,), generator=g).tolist()
    counts[experts // 2] = 140
    _product(wt, FORMS[form], R.Layout(counts, align=4, tail=3), 40, 48, 64, BF16, seed=experts)


def test_experts_that_share_weights(wt):
    _product(wt, R.NT, UNEVEN, 0, 72, 64, BF16, seed=3, share=True)
    _product(wt, R.NN, UNEVEN, 0, 72, 64, BF16, seed=3, share=True)


def test_no_rows_at_all(wt):
    lay = R.Layout([0, 0, 0])
    out = _product(wt, R.TN, lay, 40, 24, 0, F32, seed=1)
    assert bool((out == 0).all())
    lay = R.Layout([0, 0, 0], tail=20)
    _product(wt, R.NT, lay, 0, 24, 40, F32, seed=1)
    assert bool((_product(wt, R.TN, lay, 40, 24, 0, BF16, seed=1) == 0).all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("k", [4096, 7168])
def test_long_sums(wt, form, k):
    lay = R.Layout([k if form == "tn" else 70])
    _product(wt, FORMS[form], lay, 136, 72, k, F32, seed=k, dense=True)


def test_offsets_beyond_32_bits(wt):
    # 40 rows, 2^26 + 8 elements apart: the last starts at 5.2 GB
    g, far = _gen(9), 2 ** 26 + 8
    lay, keep = R.Layout([40]), []
    a, b = _normal(g, 40, 96), _normal(g, 1, 72, 96)
    buf = torch.zeros(39 * far + 96, dtype=BF16, device="cuda")
    va = torch.as_strided(buf, (40, 96), (far, 1))
    va.copy_(a)
    index = torch.arange(39, -1, -1, dtype=torch.int32)
    for use in (None, (index, 40)):
        d = wt.wt_product_desc_init()
        out, gb = _fill((40, 72), F32), _place(b)
        _rows(d, lay, keep, dense=True)
        d.form, d.n, d.k, d.out_dtype = R.NT, 72, 96, wt.WT_DT_F32
        _operands(d, va, gb, out, use, keep)
        wt.wt_expert_product(d, _stream())
        want, mag, k = R.product(R.NT, lay, a, b, use[0] if use else None)
        _check("far rows", out, want, R.bound(want, mag, k, F32))
        # as the rows of TN's operands
        d = wt.wt_product_desc_init()
        c, out = _normal(g, 40, 64), _fill((1, 64, 96), F32)
        gc = _place(c)
        _rows(d, lay, keep, dense=True)
        d.form, d.m, d.n, d.out_dtype = R.TN, 64, 96, wt.WT_DT_F32
        _operands(d, gc, va, out, use, keep)
        wt.wt_expert_product(d, _stream())
        want, mag, k = R.product(R.TN, lay, c, a, use[0] if use else None)
        _check("far rows as weights' gradient", out, want, R.bound(want, mag, k, F32))
    # as results
    out = torch.as_strided(buf, (40, 72), (far, 1))
    d = wt.wt_product_desc_init()
    ga = _place(a)
    _rows(d, lay, keep, dense=True)
    d.form, d.n, d.k = R.NT, 72, 96
    _operands(d, ga, gb, out, None, keep)
    wt.wt_expert_product(d, _stream())
    want, mag, k = R.product(R.NT, lay, a, b)
    _check("far results", out, want, R.bound(want, mag, k, BF16))


@pytest.mark.parametrize("form", FORMS)
def test_values_that_are_not_finite_stay_with_their_sums(wt, form):
    """A NaN or an infinity in an operand reaches the results whose sum it is part of, and no others."""
    f, lay, g = FORMS[form], R.Layout([70, 0, 130], align=16), _gen(4)
    m, n, k = 72, 136, 200
    if f == R.TN:
        a, b = _normal(g, lay.n_rows, m), _normal(g, lay.n_rows, n)
    else:
        a, b = _normal(g, lay.n_rows, k), _normal(g, 3, *((n, k) if f == R.NT else (k, n)))
    a[~lay.owned()] = math.nan  # rows of no expert
    if f == R.TN:
        b[~lay.owned()] = math.inf
    a[3, 5], a[100, 2], a[101, 3] = math.nan, math.inf, -math.inf
    (b if f == R.TN else b[0])[7, 9] = math.inf
    d, keep = wt.wt_product_desc_init(), []
    out = _fill((3, m, n) if f == R.TN else (lay.n_rows, n), F32)
    ga, gb = _place(a), _place(b)
    _rows(d, lay, keep)
    d.form, d.m, d.n, d.k, d.out_dtype = f, m, n, k, wt.WT_DT_F32
    _operands(d, ga, gb, out, None, keep)
    wt.wt_expert_product(d, _stream())
    torch.cuda.synchronize()
    want, mag, terms = R.product(f, lay, a, b)
    _check("not finite", out, want, R.bound(want, mag, terms, F32), None if f == R.TN else lay.owned())


def test_offsets_that_leave_the_rows_are_cut(wt):
    lay, g, keep = R.Layout([10, 20, 30]), _gen(5), []
    a, b = _normal(g, 60, 64), _normal(g, 5, 72, 64)
    offsets = torch.tensor([-5, 10, 30, 55, 100, 2 ** 31 - 1], dtype=torch.int32)
    counts = torch.tensor([15, 20, 20, 1000, 2 ** 31 - 1], dtype=torch.int32)
    d, out = wt.wt_product_desc_init(), _fill((60, 72), F32)
    ga, gb, go, gc = _place(a), _place(b), offsets.cuda(), counts.cuda()
    d.n_rows, d.n_experts, d.offsets, d.counts = 60, 5, go.data_ptr(), gc.data_ptr()
    d.form, d.n, d.k, d.out_dtype = R.NT, 72, 64, wt.WT_DT_F32
    _operands(d, ga, gb, out, None, keep)
    wt.wt_expert_product(d, _stream())
    # experts 0 .. 3 own [0, 10), [10, 30), [30, 50), [55, 60)
    cut = R.Layout([10, 20, 20])
    cut.n_rows = 60
    want, mag, k = R.product(R.NT, cut, a, b)
    want[55:], mag[55:] = a[55:].double() @ b[3].double().t(), a[55:].double().abs() @ b[3].double().abs().t()
    own = cut.owned()
    own[55:] = True
    _check("cut", out, want, R.bound(want, mag, k, F32), own)
    _untouched("between", out, ~own)


def test_without_counts(wt):
    counts = [3, 0, 40, 17]
    lay, g = R.Layout(counts), _gen(6)
    keep, a, b = [], _normal(g, 60, 64), _normal(g, 4, 72, 64)
    for f in (R.NT, R.TN):
        d = wt.wt_product_desc_init()
        ga, gb = _place(a), _place(b if f == R.NT else a)
        out = _fill((60, 72) if f == R.NT else (4, 64, 64), F32)
        _rows(d, lay, keep)
        d.counts = None
        d.form, d.m, d.n, d.k, d.out_dtype = f, 64, 72 if f == R.NT else 64, 64, wt.WT_DT_F32
        _operands(d, ga, gb, out, None, keep)
        wt.wt_expert_product(d, _stream())
        want, mag, k = R.product(f, lay, a, b if f == R.NT else a)
        _check("without counts", out, want, R.bound(want, mag, k, F32))


# ------------------------------------------------------------- gated block
def _gated(wt, lay, n, k, kind, seed, pad=0, shift=0, index=None, pre=True, dense=False):
    g, keep, d = _gen(seed), [], wt.wt_product_desc_init()
    x = _normal(g, index[1] if index is not None else lay.n_rows, k)
    w = _normal(g, len(lay.counts), 2 * n, k, std=2 * k ** -0.5)
    h, p = _fill((lay.n_rows, n), BF16, pad, shift), _fill((lay.n_rows, 2 * n), BF16, pad, shift)
    gx, gw = _place(x, pad, shift), _place(w, pad, shift)
    _rows(d, lay, keep, dense)
    d.form, d.n, d.k, d.act = R.NT, n, k, kind
    _operands(d, gx, gw, h, index, keep)
    wt.wt_gated_forward(d, p.data_ptr() if pre else 0, p.stride(0), _stream())
    torch.cuda.synchronize()
    want = R.gated(lay, x, w, kind, index[0] if index is not None else None)
    own = lay.owned()
    _check("h", h, *want["h"], own)
    _untouched("h", h, ~own)
    if pre:
        _check("pre", p, *want["pre"], own)
    _untouched("pre", p, ~own if pre else slice(None))


@pytest.mark.parametrize("kind", [R.SILU, R.GELU])
@pytest.mark.parametrize("n,k", [(64, 64), (128, 128), (8, 8), (136, 72), (24, 200), (1, 1), (5, 7), (131, 65), (66, 190), (256, 320)])
def test_gated_forward(wt, kind, n, k):
    log(f"{n} x {k}, activation {kind}")
    _gated(wt, UNEVEN, n, k, kind, seed=n + k)
    _gated(wt, UNEVEN, n, k, kind, seed=n + k, pre=False)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 129, 256, 300])
def test_gated_forward_of_a_dense_layer(wt, rows):
    _gated(wt, R.Layout([rows]), 264, 200, R.SILU, seed=rows, dense=True)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (8, 8), (4, 4), (2, 2)])
def test_gated_forward_strides_and_gathered_rows(wt, pad, shift):
    index = torch.randint(-1, 31, (UNEVEN.n_rows,), generator=_gen(8), dtype=torch.int32)
    for n, k in [(72, 136), (37, 75)]:
        _gated(wt, UNEVEN, n, k, R.SILU, seed=7, pad=pad, shift=shift)
        _gated(wt, UNEVEN, n, k, R.GELU, seed=7, pad=pad, shift=shift, index=(index, 30))


def _gated_back(wt, lay, n, k, kind, seed, pad=0, shift=0, dense=False):
    g, keep, d = _gen(seed), [], wt.wt_product_desc_init()
    dy, down = _normal(g, lay.n_rows, k), _normal(g, len(lay.counts), k, n, std=k ** -0.5)
    pre = _normal(g, lay.n_rows, 2 * n, std=2.0).clamp(-9, 9)
    out = _fill((lay.n_rows, 2 * n), BF16, pad, shift)
    gy, gd, gp = _place(dy, pad, shift), _place(down, pad, shift), _place(pre, pad, shift)
    _rows(d, lay, keep, dense)
    d.form, d.n, d.k, d.act = R.NN, n, k, kind
    _operands(d, gy, gd, out, None, keep)
    wt.wt_gated_backward(d, gp.data_ptr(), gp.stride(0), _stream())
    torch.cuda.synchronize()
    own = lay.owned()
    _check("dpre", out, *R.gated_back(lay, dy, down, pre, kind), own)
    _untouched("dpre", out, ~own)


@pytest.mark.parametrize("kind", [R.SILU, R.GELU])
@pytest.mark.parametrize("n,k", [(64, 64), (128, 128), (8, 8), (136, 72), (24, 200), (1, 1), (5, 7), (131, 65), (66, 190), (264, 320)])
def test_gated_backward(wt, kind, n, k):
    _gated_back(wt, UNEVEN, n, k, kind, seed=n + k)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (8, 8), (4, 4), (2, 2)])
def test_gated_backward_strides(wt, pad, shift):
    for n, k in [(72, 136), (37, 75)]:
        _gated_back(wt, UNEVEN, n, k, R.SILU, seed=3, pad=pad, shift=shift)
    _gated_back(wt, R.Layout([33]), 72, 136, R.GELU, seed=3, pad=pad, shift=shift, dense=True)


@pytest.mark.parametrize("kind", [R.SILU, R.GELU])
def test_activations_over_all_values(wt, kind):
    """Every BF16 value as gate: a product with a weight of 1, up = 1."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16).view(-1, 1)
    lay, keep, d = R.Layout([65536]), [], wt.wt_product_desc_init()
    rows = torch.cat([torch.where(torch.isfinite(x), x, torch.zeros_like(x)), torch.ones_like(x)], 1)
    w = torch.tensor([[[1.0, 0.0], [0.0, 1.0]]], dtype=BF16)
    h, pre, gx, gw = _fill((65536, 1), BF16), _fill((65536, 2), BF16), _place(rows), _place(w)
    _rows(d, lay, keep, dense=True)
    d.form, d.n, d.k, d.act = R.NT, 1, 2, kind
    _operands(d, gx, gw, h, None, keep)
    wt.wt_gated_forward(d, pre.data_ptr(), 2, _stream())
    torch.cuda.synchronize()
    g = rows[:, :1].double()
    want = R.act(kind, g)
    # the exponential of a large y is off by 2^-22 |y| relative; where it matters at all |y| < 90. One below 2^-126 may
    # become 0, times an x below 2^7
    tol = (R.half_step(BF16) + (4 * 90 + 8) * 2.0 ** -24) * want.abs() + 2.0 ** -119
    assert torch.equal(pre.cpu()[:, :1].double(), g)
    _check("values", h, want, tol)
    # the slope, by dh = 1: out = (up slope | value); infinities and NaN too
    p = torch.cat([x, torch.ones_like(x)], 1)
    one = torch.ones(1, 1, 1, dtype=BF16)
    d, out = wt.wt_product_desc_init(), _fill((65536, 2), BF16)
    gy, gd, gp = _place(torch.ones(65536, 1, dtype=BF16)), _place(one), _place(p)
    _rows(d, lay, keep, dense=True)
    d.form, d.n, d.k, d.act = R.NN, 1, 1, kind
    _operands(d, gy, gd, out, None, keep)
    wt.wt_gated_backward(d, gp.data_ptr(), 2, _stream())
    torch.cuda.synchronize()
    x = x.double()
    near = x.clamp(-700, 700)  # beyond, in 64 bits too, the slope is 0 or 1 and the value 0 or x
    slope, value = R.slope(kind, near), torch.where(x > 700, x, R.act(kind, near))
    slope, value = torch.where(torch.isnan(x), x, slope), torch.where(torch.isnan(x), x, value)
    hs = R.half_step(BF16)
    # near its zero the slope is a difference of terms below 1.2, each within ACT + 2^-23 of itself
    _check("slope", out[:, :1], slope, hs * slope.abs() + 2.4 * (R.ACT + 2.0 ** -23) + 2.0 ** -119)
    _check("value", out[:, 1:], value, (hs + (4 * 90 + 8) * 2.0 ** -24) * value.abs() + 2.0 ** -119)


def test_gradients_against_differences(wt):
    """The block's gradients against central differences of the block itself in 64 bits."""
    lay, g, n, k, keep = R.Layout([9, 0, 21], align=8), _gen(12), 24, 40, []
    x, w, down = _normal(g, lay.n_rows, k), _normal(g, 3, 2 * n, k, std=0.3), _normal(g, 3, k, n, std=0.3)
    dy = _normal(g, lay.n_rows, k)

    def loss(x, w):
        y, _, _ = R.product(R.NT, lay, x, w)
        z, _, _ = R.product(R.NT, lay, (R.act(R.SILU, y[:, :n]) * y[:, n:]).nan_to_num(), down.double())
        return (z * dy.double())[lay.owned()].sum()

    gx, gw, gd, gy = _place(x), _place(w), _place(down), _place(dy)
    h, pre = _fill((lay.n_rows, n), BF16), _fill((lay.n_rows, 2 * n), BF16)
    dpre, dx, dw = torch.zeros_like(pre), _fill((lay.n_rows, k), F32), _fill((3, 2 * n, k), F32)

    def desc(form, m, n, k, a, b, out):
        d = wt.wt_product_desc_init()
        _rows(d, lay, keep)
        d.form, d.m, d.n, d.k = form, m, n, k
        d.out_dtype = wt.WT_DT_F32 if out.dtype == F32 else wt.WT_DT_BF16
        _operands(d, a, b, out)
        return d

    wt.wt_gated_forward(desc(R.NT, 0, n, k, gx, gw, h), pre.data_ptr(), pre.stride(0), _stream())
    wt.wt_gated_backward(desc(R.NN, 0, n, k, gy, gd, dpre), pre.data_ptr(), pre.stride(0), _stream())
    wt.wt_expert_product(desc(R.NN, 0, k, 2 * n, dpre, gw, dx), _stream())
    wt.wt_expert_product(desc(R.TN, 2 * n, k, 0, dpre, gx, dw), _stream())
    torch.cuda.synchronize()
    x64, w64, step = x.double(), w.double(), 1e-4
    # what the gradients may be off by: pre and dpre are BF16, 2^-8 each on sums of these magnitudes (a change of pre
    # moves the slopes by at most 1.2 of itself); differences leave step^2
    dx_scale = dpre.double().abs().cpu().nan_to_num().amax() * w64.abs().sum(1).amax() * 2.0 ** -5
    for r, c in [(0, 0), (8, 39), (16, 3), (30, 17), (36, 1)]:
        up, lo = x64.clone(), x64.clone()
        up[r, c] += step
        lo[r, c] -= step
        want = (loss(up, w64) - loss(lo, w64)) / (2 * step)
        assert abs(dx[r, c].item() - want.item()) <= dx_scale
    for e, r, c in [(0, 0, 0), (0, 47, 39), (2, 5, 7), (2, 30, 1)]:
        up, lo = w64.clone(), w64.clone()
        up[e, r, c] += step
        lo[e, r, c] -= step
        want = (loss(x64, up) - loss(x64, lo)) / (2 * step)
        scale = dpre.double().cpu().abs()[lay.owned()].amax() * x64.abs().sum(0).amax() * 2.0 ** -5
        assert abs(dw[e, r, c].item() - want.item()) <= scale
    assert bool((dw[1] == 0).all())


# ----------------------------------------------------- repeats, graphs, streams
@pytest.mark.parametrize("form", FORMS)
def test_calls_repeat_bit_for_bit_and_replay(wt, form):
    f, lay, g, keep = FORMS[form], UNEVEN, _gen(21), []
    m, n, k = 136, 264, 320
    a = _normal(g, lay.n_rows, m if f == R.TN else k).cuda()
    b = (_normal(g, lay.n_rows, n) if f == R.TN else _normal(g, 8, *((n, k) if f == R.NT else (k, n)))).cuda()
    out = torch.zeros((8, m, n) if f == R.TN else (lay.n_rows, n), dtype=BF16, device="cuda")
    d = wt.wt_product_desc_init()
    off, cnt = lay.offsets.cuda(), lay.counts_t.cuda()
    d.n_rows, d.n_experts, d.offsets, d.counts = lay.n_rows, 8, off.data_ptr(), cnt.data_ptr()
    d.form, d.m, d.n, d.k = f, m, n, k
    _operands(d, a, b, out)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        wt.wt_expert_product(d, side.cuda_stream)
    side.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wt.wt_expert_product(d, torch.cuda.current_stream().cuda_stream)
    other = R.Layout([100, 3, 0, 70, 16, 2, 9, 40], align=16, lead=5)
    assert other.n_rows <= lay.n_rows
    for turn in range(4):  # the rows of the experts change between replays
        use = lay if turn % 2 == 0 else other
        off.copy_(use.offsets)
        cnt.copy_(use.counts_t)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        wt.wt_expert_product(d, _stream())
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        if turn % 2 == 0:
            own = slice(None) if f == R.TN else lay.owned().cuda()
            assert torch.equal(got[own], first[own])


def test_two_calls_at_once(wt):
    lay, g, keep = R.Layout([300, 200], align=1), _gen(22), []
    x, w = _normal(g, 500, 256), _normal(g, 2, 512, 256, std=0.1)
    want = R.gated(lay, x, w, R.SILU)["h"]
    gx, gw = _place(x), _place(w)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [_fill((500, 256), BF16) for _ in range(2)]
    off, cnt = lay.offsets.cuda(), lay.counts_t.cuda()
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            d = wt.wt_product_desc_init()
            d.n_rows, d.n_experts, d.offsets, d.counts = 500, 2, off.data_ptr(), cnt.data_ptr()
            d.form, d.n, d.k = R.NT, 256, 256
            _operands(d, gx, gw, o, None, keep)
            wt.wt_gated_forward(d, 0, 0, s.cuda_stream)
    torch.cuda.synchronize()
    for o in outs:
        _check("h", o, *want)


def test_a_step_from_logits_to_new_weights(wt):
    """Router, row map, gathered rows through the block and back, its gradients, the AdamW step on the experts' weights."""
    T, E, K, H, N = 150, 12, 3, 72, 40
    g = _gen(31)
    logits = torch.randn(T, E, generator=g).cuda()
    x, w, down = _normal(g, T, H).cuda(), _normal(g, E, 2 * N, H, std=0.2).cuda(), _normal(g, E, H, N, std=0.2).cuda()
    s = _stream()
    r = wt.wt_router_desc_init()
    r.n_tokens, r.n_experts, r.top_k, r.logits, r.logits_stride, r.normalize = T, E, K, logits.data_ptr(), E, 1
    index, weight = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    seq_counts, loss = torch.empty(1, E, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(wt.wt_router_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    wt.wt_router_forward(r, index.data_ptr(), weight.data_ptr(), 0, seq_counts.data_ptr(), loss.data_ptr(), ws.data_ptr(),
                         ws.numel(), s)
    align = 16
    n_rows = T * K + E * (align - 1)
    row_token = torch.empty(n_rows, dtype=torch.int32, device="cuda")
    pair_row = torch.empty(T, K, dtype=torch.int32, device="cuda")
    offsets, counts = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda")
    ws2 = torch.empty(wt.wt_dispatch_workspace_bytes(T, K, E), dtype=torch.uint8, device="cuda")
    wt.wt_dispatch_rows(index.data_ptr(), T, K, E, align, n_rows, row_token.data_ptr(), pair_row.data_ptr(),
                        offsets.data_ptr(), counts.data_ptr(), ws2.data_ptr(), ws2.numel(), s)

    def desc(form, m, n, k, a, b, out, gathers=False):
        d = wt.wt_product_desc_init()
        d.n_rows, d.n_experts, d.offsets, d.counts = n_rows, E, offsets.data_ptr(), counts.data_ptr()
        d.form, d.m, d.n, d.k = form, m, n, k
        _operands(d, a, b, out)
        if gathers:
            d.row_index, d.n_index_rows = row_token.data_ptr(), T
        return d

    h, pre = (torch.zeros(n_rows, c, dtype=BF16, device="cuda") for c in (N, 2 * N))
    y, dy, dx = (torch.zeros(n_rows, H, dtype=BF16, device="cuda") for _ in range(3))
    dpre, dw, ddown = torch.zeros_like(pre), torch.zeros_like(w), torch.zeros_like(down)
    wt.wt_gated_forward(desc(R.NT, 0, N, H, x, w, h, True), pre.data_ptr(), 2 * N, s)
    wt.wt_expert_product(desc(R.NT, 0, H, N, h, down, y), s)
    # the way back to the tokens, weighted, and a loss that is its sum of squares
    back = pair_row.long()
    z = (weight[:, :, None] * y[back].float()).sum(1)
    dz = 2 * z
    dy[back.flatten()] = (weight[:, :, None] * dz[:, None, :]).to(BF16).view(-1, H)
    wt.wt_gated_backward(desc(R.NN, 0, N, H, dy, down, dpre), pre.data_ptr(), 2 * N, s)
    wt.wt_expert_product(desc(R.NN, 0, H, 2 * N, dpre, w, dx), s)
    wt.wt_expert_product(desc(R.TN, 2 * N, H, 0, dpre, x, dw, True), s)
    wt.wt_expert_product(desc(R.TN, H, N, 0, dy, h, ddown), s)
    torch.cuda.synchronize()

    # token by token in 64 bits, from the selection that the router made
    x64, w64, d64 = (t.double().cpu().requires_grad_() for t in (x, w, down))
    wt64, idx = weight.double().cpu(), index.long().cpu()
    total = torch.zeros(T, H, dtype=torch.float64)
    for k in range(K):
        p = torch.einsum("th,tnh->tn", x64, w64[idx[:, k]])
        hh = R.act(R.SILU, p[:, :N]) * p[:, N:]
        total = total + wt64[:, k:k + 1] * torch.einsum("tn,thn->th", hh, d64[idx[:, k]])
    total.square().sum().backward()
    dtok = dx[back].double().sum(1).cpu()
    for name, got, want in [("z", z, total.detach()), ("dx", dtok, x64.grad), ("dw", dw, w64.grad), ("ddown", ddown, d64.grad)]:
        rel = ((got.double().cpu() - want).norm() / want.norm()).item()
        log(f"  {name}: {rel:.2e}")
        # a chain of at most 6 values rounded to BF16 (2^-8 each at most), in the norm
        assert rel < 6 * 2.0 ** -8
    # the optimizer on these gradients changes the weights that the next step reads
    m, v, m2, v2 = (torch.zeros(t.numel(), device="cuda") for t in (w, w, down, down))
    before = w.clone()
    tensors = [dict(param=t.data_ptr(), grad=gr.data_ptr(), grad_dtype=wt.WT_DT_BF16, m=a.data_ptr(), v=b.data_ptr(),
                    n=t.numel(), lr_mul=1.0, weight_decay=0.0) for t, gr, a, b in ((w, dw, m, v), (down, ddown, m2, v2))]
    with wt.AdamW(tensors) as opt:
        hyper = wt.wt_adamw_hyper_init()
        hyper.step = 1
        opt.step(hyper, s)
        torch.cuda.synchronize()
    moved = (w != before).float()
    assert moved[dw != 0].mean() > 0.5 and not bool(moved[dw == 0].any())
