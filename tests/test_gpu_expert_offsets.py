"""Offsets and counts that are not a row map's, as the header allows them: any numbers, cut to the row space."""
import pytest
import torch

import expert_ref as R
from test_gpu_expert import F32, _check, _fill, _gen, _normal, _operands, _place, _stream, _untouched

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _run(wt, form, n_rows, offsets, counts, seed, n=72, k=64):
    """(out, a, b) of a product over these tables."""
    g, E, d = _gen(seed), len(offsets) - 1, wt.wt_product_desc_init()
    a, b = _normal(g, n_rows, k), _normal(g, n_rows, n) if form == R.TN else _normal(g, E, *((n, k) if form == R.NT else (k, n)))
    out = _fill((E, k, n) if form == R.TN else (n_rows, n), F32)
    ga, gb, go = _place(a), _place(b), torch.tensor(offsets, dtype=torch.int32).cuda()
    gc = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    d.n_rows, d.n_experts, d.offsets, d.counts = n_rows, E, go.data_ptr(), gc.data_ptr() if gc is not None else None
    d.form, d.m, d.n, d.k, d.out_dtype = form, k, n, k, wt.WT_DT_F32
    _operands(d, ga, gb, out)
    wt.wt_expert_product(d, _stream())
    torch.cuda.synchronize()
    return out, a, b


def _cut(n_rows, offsets, counts):
    """First rows and ends, in numbers without an end."""
    spans = []
    for e in range(len(offsets) - 1):
        lo = offsets[e]
        hi = lo + max(0, offsets[e + 1] - lo if counts is None else counts[e])
        lo, hi = min(max(lo, 0), n_rows), min(max(hi, 0), n_rows)
        spans.append((lo, max(lo, hi)))
    return spans


TABLES = [([LOW, HIGH], None), ([-2 ** 30 - 5, 2 ** 30 + 7], None), ([LOW, LOW, 40, HIGH], None), ([20, LOW, HIGH, 3], None),
          ([LOW, 0, HIGH], [HIGH, 30, HIGH]), ([LOW, 5, 30], [LOW, HIGH])]


@pytest.mark.parametrize("offsets,counts", TABLES)
def test_offsets_are_any_numbers(wt, offsets, counts):
    n_rows = 60
    spans = _cut(n_rows, offsets, counts)
    owners = torch.zeros(n_rows, dtype=torch.int32)
    for lo, hi in spans:
        owners[lo:hi] += 1
    for form in (R.NT, R.NN, R.TN):
        out, a, b = _run(wt, form, n_rows, offsets, counts, seed=form)
        for e, (lo, hi) in enumerate(spans):
            x = a[lo:hi].double()
            if form == R.TN:
                y = b[lo:hi].double()
                want, mag = x.t() @ y, x.t().abs() @ y.abs()
                _check(f"expert {e}", out[e], want, R.bound(want, mag, max(1, hi - lo), F32))
            elif int(owners.sum()) <= n_rows:
                w = b[e].double().t() if form == R.NT else b[e].double()
                want, mag = x @ w, x.abs() @ w.abs()
                _check(f"expert {e}", out[lo:hi], want, R.bound(want, mag, 64, F32), (owners[lo:hi] == 1))
        if form != R.TN:
            _untouched("rows of no expert", out, owners == 0)


# name, n_rows, first rows and counts: one expert apart from those that overlap; the kernels of 16 x 64, 64 x 64, 128 x 128 and 256 x 256
OVERLAPS = [("within", 100, [0, 20, 60], [30, 20, 40]), ("few rows", 60, [0] * 6 + [40], [40] * 6 + [20]),
            ("64 rows", 700, [0] * 10 + [600], [600] * 10 + [100]), ("many", 9000, [0] * 10 + [8000], [8000] * 10 + [1000]),
            ("two of many", 9000, [0, 100, 8000], [8000, 7900, 1000])]


@pytest.mark.parametrize("name,n_rows,first,counts", OVERLAPS, ids=[o[0].replace(" ", "") for o in OVERLAPS])
@pytest.mark.parametrize("gated", [False, True])
def test_experts_that_overlap(wt, gated, name, n_rows, first, counts):
    """Rows of one expert hold its results or nothing new (where all experts' rows fit into n_rows: its results), rows of none
    nothing new, and nothing behind the rows is written."""
    n, k, E, g = 520, 64, len(counts), _gen(n_rows)
    a, b = _normal(g, n_rows, k), _normal(g, E, n * (1 + gated), k, std=0.2)
    buf = torch.full((n_rows + 64, n), -7.0, dtype=torch.bfloat16, device="cuda")
    ga, gb = _place(a), _place(b)
    off, cnt = torch.tensor(first + [0], dtype=torch.int32).cuda(), torch.tensor(counts, dtype=torch.int32).cuda()
    d = wt.wt_product_desc_init()
    d.n_rows, d.n_experts, d.offsets, d.counts = n_rows, E, off.data_ptr(), cnt.data_ptr()
    d.form, d.n, d.k, d.act = R.NT, n, k, R.SILU
    _operands(d, ga, gb, buf[:n_rows])
    if gated:
        wt.wt_gated_forward(d, 0, 0, _stream())
    else:
        wt.wt_expert_product(d, _stream())
    torch.cuda.synchronize()
    owners = torch.zeros(n_rows, dtype=torch.int32)
    for f, c in zip(first, counts):
        owners[f:f + c] += 1
    got = buf.cpu()
    assert bool((got[n_rows:] == -7).all()) and bool((got[:n_rows][owners == 0] == -7).all())
    for e, (f, c) in enumerate(zip(first, counts)):
        alone = torch.nonzero(owners[f:f + c] == 1)[:, 0] + f
        lay = R.Layout([len(alone)])
        if gated:
            want, bound = R.gated(lay, a[alone], b[e:e + 1], R.SILU)["h"]
        else:
            want, mag, terms = R.product(R.NT, lay, a[alone], b[e:e + 1])
            bound = R.bound(want, mag, terms, torch.bfloat16)
        right = (got[alone].double() - want).abs() <= bound
        assert bool((right | ((got[alone] == -7) if sum(counts) > n_rows else torch.zeros_like(right))).all()), f"expert {e}"
