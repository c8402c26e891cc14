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
