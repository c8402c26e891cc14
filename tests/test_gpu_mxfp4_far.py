"""MXFP4 weights of 2 GiB: a plain product's tiles start anywhere in them."""
import pytest
import torch

import expert_ref as R
from test_gpu_expert import F32, _fill, _gen, _stream
from test_gpu_mxfp4 import _random_mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    yield _wt
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [3, 200])
def test_weights_beyond_31_bits(wt, rows):
    n, k, g = 2 ** 18 + 8, 2 ** 14, _gen(rows)
    ac, asc = _random_mx(g, rows, k)
    some, some_scales = _random_mx(g, 1000, k)  # the weights' rows repeat
    gb, gbs = some.cuda().repeat(n // 1000 + 1, 1)[:n].contiguous(), some_scales.cuda().repeat(n // 1000 + 1, 1)[:n].contiguous()
    ga, gas, out = ac.cuda(), asc.cuda(), _fill((rows, n), F32)
    d = wt.wt_mxfp4_product_desc_init()
    d.n_rows, d.n, d.k, d.out_dtype = rows, n, k, wt.WT_DT_F32
    d.a, d.a_stride, d.a_scales, d.a_scale_stride = ga.data_ptr(), ga.stride(0), gas.data_ptr(), gas.stride(0)
    d.b, d.b_stride, d.b_scales, d.b_scale_stride = gb.data_ptr(), gb.stride(0), gbs.data_ptr(), gbs.stride(0)
    d.out, d.out_stride = out.data_ptr(), n
    wt.wt_mxfp4_product(d, _stream())
    torch.cuda.synchronize()
    a, b = R.mx_values(ac, asc).cuda(), R.mx_values(some, some_scales).cuda().t().contiguous()
    want, mag = a @ b, a.abs() @ b.abs()
    bound = R.sum_bound(k, mag) + R.half_step(F32) * want.abs()
    for at in range(0, n, 1000):
        part = out[:, at:at + 1000].double()
        assert bool(((part - want[:, : part.shape[1]]).abs() <= bound[:, : part.shape[1]]).all()), f"columns from {at} on"
