"""Products under every pair of scales: factors far beyond fp32's range meet as long as their product
lies inside, and a product outside is 0 or an infinity. One block, one code each, so that the values are exact."""
import math

import pytest
import torch

import expert_ref as R
from test_gpu_expert import F32, _fill, _stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


# 256 x 256 pairs; k of one block, and of many behind it whose codes are 0
@pytest.mark.parametrize("code_a,code_b", [(2, 2), (1, 7), (15, 1), (7, 7)])
@pytest.mark.parametrize("k", [1, 200])
def test_every_pair_of_scales(wt, k, code_a, code_b):
    nb = -(-k // 32)
    ac, bc = (torch.zeros(256, 16 * nb, dtype=torch.uint8) for _ in range(2))
    ac[:, 0], bc[:, 0] = code_a, code_b
    sc = torch.full((256, -(-nb // 4) * 4), 127, dtype=torch.uint8)
    sc[:, 0] = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    ga, gb, gs, out = ac.cuda(), bc.cuda(), sc.cuda(), _fill((256, 256), F32)
    d = wt.wt_mxfp4_product_desc_init()
    d.n_rows, d.n, d.k, d.out_dtype = 256, 256, k, wt.WT_DT_F32
    d.a, d.a_stride, d.b, d.b_stride = ga.data_ptr(), ga.stride(0), gb.data_ptr(), gb.stride(0)
    d.a_scales = d.b_scales = gs.data_ptr()
    d.a_scale_stride = d.b_scale_stride = gs.stride(0)
    d.out, d.out_stride = out.data_ptr(), 256
    wt.wt_mxfp4_product(d, _stream())
    torch.cuda.synchronize()
    a, b = R.mx_values(ac, sc[:, :nb])[:, :1], R.mx_values(bc, sc[:, :nb])[:, :1]
    want, got = a * b.t(), out.cpu().double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    top = torch.finfo(F32).max
    over, normal = want.abs() > top, (want.abs() >= 2.0 ** -126) & (want.abs() <= top)
    assert bool((got[normal] == want[normal]).all())
    assert torch.equal(got[over], torch.copysign(torch.full_like(want, math.inf), want)[over])
    # below the normal numbers a sum may be rounded to 0
    below = ~nan & ~over & ~normal
    assert bool(((got - want)[below].abs() <= 2.0 ** -126).all())
