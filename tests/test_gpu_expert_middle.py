"""Sizes between those of test_gpu_expert_tiles: they reach the kernels of 64 x 128
tiles, MXFP4's of 64 rows whose waves split the sum, and with odd sizes the larger
tiles of operands at any alignment."""
import pytest

import expert_ref as R
import test_gpu_expert as whole
import test_gpu_expert_tiles as tiles

pytestmark = pytest.mark.gpu

SHAPES = [("64 x 128", R.Layout([701]), 2002, 202), ("64 x 128, experts", R.Layout([300, 0, 257, 65, 64, 1], lead=1, tail=70), 1102, 998),
          ("64 x 128, few steps", R.Layout([1024]), 2048, 30), ("odd", R.Layout([2101]), 2103, 133),
          ("odd, experts", tiles.EIGHT, 3333, 71)]
IDS = [s[0].replace(" ", "") for s in SHAPES]
MX_SHAPES = [("64, split", R.Layout([500]), 2002, 1000), ("64, experts", R.Layout([100, 0, 77, 200, 65, 64], lead=2, tail=40), 1030, 3000),
             ("64, few steps", R.Layout([512]), 2048, 33)]


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


@pytest.mark.parametrize("name,lay,n,k", SHAPES, ids=IDS)
@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("gathered", [False, True])
def test_products(wt, form, gathered, name, lay, n, k):
    tiles.test_products(wt, form, gathered, name, lay, n, k)


@pytest.mark.parametrize("m,n,lay", [(702, 2000, R.Layout([300])), (260, 1002, R.Layout([100, 0, 33, 700])), (1024, 2048, R.Layout([31])),
                                     (2101, 2049, R.Layout([77])), (801, 777, R.Layout([65, 0, 500, 64, 1, 129]))])
@pytest.mark.parametrize("gathered", [False, True])
def test_gradients_of_weights(wt, gathered, m, n, lay):
    tiles.test_gradients_of_weights(wt, gathered, m, n, lay)


@pytest.mark.parametrize("name,lay,n,k", SHAPES, ids=IDS)
@pytest.mark.parametrize("act", [R.SILU, R.GELU])
def test_gated(wt, act, name, lay, n, k):
    tiles.test_gated(wt, act, name, lay, n, k)


@pytest.mark.parametrize("name,lay,n,k", MX_SHAPES, ids=[s[0].replace(" ", "") for s in MX_SHAPES])
@pytest.mark.parametrize("gated", [False, True])
def test_mxfp4_products(wt, gated, name, lay, n, k):
    tiles.test_mxfp4_products(wt, gated, name, lay, n, k)


@pytest.mark.parametrize("lay,n,k", [(R.Layout([3, 0, 5]), 131, 62), (whole.UNEVEN, 131, 64), (R.Layout([300]), 1001, 66),
                                     (R.Layout([700]), 1001, 66), (R.Layout([1030]), 2811, 34), (R.Layout([4100]), 2051, 34)])
@pytest.mark.parametrize("act", [R.SILU, R.GELU])
def test_gated_with_an_odd_number_of_columns_and_an_even_sum(wt, act, lay, n, k):
    whole._gated(wt, lay, n, k, act, seed=n, dense=len(lay.counts) == 1)


@pytest.mark.parametrize("lay,n,k", [(R.Layout([3, 0, 5]), 131, 62), (whole.UNEVEN, 131, 64), (R.Layout([1030]), 4811, 34)])
def test_products_with_an_odd_number_of_columns_and_an_even_sum(wt, lay, n, k):
    for dtype in (whole.BF16, whole.F32):
        whole._product(wt, R.NT, lay, 0, n, k, dtype, seed=n, dense=len(lay.counts) == 1)


@pytest.mark.parametrize("n,k", [(1 << 24, 2), (2, 1 << 24)])
def test_the_longest_rows_and_sums(wt, n, k):
    """Two rows of ones and -1 over weights of one element: sums of integers below 2^24, exact in fp32."""
    import torch
    a = torch.ones(2, k, dtype=torch.bfloat16, device="cuda")
    a[1] = -1
    b = torch.ones(n, k, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(2, n, device="cuda")
    d = wt.wt_product_desc_init()
    d.n_rows, d.form, d.n, d.k, d.out_dtype = 2, R.NT, n, k, wt.WT_DT_F32
    d.a, d.a_stride, d.b, d.b_stride, d.out, d.out_stride = a.data_ptr(), k, b.data_ptr(), k, out.data_ptr(), n
    wt.wt_expert_product(d, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert bool((out[0] == k).all()) and bool((out[1] == -k).all())
