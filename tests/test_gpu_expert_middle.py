"""Sizes between those of test_gpu_expert_tiles: they reach the kernels of 64 x 128
tiles, MXFP4's of 64 rows whose waves split the sum, and with odd sizes the larger
tiles of operands at any alignment."""
import pytest

import expert_ref as R
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
