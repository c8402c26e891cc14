"""Every kernel of the experts' products against the definitions in 64 bits, each at sizes that
take it (test_expert_choice holds them to that) and that end rows, columns and sums at odd places."""
import pytest

import expert_kernels as K
import expert_ref as R
import test_gpu_expert_tiles as tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


@pytest.mark.parametrize("case", K.PRODUCTS, ids=K.name)
@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("gathered", [False, True])
def test_products(wt, form, gathered, case):
    kernel, lay, n, k = case
    tiles.test_products(wt, form, gathered, kernel, lay, n, k)


@pytest.mark.parametrize("case", K.GRADIENTS, ids=K.name)
@pytest.mark.parametrize("gathered", [False, True])
def test_gradients_of_weights(wt, gathered, case):
    _, lay, m, n = case
    tiles.test_gradients_of_weights(wt, gathered, m, n, lay)


@pytest.mark.parametrize("case", K.GATED, ids=K.name)
@pytest.mark.parametrize("act", [R.SILU, R.GELU])
def test_gated_forward_and_backward(wt, act, case):
    forward, back, lay, n, k = case
    assert n % 2 == 0  # the number of columns is rounded down to an even one there
    tiles.test_gated(wt, act, f"{forward}, back {back}", lay, 2 * n, k)


@pytest.mark.parametrize("case", K.MXFP4, ids=K.name)
@pytest.mark.parametrize("gated", [False, True])
def test_mxfp4_products(wt, gated, case):
    kernel, lay, n, k = case
    assert n % 4 == 0
    tiles.test_mxfp4_products(wt, gated, kernel, lay, n, k)
