"""Refusals of the experts' products and of MXFP4 on the CPU: every call here
returns before anything is launched."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

A = 0x100000  # an address that nothing reads


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _desc(wt, **kw):
    d = wt.wt_product_desc_init()
    for k, v in dict(dict(n_rows=100, n_experts=4, form=wt.WT_PRODUCT_NT, offsets=A, counts=A, m=24, n=40, k=48, a=A,
                          a_stride=64, b=A, b_stride=64, b_expert_stride=64 * 80, out=A, out_stride=96,
                          out_expert_stride=64 * 96), **kw).items():
        setattr(d, k, v)
    return d


def _mx(wt, **kw):
    d = wt.wt_mxfp4_product_desc_init()
    for k, v in dict(dict(n_rows=100, n_experts=4, offsets=A, counts=A, n=40, k=70, a=A, a_stride=48, a_scales=A,
                          a_scale_stride=4, b=A, b_stride=48, b_expert_stride=48 * 80, b_scales=A, b_scale_stride=4,
                          b_scale_expert_stride=4 * 80, out=A, out_stride=40), **kw).items():
        setattr(d, k, v)
    return d


def _refused(wt, status, f, *a):
    with pytest.raises(wt.WtError) as e:
        f(*a)
    assert e.value.status == status, str(e.value)
    assert str(e.value).count(":") >= 2  # names the call and the reason


def test_defaults_and_null(wt):
    d = wt.wt_product_desc_init()
    assert (d.n_experts, d.out_dtype, d.form, d.act) == (1, wt.WT_DT_BF16, wt.WT_PRODUCT_NT, wt.WT_ACT_SILU)
    m = wt.wt_mxfp4_product_desc_init()
    assert (m.n_experts, m.out_dtype, m.gated) == (1, wt.WT_DT_BF16, 0)
    wt.lib.wt_product_desc_init(None)
    wt.lib.wt_mxfp4_product_desc_init(None)
    assert wt.lib.wt_expert_product(None, None) == wt.WT_E_INVAL
    assert wt.lib.wt_gated_forward(None, None, 0, None) == wt.WT_E_INVAL
    assert wt.lib.wt_gated_backward(None, None, 0, None) == wt.WT_E_INVAL
    assert wt.lib.wt_mxfp4_product(None, None) == wt.WT_E_INVAL


def test_structs_match_the_header(wt, tmp_path):
    structs = [wt.wt_product_desc, wt.wt_mxfp4_product_desc]
    lines = [f'printf("%zu ", offsetof({s.__name__}, {f}));' for s in structs for f, _ in s._fields_]
    lines += [f'printf("%zu ", sizeof({s.__name__}));' for s in structs]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "wt.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    said = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert said == [getattr(s, f).offset for s in structs for f, _ in s._fields_] + [ctypes.sizeof(s) for s in structs]


BAD = [("n_rows", -1), ("n_rows", 2 ** 27 + 1), ("n_experts", 0), ("n_experts", 1025), ("form", 3), ("form", -1),
       ("offsets", None), ("n", 0), ("n", 2 ** 24 + 1), ("k", 0), ("k", 2 ** 24 + 1), ("a_stride", 47), ("b_stride", 47),
       ("out_stride", 39), ("out_stride", 2 ** 60), ("a_stride", 2 ** 58), ("b_expert_stride", -8),
       ("b_expert_stride", 2 ** 60), ("a", None), ("b", None), ("out", None), ("out_dtype", 2)]


@pytest.mark.parametrize("field,value", BAD)
def test_products_refused(wt, field, value):
    _refused(wt, wt.WT_E_INVAL, wt.wt_expert_product, _desc(wt, **{field: value}))
    _refused(wt, wt.WT_E_INVAL, wt.wt_gated_forward, _desc(wt, **{field: value}), A, 80)


@pytest.mark.parametrize("field,value", [("m", 0), ("m", 2 ** 24 + 1), ("a_stride", 23), ("b_stride", 39),
                                         ("out_stride", 39), ("out_expert_stride", 23 * 96 + 39),
                                         ("out_expert_stride", 2 ** 60), ("out", None), ("a", None), ("b", None)])
def test_gradients_of_weights_refused(wt, field, value):
    _refused(wt, wt.WT_E_INVAL, wt.wt_expert_product, _desc(wt, form=wt.WT_PRODUCT_TN, **{field: value}))


@pytest.mark.parametrize("field,value", [("k", 0), ("a_stride", 47), ("b_stride", 39), ("out_stride", 39)])
def test_gradients_of_rows_refused(wt, field, value):
    _refused(wt, wt.WT_E_INVAL, wt.wt_expert_product, _desc(wt, form=wt.WT_PRODUCT_NN, **{field: value}))


def test_gated_refusals(wt):
    nt, nn, tn = wt.WT_PRODUCT_NT, wt.WT_PRODUCT_NN, wt.WT_PRODUCT_TN
    for form in (nn, tn):
        _refused(wt, wt.WT_E_INVAL, wt.wt_gated_forward, _desc(wt, form=form), A, 80)
    for form in (nt, tn):
        _refused(wt, wt.WT_E_INVAL, wt.wt_gated_backward, _desc(wt, form=form), A, 80)
    for field, value in [("act", 2), ("act", -1), ("out_dtype", wt.WT_DT_F32)]:
        _refused(wt, wt.WT_E_INVAL, wt.wt_gated_forward, _desc(wt, **{field: value}), A, 80)
        _refused(wt, wt.WT_E_INVAL, wt.wt_gated_backward, _desc(wt, form=nn, **{field: value}), A, 80)
    _refused(wt, wt.WT_E_INVAL, wt.wt_gated_forward, _desc(wt), A, 79)
    _refused(wt, wt.WT_E_INVAL, wt.wt_gated_backward, _desc(wt, form=nn), A, 79)
    _refused(wt, wt.WT_E_INVAL, wt.wt_gated_backward, _desc(wt, form=nn), 0, 80)
    _refused(wt, wt.WT_E_INVAL, wt.wt_gated_backward, _desc(wt, form=nn, out_stride=79), A, 80)  # 2 n columns
    _refused(wt, wt.WT_E_ALIGN, wt.wt_gated_forward, _desc(wt), A + 1, 80)


@pytest.mark.parametrize("field", ["a", "b", "out"])
def test_misaligned_addresses_refused(wt, field):
    _refused(wt, wt.WT_E_ALIGN, wt.wt_expert_product, _desc(wt, **{field: A + 1}))
    if field == "out":
        _refused(wt, wt.WT_E_ALIGN, wt.wt_expert_product, _desc(wt, out=A + 2, out_dtype=wt.WT_DT_F32))


@pytest.mark.parametrize("field", ["offsets", "counts", "row_index"])
def test_misaligned_tables_refused(wt, field):
    _refused(wt, wt.WT_E_ALIGN, wt.wt_expert_product, _desc(wt, n_index_rows=4, **{field: A + 2}))


def test_row_index_and_counts(wt):
    for n in (-1, 2 ** 31):
        _refused(wt, wt.WT_E_INVAL, wt.wt_expert_product, _desc(wt, row_index=A, n_index_rows=n))
    _refused(wt, wt.WT_E_INVAL, wt.wt_expert_product, _desc(wt, n_experts=1, offsets=None))  # counts without offsets


def test_nothing_to_do(wt):
    wt.wt_expert_product(_desc(wt, n_rows=0, a=None, out=None))
    wt.wt_expert_product(_desc(wt, n_rows=0, form=wt.WT_PRODUCT_NN))
    wt.wt_gated_forward(_desc(wt, n_rows=0), 0, 0)
    wt.wt_gated_backward(_desc(wt, n_rows=0, form=wt.WT_PRODUCT_NN), 0, 0)
    wt.wt_mxfp4_product(_mx(wt, n_rows=0, a=None, out=None))


def test_more_tiles_than_a_grid(wt):
    big = dict(n_rows=2 ** 27, n=2 ** 24, out_stride=2 ** 24, b_expert_stride=0)
    _refused(wt, wt.WT_E_INVAL, wt.wt_expert_product, _desc(wt, **big))
    big.pop("b_expert_stride")
    _refused(wt, wt.WT_E_INVAL, wt.wt_mxfp4_product, _mx(wt, **big))


@pytest.mark.parametrize("field,value", [
    ("n_rows", -1), ("n_rows", 2 ** 27 + 1), ("n_experts", 0), ("n_experts", 1025), ("offsets", None), ("gated", 2),
    ("n", 0), ("k", 0), ("n", 2 ** 24 + 1), ("a_stride", 32), ("b_stride", 32), ("a_scale_stride", 0), ("b_scale_stride", 2),
    ("out_stride", 39), ("b_expert_stride", -16), ("b_scale_expert_stride", -4), ("a", None), ("b", None),
    ("a_scales", None), ("b_scales", None), ("out", None), ("out_dtype", 2)])
def test_mxfp4_products_refused(wt, field, value):
    _refused(wt, wt.WT_E_INVAL, wt.wt_mxfp4_product, _mx(wt, **{field: value}))


def test_mxfp4_gated_and_alignment(wt):
    _refused(wt, wt.WT_E_INVAL, wt.wt_mxfp4_product, _mx(wt, gated=1, act=2))
    _refused(wt, wt.WT_E_INVAL, wt.wt_mxfp4_product, _mx(wt, gated=1, out_dtype=wt.WT_DT_F32))
    for field, value in [("a", A + 8), ("b", A + 4), ("a_stride", 56), ("b_stride", 52), ("b_expert_stride", 8),
                         ("a_scales", A + 2), ("b_scales", A + 1), ("a_scale_stride", 5), ("b_scale_stride", 6),
                         ("b_scale_expert_stride", 2), ("out", A + 1), ("offsets", A + 1)]:
        _refused(wt, wt.WT_E_ALIGN, wt.wt_mxfp4_product, _mx(wt, **{field: value}))


def test_rounding_refusals(wt):
    good = dict(x=A, dtype=0, n_rows=10, cols=70, x_row_stride=70, row_index=0, n_out=10, codes=A, code_row_stride=48,
                scales=A, scale_row_stride=3)
    for field, value in [("dtype", 2), ("n_rows", -1), ("n_out", -1), ("cols", 0), ("cols", 2 ** 31), ("x_row_stride", 69),
                         ("x_row_stride", 2 ** 60), ("code_row_stride", 44), ("scale_row_stride", 2), ("x", 0), ("codes", 0),
                         ("scales", 0), ("n_out", 2 ** 30)]:
        _refused(wt, wt.WT_E_INVAL, wt.wt_mxfp4_quantize, *dict(good, **{field: value}).values())
    for field, value in [("x", A + 2), ("row_index", A + 2), ("codes", A + 2), ("code_row_stride", 50)]:
        _refused(wt, wt.WT_E_ALIGN, wt.wt_mxfp4_quantize, *dict(good, **{field: value}).values())
    wt.wt_mxfp4_quantize(*dict(good, n_out=0, x=0, codes=0).values())
    good = dict(codes=A, code_row_stride=48, scales=A, scale_row_stride=3, n_rows=10, cols=70, out=A, dtype=1,
                out_row_stride=70)
    for field, value in [("dtype", -1), ("n_rows", -1), ("cols", 0), ("out_row_stride", 69), ("code_row_stride", 32),
                         ("scale_row_stride", 1), ("codes", 0), ("scales", 0), ("out", 0), ("n_rows", 2 ** 30)]:
        _refused(wt, wt.WT_E_INVAL, wt.wt_mxfp4_dequantize, *dict(good, **{field: value}).values())
    for field, value in [("out", A + 1), ("codes", A + 1), ("code_row_stride", 54)]:
        _refused(wt, wt.WT_E_ALIGN, wt.wt_mxfp4_dequantize, *dict(good, **{field: value}).values())
    wt.wt_mxfp4_dequantize(*dict(good, n_rows=0, out=0).values())
