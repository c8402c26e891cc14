"""The AdamW step's host side on the CPU: defaults, the table's validation and
shape, and the refusals of hyper values. No GPU call is made here."""
import math

import pytest


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _t(wt, **kw):
    d = dict(param=0x100000, master=0x200000, grad=0x300000, m=0x400000, v=0x500000, m_scale=0x600000,
             v_scale=0x700000, n=1000, grad_dtype=wt.WT_DT_BF16)
    d.update(kw)
    return d


def _status(wt, tensors, bits=32):
    o = wt.wt_adamw_options_init()
    o.state_bits = bits
    try:
        wt.wt_adamw_check(wt.AdamWTable(tensors), o)
        return 0
    except wt.WtError as e:
        assert len(str(e)) > 20
        return e.status


def test_defaults(wt):
    o, h = wt.wt_adamw_options_init(), wt.wt_adamw_hyper_init()
    assert (o.state_bits, o.device) == (32, -1)
    assert (h.lr, h.beta1, h.beta2, h.eps, h.grad_scale, h.max_norm, h.step) == (1e-3, 0.9, 0.999, 1e-8, 1.0, 0.0, 1)
    assert not h.step_dev and not h.lr_dev and not h.norm_out


def test_shape(wt):
    info = wt.wt_adamw_check(wt.AdamWTable([_t(wt), {"n": 0}, _t(wt, param=0x1100002, master=0x1200000, grad=0x1300000,
                                                                  m=0x1400000, v=0x1500000, n=4097)]))
    assert info["n_tensors"] == 2 and info["n_elements"] == 5097 and info["n_blocks"] == 8 + 33
    assert info["n_items"] == 1 + 2 and info["n_vector_tensors"] == 1 and info["table_bytes"] > 0


@pytest.mark.parametrize("bits", [32, 8])
def test_refusals(wt, bits):
    E = wt
    assert _status(wt, [_t(wt)], bits) == 0
    assert _status(wt, [], bits) == E.WT_E_INVAL
    for k in ("grad", "m", "v"):
        assert _status(wt, [_t(wt, **{k: 0})], bits) == E.WT_E_INVAL
    assert _status(wt, [_t(wt, param=0)], bits) == 0
    assert _status(wt, [_t(wt, master=0)], bits) == 0
    assert _status(wt, [_t(wt, param=0, master=0)], bits) == E.WT_E_INVAL
    for k in ("m_scale", "v_scale"):
        assert _status(wt, [_t(wt, **{k: 0})], bits) == (E.WT_E_INVAL if bits == 8 else 0)
    assert _status(wt, [_t(wt, n=-1)], bits) == E.WT_E_INVAL
    assert _status(wt, [_t(wt, n=1 << 47)], bits) == E.WT_E_INVAL
    assert _status(wt, [_t(wt, grad_dtype=2)], bits) == E.WT_E_INVAL
    for k in ("lr_mul", "weight_decay"):
        for x in (-1.0, math.nan, math.inf, 2e6):
            assert _status(wt, [_t(wt, **{k: x})], bits) == E.WT_E_INVAL
    assert _status(wt, [_t(wt, param=0x100001)], bits) == E.WT_E_ALIGN
    assert _status(wt, [_t(wt, master=0x200002)], bits) == E.WT_E_ALIGN
    assert _status(wt, [_t(wt, grad=0x300001)], bits) == E.WT_E_ALIGN
    assert _status(wt, [_t(wt, grad=0x300002, grad_dtype=wt.WT_DT_F32)], bits) == E.WT_E_ALIGN
    assert _status(wt, [_t(wt, m=0x400001)], bits) == (E.WT_E_ALIGN if bits == 32 else 0)
    assert _status(wt, [_t(wt, v_scale=0x700002)], bits) == (E.WT_E_ALIGN if bits == 8 else 0)
    assert _status(wt, [_t(wt, master=(1 << 64) - 16)], bits) == E.WT_E_RANGE
    assert _status(wt, [_t(wt)], 16) == E.WT_E_INVAL


@pytest.mark.parametrize("bits", [32, 8])
def test_more_elements_than_a_launch_holds(wt, bits):
    # a thread updates eight elements, and a launch holds fewer than 2^32 threads
    big = dict(param=1 << 44, master=0, grad=2 << 44, m=3 << 44, v=4 << 44, m_scale=5 << 44, v_scale=6 << 44)
    assert _status(wt, [_t(wt, n=2 ** 35, **big)], bits) == wt.WT_E_INVAL
    with pytest.raises(wt.WtError, match="too many elements"):
        o = wt.wt_adamw_options_init()
        o.state_bits = bits
        wt.wt_adamw_check(wt.AdamWTable([_t(wt, n=2 ** 35, **big)]), o)


def test_overlaps(wt):
    E = wt
    base = 0x100000
    # param ends where the master starts: fine; one element into it: not
    assert _status(wt, [_t(wt, param=base, master=base + 2000)]) == 0
    assert _status(wt, [_t(wt, param=base, master=base + 1996)]) == E.WT_E_OVERLAP
    # a gradient may be shared, not written over
    far = dict(param=0x1100000, master=0x1200000, m=0x1400000, v=0x1500000)
    assert _status(wt, [_t(wt), _t(wt, **far)]) == 0
    assert _status(wt, [_t(wt), _t(wt, **dict(far, m=0x300000 + 400))]) == E.WT_E_OVERLAP
    assert _status(wt, [_t(wt), _t(wt, **dict(far, grad=0x400000 + 8))]) == E.WT_E_OVERLAP
    assert _status(wt, [_t(wt), _t(wt)]) == E.WT_E_OVERLAP
    # a long range hides a short one behind it
    assert _status(wt, [_t(wt, grad=0x300000, n=100000, m=0x8000000, v=0x9000000, param=0x300000 + 150000,
                           master=0xa000000)]) == E.WT_E_OVERLAP
    assert "overlaps" in wt.wt_plan_last_error(None)


def test_create_refuses_before_touching_a_gpu(wt):
    with pytest.raises(wt.WtError) as e:
        wt.AdamW([_t(wt, param=0, master=0)])
    assert e.value.status == wt.WT_E_INVAL
    with pytest.raises(wt.WtError) as e:
        wt.wt_adamw_step(0, wt.wt_adamw_hyper_init())
    assert e.value.status == wt.WT_E_INVAL
    with pytest.raises(wt.WtError):
        wt.wt_adamw_get_info(0)
    wt.wt_adamw_destroy(0)
