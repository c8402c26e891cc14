"""Refusals and sizes of the router's and the row map's calls on the CPU: every
call here returns before anything is launched."""
import math

import pytest

A = 0x100000  # an address that nothing reads


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _desc(wt, **kw):
    d = wt.wt_router_desc_init()
    for k, v in dict(dict(n_tokens=100, n_experts=48, top_k=4, logits=A, logits_stride=48, seq_offsets=A, n_seqs=2,
                          balance_coef=0.01), **kw).items():
        setattr(d, k, v)
    return d


def _refused(wt, status, f, *a):
    with pytest.raises(wt.WtError) as e:
        f(*a)
    assert e.value.status == status, str(e.value)
    assert str(e.value).count(":") >= 2  # names the call and the reason


BAD_DESC = [("n_tokens", -1), ("n_tokens", 2 ** 31 // 4), ("n_experts", 0), ("n_experts", 1025), ("top_k", 0),
            ("top_k", 33), ("top_k", 49), ("logits_dtype", 2), ("score", 2), ("normalize", 2), ("scale", math.nan),
            ("scale", math.inf), ("balance_coef", math.inf), ("n_seqs", 0), ("n_seqs", 2 ** 20 + 1),
            ("seq_offsets", None)]


def test_defaults(wt):
    d = wt.wt_router_desc_init()
    assert (d.top_k, d.n_seqs, d.scale, d.score, d.normalize) == (1, 1, 1.0, wt.WT_SCORE_SIGMOID, 0)


@pytest.mark.parametrize("field,value", BAD_DESC)
def test_descriptions_refused(wt, field, value):
    d = _desc(wt, **{field: value})
    _refused(wt, wt.WT_E_INVAL, wt.wt_router_workspace_bytes, d)
    _refused(wt, wt.WT_E_INVAL, wt.wt_router_forward, d, A, A, A, A, A, A, 1 << 40)
    _refused(wt, wt.WT_E_INVAL, wt.wt_router_backward, d, A, A, A, A, A, 48)


def test_more_tokens_than_a_launch_holds(wt):
    # one place per token: index and weight would still have 32-bit sizes, the grid and the token numbers not
    assert wt.wt_router_workspace_bytes(_desc(wt, n_tokens=2 ** 27, top_k=1)) > 2 ** 27
    for n in (2 ** 27 + 1, 2 ** 31 - 1):
        _refused(wt, wt.WT_E_INVAL, wt.wt_router_workspace_bytes, _desc(wt, n_tokens=n, top_k=1))
        _refused(wt, wt.WT_E_INVAL, wt.wt_router_backward, _desc(wt, n_tokens=n, top_k=1), A, A, A, A, A, 48)


def test_forward_refusals(wt):
    n = wt.wt_router_workspace_bytes(_desc(wt))
    assert 0 < n < 1 << 20

    def f(status, d=None, **kw):
        a = dict(index=A, weight=A, counts=A, seq_counts=A, loss=A, workspace=A, workspace_bytes=n)
        a.update(kw)
        _refused(wt, status, wt.wt_router_forward, d or _desc(wt), *a.values())

    for k in ("index", "weight", "seq_counts", "loss", "workspace"):
        f(wt.WT_E_INVAL, **{k: 0})
    for k in ("index", "weight", "counts", "seq_counts", "loss"):
        f(wt.WT_E_ALIGN, **{k: A + 2})
    f(wt.WT_E_ALIGN, workspace=A + 8)
    f(wt.WT_E_RANGE, workspace_bytes=n - 1)
    f(wt.WT_E_INVAL, _desc(wt, logits=None))
    f(wt.WT_E_INVAL, _desc(wt, logits_stride=47))
    f(wt.WT_E_INVAL, _desc(wt, logits_stride=2 ** 60 // 100 + 1))
    f(wt.WT_E_ALIGN, _desc(wt, logits=A + 2))
    f(wt.WT_E_ALIGN, _desc(wt, logits=A + 1, logits_dtype=wt.WT_DT_BF16))
    f(wt.WT_E_ALIGN, _desc(wt, bias=A + 1))
    f(wt.WT_E_ALIGN, _desc(wt, seq_offsets=A + 2))


def test_backward_refusals(wt):
    def f(status, d=None, **kw):
        a = dict(index=A, seq_counts=A, dweight=A, dloss=A, dlogits=A + 0x100000, stride=48)
        a.update(kw)
        _refused(wt, status, wt.wt_router_backward, d or _desc(wt), *a.values())

    f(wt.WT_E_INVAL, dlogits=0)
    f(wt.WT_E_INVAL, index=0)
    f(wt.WT_E_INVAL, seq_counts=0)
    f(wt.WT_E_INVAL, stride=47)
    f(wt.WT_E_INVAL, stride=2 ** 62)
    f(wt.WT_E_ALIGN, dlogits=A + 2)
    for k in ("index", "seq_counts", "dweight", "dloss"):
        f(wt.WT_E_ALIGN, **{k: A + 2})
    f(wt.WT_E_OVERLAP, dlogits=A, stride=64)
    wt.wt_router_backward(_desc(wt, n_tokens=0), 0, 0, 0, 0, 0, 48)  # nothing to do


def test_rows_refusals(wt):
    n = wt.wt_dispatch_workspace_bytes(100, 4, 48)
    for a in ((-1, 4, 48), (100, 0, 48), (100, 4, 0), (100, 4, 1025), (2 ** 31, 1, 48)):
        _refused(wt, wt.WT_E_INVAL, wt.wt_dispatch_workspace_bytes, *a)

    def f(status, **kw):
        a = dict(index=A, n_tokens=100, top_k=4, n_experts=48, row_align=16, n_rows=1000, row_token=A, pair_row=A,
                 offsets=A, counts=A, workspace=A, workspace_bytes=n)
        a.update(kw)
        _refused(wt, status, wt.wt_dispatch_rows, *a.values())

    for k, v in (("index", 0), ("offsets", 0), ("workspace", 0), ("row_align", 0), ("row_align", 4097),
                 ("n_rows", -1), ("n_rows", 2 ** 31), ("n_experts", 0), ("top_k", 0), ("n_tokens", -1)):
        f(wt.WT_E_INVAL, **{k: v})
    f(wt.WT_E_INVAL, n_tokens=2 ** 31 - 1, top_k=1, n_experts=1024, row_align=4096, workspace_bytes=1 << 40)
    for k in ("index", "row_token", "pair_row", "offsets", "counts", "workspace"):
        f(wt.WT_E_ALIGN, **{k: A + 1})
    f(wt.WT_E_RANGE, workspace_bytes=n - 1)
