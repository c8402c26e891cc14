"""Calls whose workgroups have 2^32 threads or more in all, which no single launch takes: the weights' gradients
of many experts, MXFP4 and back, FP8 activations, over more blocks than fit. Values are exact, so that every element can be compared."""
import pytest
import torch

import expert_ref as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    yield _wt
    torch.cuda.empty_cache()


def _stream():
    return torch.cuda.current_stream().cuda_stream


# 1024 experts x 2^21 rows of out: 2^25 tiles, 2^33 threads; one column: the kernel of any alignment
@pytest.mark.parametrize("n", [1, 2])
def test_gradients_of_many_weights(wt, n):
    m, E = 1 << 21, 1024
    pattern = torch.arange(-96, 97, dtype=torch.float32, device="cuda").to(BF16)
    a = pattern.repeat(E * m // 193 + 1)[: E * m].view(E, m)
    b = torch.randint(1, 3, (E, n), generator=torch.Generator().manual_seed(n)).to(BF16).cuda()
    out = torch.full((E, m, n), -7.0, dtype=BF16, device="cuda")
    offsets = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    d = wt.wt_product_desc_init()
    d.n_rows, d.n_experts, d.offsets, d.form, d.m, d.n = E, E, offsets.data_ptr(), R.TN, m, n
    d.a, d.a_stride, d.b, d.b_stride = a.data_ptr(), m, b.data_ptr(), n
    d.out, d.out_stride, d.out_expert_stride = out.data_ptr(), n, m * n
    wt.wt_expert_product(d, _stream())
    torch.cuda.synchronize()
    for e in range(E):
        assert torch.equal(out[e], a[e][:, None] * b[e][None, :]), f"expert {e}"


def test_mxfp4_there_and_back(wt):
    rows, period = (1 << 30) + 1000, 1000
    some = torch.randn(period, 1, generator=torch.Generator().manual_seed(3)).to(BF16)
    x = some.cuda().repeat(rows // period + 1, 1)[:rows].contiguous()
    codes = torch.full((rows, 16), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 1), 0xA5, dtype=torch.uint8, device="cuda")
    wt.wt_mxfp4_quantize(x.data_ptr(), wt.WT_DT_BF16, rows, 1, 1, 0, rows, codes.data_ptr(), 16, scales.data_ptr(), 1, _stream())
    want_codes, want_scales = R.mx_round(some)
    want_codes = R.mx_pack(want_codes)
    back = torch.full((rows, 1), -7.0, dtype=BF16, device="cuda")
    wt.wt_mxfp4_dequantize(codes.data_ptr(), 16, scales.data_ptr(), 1, rows, 1, back.data_ptr(), wt.WT_DT_BF16, 1, _stream())
    torch.cuda.synchronize()
    want_back = R.mx_values(want_codes, want_scales)[:, :1].to(BF16)
    for name, got, want in (("codes", codes, want_codes), ("scales", scales, want_scales), ("back", back, want_back)):
        want = want.cuda()
        for at in range(0, rows, 10 ** 8):  # a multiple of the period
            part = got[at:at + 10 ** 8]
            whole = len(part) // period * period
            assert bool((part[:whole].view(-1, *want.shape) == want).all()), f"{name} from {at} on"
            assert torch.equal(part[whole:], want[: len(part) - whole]), f"{name}: the end"


# blocks of 16 lanes (any alignment) and of 8 (rows of 8 elements)
@pytest.mark.parametrize("rows,cols", [((1 << 28) + 1000, 1), ((1 << 29) + 1000, 8)])
def test_fp8_activations(wt, rows, cols):
    period = 1000
    some = torch.randn(period, cols, generator=torch.Generator().manual_seed(cols)).to(BF16)
    some[7] = 0
    x = some.cuda().repeat(rows // period + 1, 1)[:rows].contiguous()
    q = torch.full((rows, cols), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows,), -7.0, device="cuda")
    wt.wt_quantize_act_b128(x.data_ptr(), rows, cols, cols, 0, rows, q.data_ptr(), cols, scales.data_ptr(), 4, _stream())
    torch.cuda.synchronize()
    amax = some.float().abs().amax(1)
    want_scales = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    want = (some.float() / want_scales[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    for name, got, want in (("codes", q, want), ("scales", scales, want_scales)):
        want = want.cuda()
        for at in range(0, rows, 10 ** 8):  # a multiple of the period
            part = got[at:at + 10 ** 8]
            whole = len(part) // period * period
            assert bool((part[:whole].view(-1, *want.shape) == want).all()), f"{name} from {at} on"
            assert torch.equal(part[whole:], want[: len(part) - whole]), f"{name}: the end"
