"""Calls that the documentation of the experts' products allows beside the ordinary
ones: the gated backward pass over its own operand, the null stream, a stream
beside another's work, and captured calls that share their operands."""
import pytest
import torch

import expert_ref as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wt():
    from bf16_fp8_weight_amd import wt as _wt
    return _wt


def _normal(seed, *shape):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g).to(BF16).cuda()


def _desc(wt, lay, form, n, k, a, b, out, keep):
    d = wt.wt_product_desc_init()
    off, cnt = lay.offsets.cuda(), lay.counts_t.cuda()
    keep += [off, cnt]
    d.offsets, d.counts, d.n_experts, d.n_rows = off.data_ptr(), cnt.data_ptr(), len(lay.counts), lay.n_rows
    d.form, d.n, d.k = form, n, k
    d.a, d.a_stride, d.b, d.b_stride, d.b_expert_stride = a.data_ptr(), a.stride(0), b.data_ptr(), b.stride(1), b.stride(0)
    d.out, d.out_stride = out.data_ptr(), out.stride(0)
    return d


# counts, n, k: every tile size, and odd sizes
SHAPES = [([3, 0, 9], 40, 64), ([70, 1, 0, 200], 256, 128), ([300, 900, 40], 1024, 96), ([1500, 20, 700, 800], 4096, 64),
          ([33, 130], 131, 65), ([5, 0, 17], 1, 7)]


@pytest.mark.parametrize("act", [R.SILU, R.GELU])
@pytest.mark.parametrize("counts,n,k", SHAPES)
def test_backward_over_its_own_operand(wt, counts, n, k, act):
    lay, keep = R.Layout(counts, lead=2, tail=3), []
    dy, down, pre = _normal(1, lay.n_rows, k), _normal(2, len(counts), k, n), _normal(3, lay.n_rows, 2 * n)
    out = pre.clone()
    stream = torch.cuda.current_stream().cuda_stream
    d = _desc(wt, lay, R.NN, n, k, dy, down, out, keep)
    d.act = act
    wt.wt_gated_backward(d, pre.data_ptr(), 2 * n, stream)
    over = pre.clone()
    d.out = over.data_ptr()
    wt.wt_gated_backward(d, over.data_ptr(), 2 * n, stream)
    torch.cuda.synchronize()
    assert torch.equal(out, over)
    owned = lay.owned().cuda()
    assert torch.equal(over[~owned], pre[~owned]) and not torch.equal(over[owned], pre[owned])


def test_streams(wt):
    lay, keep = R.Layout([100, 0, 300]), []
    a, b = _normal(4, lay.n_rows, 256), _normal(5, 3, 512, 256)
    outs = [torch.zeros(lay.n_rows, 512, dtype=BF16, device="cuda") for _ in range(3)]
    d = _desc(wt, lay, R.NT, 512, 256, a, b, outs[0], keep)
    torch.cuda.synchronize()
    wt.wt_expert_product(d, 0)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    d.out = outs[1].data_ptr()
    wt.wt_expert_product(d, one.cuda_stream)
    d.out = outs[2].data_ptr()
    wt.wt_expert_product(d, two.cuda_stream)
    torch.cuda.synchronize()
    assert bool(outs[0].any()) and torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_two_graphs_share_their_operands(wt):
    lay, keep = R.Layout([37, 200, 0, 64]), []
    n, k, E = 192, 320, 4
    x, w, down = _normal(6, lay.n_rows, k), _normal(7, E, 2 * n, k), _normal(8, E, k, n)
    h, pre = torch.zeros(lay.n_rows, n, dtype=BF16, device="cuda"), torch.zeros(lay.n_rows, 2 * n, dtype=BF16, device="cuda")
    dpre = torch.zeros_like(pre)
    forward = _desc(wt, lay, R.NT, n, k, x, w, h, keep)
    backward = _desc(wt, lay, R.NN, n, k, x, down, dpre, keep)

    def run():
        s = torch.cuda.current_stream().cuda_stream
        wt.wt_gated_forward(forward, pre.data_ptr(), 2 * n, s)
        wt.wt_gated_backward(backward, pre.data_ptr(), 2 * n, s)

    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for replay in range(6):
        x.copy_(_normal(20 + replay, lay.n_rows, k))
        for t in (h, pre, dpre):
            t.fill_(-3.0)
        graphs[replay % 2].replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, pre, dpre)]
        run()
        torch.cuda.synchronize()
        for name, g, t in zip(("h", "pre", "dpre"), got, (h, pre, dpre)):
            assert torch.equal(g, t), f"replay {replay}: {name}"
