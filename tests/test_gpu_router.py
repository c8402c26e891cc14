"""The expert router (wt_router_forward / wt_router_backward) and the dispatch's
row map (wt_dispatch_rows) on the GPU against their definitions in 64 bits:
both scores, logits types, biases, odd expert counts, strides, ties and near
ties, experts switched off, rows with nothing left, infinities and NaN,
sequences of any length with padding around them, gradients against automatic
ones and against differences, capture and replay, and the way of a batch from
its logits to quantized rows per expert and back to an optimizer step. Marked
gpu."""
import math

import numpy as np
import pytest
import torch

import oracle
import router_ref as R
from bf16_fp8_weight_amd import workloads as W
from gpu_util import log

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24


@pytest.fixture(scope="module")
def wt():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    from bf16_fp8_weight_amd import wt as _wt
    yield _wt
    torch.cuda.synchronize()


class Case:
    def __init__(self, wt, x, top_k, kind="sigmoid", normalize=True, scale=2.5, bias=None, offsets=None, coef=0.01,
                 pad=0, null_offsets=False):
        """x: CPU tensor [T, E], fp32 or BF16."""
        T, E = x.shape
        self.wt, self.x, self.T, self.E, self.K = wt, x, T, E, top_k
        self.kind, self.normalize, self.scale, self.coef = kind, normalize, float(np.float32(scale)), float(np.float32(coef))
        self.offsets = [0, T] if offsets is None else list(offsets)
        self.S = len(self.offsets) - 1
        self.dev = torch.full((T, E + pad), 7.0, dtype=x.dtype, device="cuda")
        self.dev[:, :E] = x.cuda()
        self.bias = None if bias is None else bias.cuda().float()
        self.off = torch.tensor(self.offsets, dtype=torch.int32, device="cuda")
        d = wt.wt_router_desc_init()
        d.n_tokens, d.n_experts, d.top_k, d.n_seqs = T, E, top_k, self.S
        d.logits, d.logits_stride = self.dev.data_ptr(), E + pad
        d.logits_dtype = wt.WT_DT_BF16 if x.dtype == torch.bfloat16 else wt.WT_DT_F32
        d.score = wt.WT_SCORE_SIGMOID if kind == "sigmoid" else wt.WT_SCORE_SOFTMAX
        d.normalize, d.scale, d.balance_coef = int(normalize), scale, coef
        d.bias = self.bias.data_ptr() if bias is not None else None
        d.seq_offsets = None if null_offsets else self.off.data_ptr()
        self.d = d
        n = lambda *s, **k: torch.full(s, -77, device="cuda", **k)  # noqa: E731
        self.index, self.weight = n(T + 1, top_k, dtype=torch.int32), n(T + 1, top_k, dtype=torch.float32)
        self.counts, self.seq_counts = n(E, dtype=torch.int32), n(self.S, E, dtype=torch.int32)
        self.loss = n(2, dtype=torch.float32)
        size = wt.wt_router_workspace_bytes(d)
        self.ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws_bytes = size

    def forward(self, stream=0):
        self.wt.wt_router_forward(self.d, self.index.data_ptr(), self.weight.data_ptr(), self.counts.data_ptr(),
                                  self.seq_counts.data_ptr(), self.loss.data_ptr(), self.ws.data_ptr(), self.ws_bytes,
                                  stream)

    def want(self):
        bias = None if self.bias is None else self.bias.cpu().double().numpy()
        return R.forward(self.x.double().numpy(), kind=self.kind, top_k=self.K, normalize=self.normalize,
                         scale=self.scale, bias=bias, offsets=self.offsets, coef=self.coef)

    def check_forward(self):
        self.forward()
        torch.cuda.synchronize()
        assert bool((self.ws[self.ws_bytes:] == 0xA5).all())
        assert bool((self.index[self.T] == -77).all()) and bool((self.weight[self.T] == -77).all())
        assert float(self.loss[1]) == -77
        index, weight, seq_counts, loss = self.want()
        got = self.index[:self.T].cpu().numpy()
        bad = np.argwhere(got != index)
        assert bad.size == 0, f"{len(bad)} places differ, first {tuple(bad[0])}: got {got[bad[0][0]]} want {index[bad[0][0]]}"
        assert np.array_equal(self.seq_counts.cpu().numpy(), seq_counts)
        assert np.array_equal(self.counts.cpu().numpy(), seq_counts.sum(0))
        g = self.weight[:self.T].cpu().numpy()
        # score: exponential (1 ulp = 2 EPS32) of an argument rounded once (its error times the argument, at most
        # 30 where the score matters), sum of E terms (log2-deep, 16 roundings at most), quotient; then the sum of
        # top_k, a quotient and the scale: 30 + 2 + 16 + 2 + 2 (6 + 2) + 2 roundings cover it
        tol = 64 * EPS32 * np.abs(weight) + 1e-30
        assert np.array_equal(np.isnan(g), np.isnan(weight))
        fine = ~np.isnan(weight)
        assert np.all(np.abs(g - weight)[fine] <= tol[fine]), np.max(np.abs(g - weight)[fine] / tol[fine])
        got = float(self.loss[0])
        if math.isnan(loss):
            assert math.isnan(got)
        else:
            # the probabilities' error and fp32 sums over at most 16 tokens of a wave, the rest in 64 bits
            assert abs(got - loss) <= 80 * EPS32 * abs(loss) + 1e-30, (got, loss)
        return index, weight

    def check_backward(self, dweight=True, dloss=0.7, in_place=False, index=None, seed=1):
        gen = torch.Generator().manual_seed(seed)
        idx = self.index[:self.T] if index is None else index.cuda()
        dw = torch.randn(self.T, self.K, generator=gen) if dweight else None
        out = self.dev if in_place else torch.full((self.T, self.E + 3), 9.0, dtype=self.x.dtype, device="cuda")
        dwd = dw.cuda() if dweight else None
        dl = torch.tensor([0.0 if dloss is None else dloss], device="cuda")
        seqc = self.seq_counts
        self.wt.wt_router_backward(self.d, idx.data_ptr(), seqc.data_ptr(), dwd.data_ptr() if dweight else 0,
                                   dl.data_ptr() if dloss is not None else 0, out.data_ptr(), out.stride(0))
        torch.cuda.synchronize()
        x = self.x.double().requires_grad_()
        v = R.value(x, idx.cpu().long(), seqc.cpu(), dw.double() if dweight else None,
                    None if dloss is None else float(dl), kind=self.kind, top_k=self.K, normalize=self.normalize,
                    scale=self.scale, offsets=self.offsets, coef=self.coef)
        want = torch.autograd.grad(v, x)[0].numpy() if v.requires_grad else np.zeros((self.T, self.E))
        got = out[:, :self.E].float().cpu().numpy().astype(np.float64)
        if not in_place:
            assert bool((out[:, self.E:] == 9.0).all())
        # a gradient is a sum of parts that cancel: the error is relative to the parts, which the largest
        # entry of dweight / dloss times the scale bounds
        part = (float(dw.abs().max()) * abs(self.scale) * 4 / (1 if not self.normalize else
                self._least_mass(idx)) if dweight else 0.0)
        part += 0 if dloss is None else abs(dloss * self.coef) * self.E / min(
            [b - a for a, b in zip(self.offsets, self.offsets[1:]) if b > a] or [1])
        tol = 64 * EPS32 * part + (2.0 ** -8 * np.abs(want) if self.x.dtype == torch.bfloat16 else 0.0)
        bad = np.argwhere(~(np.abs(got - want) <= tol))
        assert bad.size == 0, (len(bad), tuple(bad[0]), got[tuple(bad[0])], want[tuple(bad[0])])
        for t in list(range(0, self.offsets[0])) + list(range(self.offsets[-1], self.T)):
            assert not got[t].any()
        return want

    def _least_mass(self, idx):
        s = torch.sigmoid(self.x.double()) if self.kind == "sigmoid" else torch.softmax(self.x.double(), 1)
        idx = idx.cpu().long()
        m = (s.gather(1, idx.clamp(0, self.E - 1)) * ((idx >= 0) & (idx < self.E))).sum(1)
        m = m[m > 0]
        return min(1.0, float(m.min())) if m.numel() else 1.0


def logits(T, E, dtype=torch.float32, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * spread + 0.5 * torch.randn(1, E, generator=g)
    return x.to(dtype)


def bias(E, seed=0):
    return 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(1000 + seed))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_forward_and_backward(wt, kind, dtype, with_bias, normalize):
    for i, (T, E, K) in enumerate([(1, 1, 1), (3, 8, 2), (70, 63, 5), (257, 64, 8), (130, 65, 1), (50, 160, 6),
                                   (33, 256, 32), (129, 384, 8), (20, 500, 7), (9, 1024, 12)]):
        c = Case(wt, logits(T, E, dtype, i), K, kind, normalize, bias=bias(E, i) if with_bias else None,
                 pad=[0, 1, 8][i % 3], null_offsets=i % 2 == 0)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("offsets", [
    [0, 300], [0, 0, 300], [0, 1, 2, 3, 300, 300], [17, 100, 250], [0, 64, 128, 192, 256], [300, 300], [0, 0],
    [5, 5, 6, 37, 38, 38, 299], list(range(0, 301)),
])
def test_sequences_and_padding(wt, kind, offsets):
    c = Case(wt, logits(300, 96, seed=3), 4, kind, True, bias=bias(96), offsets=offsets)
    c.check_forward()
    c.check_backward()
    c.check_backward(dweight=False)
    c.check_backward(dloss=None)


def test_long_batch_with_larger_tiles(wt):
    # enough tokens for tiles of 64, and sequences that end inside them
    T = 70001
    offsets = [3, 10, 4096, 4097, 40000, 69990]
    c = Case(wt, logits(T, 16, seed=8), 2, "softmax", True, bias=bias(16), offsets=offsets)
    c.forward()
    torch.cuda.synchronize()
    x = c.x.double()
    s = torch.softmax(x, 1)
    top = torch.sort(s + c.bias.cpu().double(), dim=1, descending=True, stable=True).indices[:, :2]
    live = torch.zeros(T, 1, dtype=torch.bool)
    live[3:69990] = True
    assert torch.equal(c.index[:T].cpu().long(), torch.where(live, top, -1))
    loss = 0.0
    for a, b in zip(offsets, offsets[1:]):
        n = torch.bincount(top[a:b].flatten(), minlength=16)
        assert torch.equal(c.seq_counts[offsets.index(a)].cpu().long(), n)
        loss += float((16 * n.double() / (2 * (b - a)) * s[a:b].mean(0)).sum())
    assert abs(float(c.loss[0]) - c.coef / 5 * loss) <= 80 * EPS32 * c.coef * loss
    c.check_backward()


def test_thousands_of_sequences(wt):
    # more sequences than one probe of the search covers, many of them empty, padding at both ends
    T, E, K, S = 3000, 16, 2, 5000
    g = torch.Generator().manual_seed(1)
    offsets = torch.sort(torch.randint(5, T - 7, (S + 1,), generator=g)).values
    c = Case(wt, logits(T, E, seed=21), K, "sigmoid", bias=bias(E), offsets=offsets.tolist())
    c.forward()
    torch.cuda.synchronize()
    x = c.x.double()
    s = torch.sigmoid(x)
    p = s / s.sum(1, keepdim=True)
    top = torch.sort(s + c.bias.cpu().double(), dim=1, descending=True, stable=True).indices[:, :K]
    t = torch.arange(T)
    live = (t >= offsets[0]) & (t < offsets[-1])
    assert torch.equal(c.index[:T].cpu().long(), torch.where(live[:, None], top, -1))
    seq = torch.searchsorted(offsets, t[live], right=True) - 1
    n = torch.bincount(seq, minlength=S).double()
    counts = torch.zeros(S, E, dtype=torch.float64).index_add_(0, seq, torch.zeros(int(live.sum()), E, dtype=torch.float64).scatter_(1, top[live], 1.0))
    assert torch.equal(c.seq_counts.cpu().double(), counts) and torch.equal(c.counts.cpu().double(), counts.sum(0))
    psum = torch.zeros(S, E, dtype=torch.float64).index_add_(0, seq, p[live])
    loss = c.coef / S * float((E / K * counts * psum).sum(1).div(n.clamp(min=1) ** 2).sum())
    assert abs(float(c.loss[0]) - loss) <= 80 * EPS32 * loss
    c.check_backward()


def test_two_calls_at_once(wt):
    # two streams, each with buffers of its own, many calls in flight on both
    cs = [Case(wt, logits(2500, 200, seed=k), 6, "sigmoid", bias=bias(200), offsets=[0, 900, 2490]) for k in (1, 2)]
    want = []
    for c in cs:
        c.forward()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (c.index, c.weight, c.counts, c.seq_counts, c.loss)])
    n_rows = 2500 * 6
    rows = []
    for c in cs:
        size = wt.wt_dispatch_workspace_bytes(2500, 6, 200)
        i32 = dict(dtype=torch.int32, device="cuda")
        rows.append((torch.empty(n_rows, **i32), torch.empty(2500, 6, **i32), torch.empty(201, **i32),
                     torch.empty(size, dtype=torch.uint8, device="cuda")))
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(20):
        for c, r, s in zip(cs, rows, streams):
            c.forward(s.cuda_stream)
            wt.wt_dispatch_rows(c.index.data_ptr(), 2500, 6, 200, 1, n_rows, r[0].data_ptr(), r[1].data_ptr(),
                                r[2].data_ptr(), 0, r[3].data_ptr(), r[3].numel(), s.cuda_stream)
    torch.cuda.synchronize()
    for c, w, r in zip(cs, want, rows):
        for t, x in zip((c.index, c.weight, c.counts, c.seq_counts, c.loss), w):
            assert torch.equal(t, x)
        ref = R.rows(c.index[:2500].cpu().numpy(), 200, 1, n_rows)
        assert np.array_equal(r[0].cpu().numpy(), ref[0]) and np.array_equal(r[1].cpu().numpy(), ref[1])


def test_no_tokens(wt):
    c = Case(wt, torch.zeros(0, 24), 3, offsets=[0, 0, 0])
    c.forward()
    torch.cuda.synchronize()
    assert not c.counts.any() and not c.seq_counts.any() and float(c.loss[0]) == 0.0


def test_ties_go_to_the_lower_index(wt):
    # equal logits and equal biases: whole rows of ties, ties across the border of the selection
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-2, 3, (400, 200), generator=g).float()
    for b in (None, torch.zeros(200), torch.randint(0, 2, (200,), generator=g).float() * 0.25):
        for kind in ("sigmoid", "softmax"):
            Case(wt, x, 8, kind, bias=b).check_forward()
            Case(wt, torch.zeros(5, 200), 8, kind, bias=b).check_forward()


def test_near_ties_are_decided_in_64_bits(wt):
    # keys that 32 bits cannot order: biases that cancel the difference of two scores up to a few 2^-26
    E, T = 128, 256
    g = torch.Generator().manual_seed(6)
    x = torch.randn(T, E, generator=g)
    x[:] = x[0]  # every token the same logits, so that a bias can be made for them
    s = torch.sigmoid(x[0].double())
    b = (2.0 - s).float()  # keys all 2 within the rounding of the bias
    key = s + b.double()
    gaps = torch.sort(key).values.diff()
    assert float(gaps.max()) < 2 ** -22 and float(gaps.min()) > 1e-12
    c = Case(wt, x, 10, "sigmoid", bias=b)
    index, _ = c.check_forward()
    assert (index == index[0]).all()
    # a mix of ordinary tokens and near ties
    y = torch.randn(T, E, generator=g)
    y[::3] = x[0]
    Case(wt, y, 10, "sigmoid", bias=b).check_forward()
    p = torch.softmax(x[0].double(), 0)
    b = (0.5 - p).float()
    Case(wt, x, 10, "softmax", bias=b).check_forward()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("centre", [0.0, 100.0, -60.0])
@pytest.mark.parametrize("spread", [1e-2, 1e-4, 1e-6, 0.0])
def test_logits_close_together(wt, kind, centre, spread):
    # a router at its start: all keys nearly alike, so that thresholds far below the greatest separate nothing
    E, T = 384, 40
    x = centre + spread * torch.randn(T, E, generator=torch.Generator().manual_seed(3))
    for b in (None, torch.zeros(E), 0.01 * bias(E)):
        Case(wt, x, 8, kind, bias=b).check_forward()
    Case(wt, x.to(torch.bfloat16), 8, kind).check_forward()


def test_as_many_places_as_experts(wt):
    for E, K in ((32, 32), (64, 32), (33, 32), (2, 2), (5, 5)):
        for b in (None, bias(E)):
            c = Case(wt, logits(50, E, seed=E), K, "sigmoid", bias=b)
            c.check_forward()
            c.check_backward()
            Case(wt, logits(50, E, torch.bfloat16, seed=E), K, "softmax", bias=b).check_forward()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_experts_switched_off(wt, kind, with_bias):
    # -infinity: some experts, all but two (fewer than top_k), all
    x = logits(40, 70, seed=4)
    x[:, 5:20] = -math.inf
    x[7] = -math.inf
    x[8, 2:] = -math.inf
    x[9, :] = -math.inf
    x[9, 69] = -3.0
    c = Case(wt, x, 6, kind, True, bias=bias(70) if with_bias else None)
    index, weight = c.check_forward()
    assert (index[7] == -1).all() and (weight[7] == 0).all() and (index[8] >= 0).sum() == 2
    y = x.clone()
    y[7] = 0.0  # the gradient's reference knows no row without experts
    c2 = Case(wt, y, 6, kind, True, bias=bias(70) if with_bias else None)
    c2.check_forward()
    c2.check_backward()
    dl = torch.tensor([1.0], device="cuda")
    dw = torch.ones(40, 6, device="cuda")
    out = torch.full((40, 70), 5.0, device="cuda")
    wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), dw.data_ptr(), dl.data_ptr(), out.data_ptr(), 70)
    torch.cuda.synchronize()
    assert bool((out[7] == 0).all()) and bool(torch.isfinite(out).all()) and bool((out[:, 5:20] == 0).all())


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_infinities_and_nan(wt, kind, with_bias):
    x = logits(12, 40, seed=5)
    x[2, 3] = math.nan
    x[4] = math.nan
    x[6, 1] = math.inf
    x[8] = 200.0
    x[9] = -200.0
    c = Case(wt, x, 4, kind, True, bias=bias(40) if with_bias else None)
    index, weight = c.check_forward()
    assert (index[4] == -1).all() and not (index[2] == 3).any()
    # the same without the ones that make the loss NaN
    x[2, 3], x[4], x[6, 1] = 0.0, 1.0, 3e38
    c = Case(wt, x, 4, kind, False, bias=bias(40) if with_bias else None)
    c.check_forward()
    dl = torch.tensor([1.0], device="cuda")
    out = torch.zeros(12, 40, device="cuda")
    wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), 0, dl.data_ptr(), out.data_ptr(), 40)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masks_of_the_lowest_value_and_endless_biases(wt, kind, dtype, with_bias):
    x = logits(30, 70, dtype, seed=6)
    x[:, 3:9] = torch.finfo(dtype).min
    x[4] = torch.finfo(dtype).min
    x[5, 8:] = torch.finfo(dtype).min
    x[6] = -math.inf
    b = None
    if with_bias:
        b = bias(70)
        b[10], b[11], b[12], b[13] = math.inf, -math.inf, math.nan, math.inf
    c = Case(wt, x, 6, kind, True, bias=b)
    index, _ = c.check_forward()
    if with_bias:
        live = index[[t for t in range(30) if t != 6]]
        assert (live[:, 0] == 10).all() and (live[:, 1] == 13).all() and not np.isin(index, [11, 12]).any()
    c.check_backward(dweight=False)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K", [(20, 4), (40, 8), (63, 8), (63, 32), (64, 8), (200, 8)])
@pytest.mark.parametrize("live", [0, 2, 3])
def test_biases_of_the_lowest_value(wt, kind, dtype, E, K, live):
    # a step below the lowest fp32 value is -infinity, the key of experts that are switched off and of the columns
    # behind the last one: none of them is selected, whatever lies behind the rows and behind the bias
    x = logits(9, E, dtype, seed=E)
    x[3, 5] = -math.inf
    b = torch.full((E,), torch.finfo(torch.float32).min)
    b[torch.randperm(E, generator=torch.Generator().manual_seed(E))[:live]] = 0.0
    c = Case(wt, x, K, kind, True, bias=b, pad=64)  # sevens behind each row
    wide = torch.full((E + 64,), 100.0, device="cuda")
    wide[:E] = c.bias
    c.d.bias = wide.data_ptr()
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,K", [(2, 1), (3, 2), (8, 2), (8, 7), (16, 8), (17, 8), (33, 32), (70, 6)])
@pytest.mark.parametrize("where", ["logits", "bias", "both"])
def test_few_experts_masked_by_the_lowest_value(wt, kind, E, K, where):
    # the lowest finite value is a key like any other: the ordinary experts first, then the masked ones by their index
    T, low = 40, torch.finfo(torch.float32).min
    g = torch.Generator().manual_seed(E)
    x = logits(T, E, seed=E)
    b = None if where == "logits" else bias(E)
    for t in range(T):  # none to K experts left, or all of them
        off = torch.randperm(E, generator=g)[(t % (K + 1)):]
        if where != "bias" and t % (K + 2) <= K:
            x[t, off] = low
    if where != "logits":
        b[torch.randperm(E, generator=g)[K // 2:]] = low
    c = Case(wt, x, K, kind, True, bias=b)
    index, _ = c.check_forward()
    assert (index >= 0).all()
    # one step above it, and half of it
    for other in (float(np.nextafter(np.float32(low), np.float32(0))), low / 2):
        y = torch.where(x == low, other, x)
        Case(wt, y, K, kind, False, bias=None if b is None else torch.where(b == low, other, b)).check_forward()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_places_without_an_expert_next_to_nan_scores(wt, kind, normalize, value):
    # a softmax with a NaN or an infinity is NaN; a place that no expert takes holds weight 0 all the same
    x = logits(8, 20, seed=17)
    x[:, 6:] = -math.inf
    x[::2, 3] = value
    x[5, 2:] = math.nan
    c = Case(wt, x, 9, kind, normalize)
    index, weight = c.check_forward()
    assert (index[:, 6:] == -1).all() and bool((c.weight[:8, 6:] == 0).all())
    assert np.isnan(weight[0, :5]).all() == (kind == "softmax")


def test_offsets_that_make_no_sense_stay_inside_the_arrays(wt):
    # falling, negative and too large offsets: the results mean nothing, the guards stay whole
    for offsets in ([50, 10, 90, 0], [-5, 1 << 30], [100, 0], [7, -7, 7, -7, 7], [2 ** 31 - 1, -(2 ** 31)]):
        c = Case(wt, logits(100, 48), 3, offsets=offsets)
        c.ws.zero_()
        c.ws[c.ws_bytes:] = 0xA5
        c.forward()
        dl = torch.tensor([1.0], device="cuda")
        out = torch.full((101, 48), 5.0, device="cuda")
        wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), c.weight.data_ptr(), dl.data_ptr(),
                              out.data_ptr(), 48)
        torch.cuda.synchronize()
        assert bool((c.ws[c.ws_bytes:] == 0xA5).all()) and bool((c.index[100] == -77).all())
        assert bool((out[100] == 5.0).all())


def test_gradient_in_place_and_foreign_indices(wt):
    c = Case(wt, logits(60, 90, seed=9), 5, "softmax", False, pad=6)
    c.check_forward()
    c.check_backward(in_place=True)
    # indices that no selection wrote: out of range, the same expert twice
    idx = torch.randint(0, 90, (60, 5), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    idx[::4, 1] = idx[::4, 0]
    idx[::5, 2] = 90
    idx[::7, 3] = -2 ** 31
    idx[3] = 2 ** 31 - 1
    for kind in ("softmax", "sigmoid"):
        c = Case(wt, logits(60, 90, seed=9), 5, kind, True)
        c.forward()
        torch.cuda.synchronize()
        c.check_backward(index=idx)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_an_expert_in_several_places_adds_up_in_their_order(wt, kind):
    # sums that depend on their order in fp32: bit for bit those of the places from the first to the last
    T, E, K = 64, 150, 8
    g = torch.Generator().manual_seed(5)
    c = Case(wt, logits(T, E, seed=14), K, kind, False, scale=1.0)
    index = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(torch.int32)
    dw = torch.randn(T, K, generator=g) * torch.exp(6.0 * torch.randn(T, K, generator=g))
    one, sums = index.clone(), dw.clone()
    for t in range(T):
        places = sorted(torch.randperm(K, generator=g)[:2 + t % (K - 1)].tolist())
        total = np.float32(0)
        for k in places:
            total = np.float32(total + np.float32(dw[t, k]))
            index[t, k] = int(index[t, places[0]])
            one[t, k] = -1
        one[t, places[0]] = index[t, places[0]]
        sums[t, places[0]] = float(total)
    outs = []
    for i, w in ((index, dw), (one, sums)):
        out = torch.full((T, E), 9.0, device="cuda")
        i, w = i.cuda(), w.cuda()
        wt.wt_router_backward(c.d, i.data_ptr(), 0, w.data_ptr(), 0, out.data_ptr(), E)
        torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_a_gradient_that_cancels(wt, kind):
    # one selected expert with a normalized weight: the weight is 1 whatever the logits are, up to the 1e-20
    c = Case(wt, logits(300, 70, seed=8), 1, kind, True)
    c.check_forward()
    dw = torch.randn(300, 1, device="cuda")
    out = torch.full((300, 70), 5.0, device="cuda")
    wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), dw.data_ptr(), 0, out.data_ptr(), 70)
    torch.cuda.synchronize()
    # |dweight| scale 1e-20 / score <= 5 * 2.5 * 1e-20 / (1 / 70), with room for the roundings
    assert float(out.abs().max()) <= 1e-17
    # gradients that are alike: the true one is what is left of their difference
    c = Case(wt, logits(300, 70, seed=9), 6, kind, True)
    c.check_forward()
    dw = 1000.0 + torch.rand(300, 6, generator=torch.Generator().manual_seed(1))
    out2 = torch.full((300, 70), 5.0, device="cuda")
    dwd = dw.cuda()
    wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), dwd.data_ptr(), 0, out2.data_ptr(), 70)
    torch.cuda.synchronize()
    x = c.x.double().requires_grad_()
    v = R.value(x, c.index[:300].cpu().long(), c.seq_counts.cpu(), dw.double(), None, kind=kind, top_k=6,
                normalize=True, scale=c.scale, offsets=c.offsets, coef=c.coef)
    want = torch.autograd.grad(v, x)[0]
    # d - d_0 is exact up to the rounding of d scale (1 in 2^24 of 2502); a difference of at most 2.5 over the mass m of
    # the selected, with 64 roundings of the sums, scores and quotients; each times a score's slope, at most 1 / 4
    m = c._least_mass(c.index[:300])
    tol = (2 * EPS32 * 2502.5 + 64 * EPS32 * 2.5) / m / 4
    assert float((out2.cpu().double() - want).abs().max()) <= tol


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [9, 64, 65, 129, 193, 257, 384, 385, 513, 1024])  # every number of columns
def test_gradient_of_the_balance_loss(wt, kind, dtype, E):
    # alone, and beside weights' gradients of its own size, with a tolerance relative to what it is made of
    T, K, offsets = 37, 8, [0, 11, 35]
    c = Case(wt, logits(T, E, dtype, seed=E), K, kind, False, scale=1.0, offsets=offsets, coef=1.0)
    index, _ = c.check_forward()
    x = c.x.double()
    s = torch.sigmoid(x) if kind == "sigmoid" else torch.softmax(x, 1)
    z = s.sum(1, keepdim=True)
    d = torch.zeros(T, E, dtype=torch.float64)  # of the loss by each probability
    for q, (a, b) in enumerate(zip(offsets, offsets[1:])):
        d[a:b] = 0.7 / 2 * E / (K * (b - a)) / (b - a) * c.seq_counts[q].cpu().double()
    idx = torch.from_numpy(index).long()
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(E)) * float((d[:35] / z[:35]).mean())
    dl, out = torch.tensor([0.7], device="cuda"), torch.full((T, E), 9.0, dtype=dtype, device="cuda")
    dwd = dw.cuda()
    for both in (False, True):
        wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), dwd.data_ptr() if both else 0,
                              dl.data_ptr(), out.data_ptr(), E)
        torch.cuda.synchronize()
        g = torch.zeros(T, E, dtype=torch.float64)
        if both:
            g[:35].scatter_(1, idx[:35], dw[:35].double())
        if kind == "sigmoid":
            want = ((d - (d * s).sum(1, keepdim=True) / z) / z + g) * s * torch.sigmoid(-x)
            # d: 7 roundings; a score 7, a sum over the experts 16 + 6, the quotient of two such sums 61, a difference
            # 1, the reciprocal of a sum 32, the slope 12 + 2 |x| with |x| below 6: 125
            part = (d.amax(1, keepdim=True) / z + g.abs()) * s * torch.sigmoid(-x)
        else:
            want = s * (d + g - ((d + g) * s).sum(1, keepdim=True))
            # a score: argument and exponential 18, sum 22, reciprocal and product 3; the mean of d + g by the scores
            # 7 + 1 + 43 + 1 + 22 of their greatest, differences 2, the score again and products 45: 121
            part = s * (d + g.abs()).amax(1, keepdim=True)
        tol = 128 * EPS32 * part + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0.0)
        err = (out.cpu().double() - want).abs()
        assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-30)).max())
        assert float(want[:35].abs().max()) > 100 * float((128 * EPS32 * part).max()) and not out[35:].any()


@pytest.mark.parametrize("E", [20, 100])
def test_slope_of_confident_scores(wt, E):
    # sigmoid scores next to 1 and next to 0: s (1 - s) has all its digits, whichever of the two is small
    T, K = 50, 6
    g = torch.Generator().manual_seed(E)
    x = (torch.rand(T, E, generator=g) * 40.0 - 20.0)
    x[:5] = 8.0 + 12.0 * torch.rand(5, E, generator=g)
    c = Case(wt, x, K, "sigmoid", False, bias=bias(E), offsets=[0, 20, T], coef=2.0)
    index, _ = c.check_forward()
    dw = torch.rand(T, K, generator=g) + 0.5
    dl, out = torch.tensor([0.7], device="cuda"), torch.full((T, E), 9.0, device="cuda")
    dwd = dw.cuda()
    idx = torch.from_numpy(index).long()
    y = x.double()
    s, slope = torch.sigmoid(y), torch.sigmoid(y) * torch.sigmoid(-y)
    # y = exp(-x): the argument's product and factor are rounded (|x| 2 EPS32 of y together), then the exponential (2);
    # y / (1 + y)^2 moves by at most as much as y; sum, reciprocal (2), twice, and three products: 2 |x| + 16 with dw's
    rel = (2.0 * y.abs() + 16.0) * EPS32
    wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), dwd.data_ptr(), 0, out.data_ptr(), E)
    torch.cuda.synchronize()
    want = torch.zeros(T, E, dtype=torch.float64).scatter_(1, idx, dw.double() * c.scale) * slope
    bad = (out.cpu().double() - want).abs() > rel * want
    assert not bad.any(), (out.cpu()[bad][:4], want[bad][:4], x[bad][:4])
    # of the loss: b - sum(b s) / z, with errors of the greatest b (7 roundings of its own, and of the quotient of two
    # sums over experts: 7 of the scores and 8 of the sum each, 3 beside them), times 1 / z (18) and the slope (12)
    wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), 0, dl.data_ptr(), out.data_ptr(), E)
    torch.cuda.synchronize()
    z = s.sum(1, keepdim=True)
    for a, b, q in ((0, 20, 0), (20, T, 1)):
        d = float(dl) * c.coef / 2 * E / (K * (b - a)) / (b - a) * c.seq_counts[q].cpu().double()
        want = (d - (d * s[a:b]).sum(1, keepdim=True) / z[a:b]) / z[a:b] * slope[a:b]
        tol = (72.0 + 2.0 * y[a:b].abs()) * EPS32 * d.max() / z[a:b] * slope[a:b]
        assert bool(((out[a:b].cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_gradient_against_differences(wt, kind):
    # the formula's own gradient (float64 differences of the forward definition with the selection held)
    T, E, K = 6, 20, 3
    c = Case(wt, logits(T, E, seed=12), K, kind, True, offsets=[0, 2, 6], coef=0.5)
    c.check_forward()
    want = c.check_backward(dloss=2.0)
    g = torch.Generator().manual_seed(1)
    dw = torch.randn(T, K, generator=g).double()
    idx, seqc = c.index[:T].cpu().long(), c.seq_counts.cpu()

    def f(x):
        return float(R.value(x, idx, seqc, dw, 2.0, kind=kind, top_k=K, normalize=True, scale=c.scale,
                             offsets=c.offsets, coef=c.coef))

    x = c.x.double()
    for t in range(T):
        for e in range(0, E, 3):
            d = torch.zeros_like(x)
            d[t, e] = 1e-5
            diff = (f(x + d) - f(x - d)) / 2e-5
            assert abs(diff - want[t, e]) < 1e-8


def test_repeats_bit_for_bit_and_in_a_graph(wt):
    c = Case(wt, logits(3000, 384, seed=2), 8, "sigmoid", True, bias=bias(384), offsets=[0, 700, 701, 2999])
    c.forward()
    torch.cuda.synchronize()
    first = [t.clone() for t in (c.index, c.weight, c.counts, c.seq_counts, c.loss)]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    dl = torch.tensor([1.0], device="cuda")
    out = torch.zeros(3000, 384, device="cuda")

    def both(stream):
        c.forward(stream)
        wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), c.weight.data_ptr(), dl.data_ptr(),
                              out.data_ptr(), 384, stream)

    both(0)
    torch.cuda.synchronize()
    grad = out.clone()
    with torch.cuda.graph(g, stream=s):
        both(s.cuda_stream)
    for _ in range(4):
        for t in (c.index, c.weight, c.counts, c.seq_counts, c.loss):
            t.fill_(-77)
        c.ws.fill_(0x5A)
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        for t, w in zip((c.index, c.weight, c.counts, c.seq_counts, c.loss), first):
            assert torch.equal(t[:w.shape[0]], w) or t is c.loss and float(t[0]) == float(w[0])
        assert torch.equal(out, grad)
        both(0)  # the program's own eager work between the replays
        torch.cuda.synchronize()


def test_row_offsets_past_32_bits(wt):
    # rows 2^20 elements apart: the last rows' bytes lie past 2^32
    T, E, stride = 1200, 48, 1 << 20
    big = torch.empty(T * stride, device="cuda")
    x = logits(T, E, seed=3)
    view = big.view(T, stride)[:, :E]
    view.copy_(x.cuda())
    c = Case(wt, x, 4, "sigmoid", True)
    c.d.logits, c.d.logits_stride = big.data_ptr(), stride
    c.check_forward()
    dl = torch.tensor([1.0], device="cuda")
    a, b = torch.zeros(T, E, device="cuda"), torch.zeros(T, E, device="cuda")
    wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), c.weight.data_ptr(), dl.data_ptr(), a.data_ptr(), E)
    c.d.logits, c.d.logits_stride = c.dev.data_ptr(), E
    wt.wt_router_backward(c.d, c.index.data_ptr(), c.seq_counts.data_ptr(), c.weight.data_ptr(), dl.data_ptr(), b.data_ptr(), E)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


# ------------------------------------------------------------------ row map
def run_rows(wt, index, E, align, n_rows, with_token=True, with_pair=True, with_counts=True, stream=0):
    T, K = index.shape
    n = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
    tok, pair, off, cnt = n(n_rows + 1), n(T + 1, K), n(E + 2), n(E + 1)
    size = wt.wt_dispatch_workspace_bytes(T, K, E)
    ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    dev = index.cuda()
    wt.wt_dispatch_rows(dev.data_ptr(), T, K, E, align, n_rows, tok.data_ptr() if with_token else 0,
                        pair.data_ptr() if with_pair else 0, off.data_ptr(), cnt.data_ptr() if with_counts else 0,
                        ws.data_ptr(), size, stream)
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0xA5).all())
    for t in (tok, pair.reshape(-1)[T * K:], off, cnt):
        assert int(t[-1]) == -77
    want = R.rows(index.numpy(), E, align, n_rows)
    assert np.array_equal(off[:-1].cpu().numpy(), want[2])
    if with_counts:
        assert np.array_equal(cnt[:-1].cpu().numpy(), want[3])
    if with_token:
        assert np.array_equal(tok[:-1].cpu().numpy(), want[0])
    if with_pair:
        assert np.array_equal(pair[:T].cpu().numpy(), want[1])
    return want


@pytest.mark.parametrize("T,K,E", [(0, 2, 5), (1, 1, 1), (1, 8, 384), (31, 3, 7), (128, 8, 384), (257, 8, 256),
                                   (1000, 5, 1024), (4100, 2, 3), (700, 12, 100)])
@pytest.mark.parametrize("align", [1, 16, 128])
def test_rows(wt, T, K, E, align):
    g = torch.Generator().manual_seed(T + E)
    # some experts popular, some unused, padding rows, values that are no expert, experts twice in a row
    e = (torch.rand(T, K, generator=g) ** 3 * E).long().clamp(max=E - 1).to(torch.int32)
    e[torch.rand(T, K, generator=g) < 0.05] = -1
    e[torch.rand(T, K, generator=g) < 0.02] = E
    e[torch.rand(T, K, generator=g) < 0.01] = -2 ** 31
    cap = T * K + min(E, T * K) * (align - 1)
    want = run_rows(wt, e, E, align, cap)
    assert want[2][-1] <= cap
    run_rows(wt, e, E, align, cap // 2)          # copies behind the last row are dropped
    run_rows(wt, e, E, align, cap + 1000)
    run_rows(wt, e, E, align, cap, with_token=False)
    run_rows(wt, e, E, align, cap, with_pair=False, with_counts=False)
    run_rows(wt, e, E, align, 0)


@pytest.mark.parametrize("T", [0, 3, 300])
def test_many_more_rows_than_copies(wt, T):
    # whole row tiles of many unused experts' neighbours, and a long array behind the last expert
    g = torch.Generator().manual_seed(T)
    e = torch.randint(0, 900, (T, 8), generator=g, dtype=torch.int32)
    run_rows(wt, e, 900, 4096, 8 * T + min(900, 8 * T) * 4095)
    run_rows(wt, e, 900, 1, 400001)


@pytest.mark.parametrize("T,E", [(3000, 381), (40000, 6)])
def test_rows_with_a_workspace_at_any_word(wt, T, E):
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(0, E, (T, 4), generator=g, dtype=torch.int32)
    want = R.rows(idx.numpy(), E, 32, 4 * T + 31 * E)
    dev = idx.cuda()
    size = wt.wt_dispatch_workspace_bytes(T, 4, E)
    for word in range(4):
        ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        tok, pair, off, cnt = (torch.full(s, -77, dtype=torch.int32, device="cuda")
                               for s in ((4 * T + 31 * E,), (T, 4), (E + 1,), (E,)))
        wt.wt_dispatch_rows(dev.data_ptr(), T, 4, E, 32, tok.numel(), tok.data_ptr(), pair.data_ptr(), off.data_ptr(),
                            cnt.data_ptr(), ws.data_ptr() + 4 * word, size)
        torch.cuda.synchronize()
        assert bool((ws[4 * word + size:] == 0xA5).all()) and bool((ws[:4 * word] == 0xA5).all())
        for got, w in zip((tok, pair, off, cnt), want):
            assert np.array_equal(got.cpu().numpy(), w)


def test_all_copies_to_one_expert(wt):
    run_rows(wt, torch.full((3000, 4), 17, dtype=torch.int32), 40, 128, 13000)
    run_rows(wt, torch.full((300, 4), -1, dtype=torch.int32), 40, 128, 100)


def test_from_logits_to_rows_and_back_to_the_weights(wt):
    # a routed layer's training step as a rank runs it: the router's projection, selection and balance loss;
    # the copies grouped by expert and quantized into whole row tiles; the gradient of the router's weight; the
    # optimizer step on that weight; and its transfer
    T, H, E, K = 320, 256, 48, 4
    g = torch.Generator(device="cuda").manual_seed(11)
    h = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    wl = W.custom([(E, H)], kind=W.BF16, n_shards=1, device="cuda")
    w = wl.outputs[0].parts[0].shards[0]
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")  # twenty rows of padding
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st = s.cuda_stream
        x = h.float() @ w.float().t()
        d = wt.wt_router_desc_init()
        d.n_tokens, d.n_experts, d.top_k, d.n_seqs = T, E, K, 2
        d.logits, d.logits_stride, d.logits_dtype, d.score = x.data_ptr(), E, wt.WT_DT_F32, wt.WT_SCORE_SIGMOID
        d.normalize, d.balance_coef, d.seq_offsets = 1, 0.1, off.data_ptr()
        i32 = dict(dtype=torch.int32, device="cuda")
        index, weight = torch.empty(T, K, **i32), torch.empty(T, K, device="cuda")
        counts, seq_counts, loss = torch.empty(E, **i32), torch.empty(2, E, **i32), torch.empty(1, device="cuda")
        ws = torch.empty(wt.wt_router_workspace_bytes(d), dtype=torch.uint8, device="cuda")
        wt.wt_router_forward(d, index.data_ptr(), weight.data_ptr(), counts.data_ptr(), seq_counts.data_ptr(),
                             loss.data_ptr(), ws.data_ptr(), ws.numel(), st)
        n_rows = T * K + E * 15
        row_token, pair_row = torch.empty(n_rows, **i32), torch.empty(T, K, **i32)
        offsets, copies = torch.empty(E + 1, **i32), torch.empty(E, **i32)
        ws2 = torch.empty(wt.wt_dispatch_workspace_bytes(T, K, E), dtype=torch.uint8, device="cuda")
        wt.wt_dispatch_rows(index.data_ptr(), T, K, E, 16, n_rows, row_token.data_ptr(), pair_row.data_ptr(),
                            offsets.data_ptr(), copies.data_ptr(), ws2.data_ptr(), ws2.numel(), st)
        q = torch.full((n_rows, H), 0xA5, dtype=torch.uint8, device="cuda")
        sc = torch.full((n_rows, 4 * (H // 128)), 0xA5, dtype=torch.uint8, device="cuda")
        wt.wt_quantize_act_b128(h.data_ptr(), T, H, H, row_token.data_ptr(), n_rows, q.data_ptr(), H, sc.data_ptr(),
                                sc.shape[1], st)
        dweight = torch.randn(T, K, generator=g, device="cuda")
        dloss = torch.ones(1, device="cuda")
        dx = torch.empty_like(x)
        wt.wt_router_backward(d, index.data_ptr(), seq_counts.data_ptr(), dweight.data_ptr(), dloss.data_ptr(),
                              dx.data_ptr(), E, st)
        dw = dx.t().contiguous() @ h.float()
        dst = torch.full((wl.dst_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
        hy = wt.wt_adamw_hyper_init()
        hy.max_norm = 1.0
        before = w.clone()
        opt = wt.AdamW.for_workload(wl, [dw], state_bits=8)
        plan = wt.Plan(wl, dst)
        opt.step(hy, st)
        plan.prepare(st)
    s.synchronize()
    want = R.rows(index.cpu().numpy(), E, 16, n_rows)
    assert np.array_equal(row_token.cpu().numpy(), want[0]) and np.array_equal(pair_row.cpu().numpy(), want[1])
    assert torch.equal(counts, copies) and int(counts.sum()) == 300 * K and bool((index[300:] == -1).all())
    wq = np.full((n_rows, H), 0xA5, dtype=np.uint8)
    ws_ = np.full((n_rows, sc.shape[1]), 0xA5, dtype=np.uint8)
    oracle.quantize_act(h.view(torch.int16).cpu().numpy().view(np.uint16), cols=H, index=want[0], n_out=n_rows, q=wq, scales=ws_)
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(sc.cpu().numpy(), ws_)
    xx = (h.double().cpu() @ before.double().cpu().t()).requires_grad_()
    v = R.value(xx, index.cpu().long(), seq_counts.cpu(), dweight.double().cpu(), 1.0, kind="sigmoid", top_k=K,
                normalize=True, scale=1.0, offsets=[0, 100, 300], coef=float(np.float32(0.1)))
    ref = (torch.autograd.grad(v, xx)[0].t() @ h.double().cpu()).numpy()
    # fp32 products over 256 and 320 terms on logits and gradients of unit scale
    assert np.abs(dw.cpu().numpy() - ref).max() <= 1e-4 * np.abs(ref).max()
    moved = (w.float() - before.float()).cpu().numpy()
    big = np.abs(ref) > 1e-3 * np.abs(ref).max()
    assert np.all(np.sign(moved[big]) * np.sign(ref[big]) <= 0) and (moved != 0).mean() > 0.5
    o = wl.outputs[0]
    assert torch.equal(dst[o.dst_offset:o.dst_offset + o.data_bytes], w.reshape(-1).view(torch.uint8))
    opt.close()
    plan.close()
