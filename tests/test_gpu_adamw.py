"""The AdamW step over many shards (wt_adamw_* through the C ABI) on the GPU
against its definition in 64 bits: every combination of state width, gradient
type and master copy over sizes around the block, wave and item borders,
misaligned arrays, clipping, gradients that are not finite, empty and tiny
blocks, the mean of the random rounding, capture and replay, another stream,
offsets past 32 bits, and the step followed by a prepare of the same shards.
Marked gpu."""
import math

import numpy as np
import pytest
import torch

import adamw_ref as R
from bf16_fp8_weight_amd import workloads as W
from gpu_util import assert_images_equal, log, oracle_image_threaded

pytestmark = pytest.mark.gpu

HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, grad_scale=0.5, max_norm=0.0, step=7, seed=0x1234567890)


@pytest.fixture(scope="module")
def wt():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    from bf16_fp8_weight_amd import wt as _wt
    yield _wt
    torch.cuda.synchronize()


class Tensor:
    """One shard's arrays, each inside a buffer of its own with guard bytes on
    both sides; `shift` moves every array by that many of its elements."""

    GUARD = 64

    def __init__(self, n, bits, grad, master, param, shift=0, seed=0, spread=1.0, wd=0.1, lr_mul=1.0):
        self.n, self.bits, self.shift, self.wd, self.lr_mul = n, bits, shift, wd, lr_mul
        rng = np.random.default_rng(seed)
        nb = R.blocks(n)
        std = np.repeat(np.exp(spread * rng.standard_normal(nb)), 128)[:n]
        self.buf, self.dtype = {}, {}
        g = (rng.standard_normal(n) * 1e-2 * std).astype(np.float32)
        p = (rng.standard_normal(n) * 0.02).astype(np.float32)
        m = (rng.standard_normal(n) * 3e-3 * std).astype(np.float32)
        r = (np.exp(0.7 * rng.standard_normal(n)) * 1e-2 * std).astype(np.float32)
        t = torch.from_numpy
        self._put("grad", t(g).to(torch.bfloat16) if grad == "bf16" else t(g))
        if master:
            self._put("master", t(p))
        if param:
            self._put("param", t(p).to(torch.bfloat16))
        if bits == 32:
            self._put("m", t(m))
            self._put("v", t(r * r))
        else:
            codes = rng.integers(0, 256, n).astype(np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x38
            rcodes = rng.integers(0, 0x7F, n).astype(np.uint8)
            self._put("m", t(codes))
            self._put("v", t(rcodes))
            top = np.exp(spread * rng.standard_normal(nb)).astype(np.float32)
            self._put("m_scale", t(top * np.float32(1e-2 / 448)))
            self._put("v_scale", t(top * np.float32(3e-2 / 448)))

    def _put(self, name, x):
        size, off = x.element_size(), self.GUARD + self.shift * x.element_size()
        raw = torch.full((off + x.numel() * size + self.GUARD,), 0xA5, dtype=torch.uint8)
        raw[off:off + x.numel() * size] = x.contiguous().view(torch.uint8).reshape(-1)
        self.buf[name] = raw.cuda()
        self.dtype[name] = x.dtype

    def set(self, name, x):
        self._put(name, x)

    def ptr(self, name):
        size = torch.empty(0, dtype=self.dtype[name]).element_size()
        return self.buf[name].data_ptr() + self.GUARD + self.shift * size

    def entry(self, wt):
        d = {k: self.ptr(k) for k in self.buf}
        return dict(d, n=self.n, lr_mul=self.lr_mul, weight_decay=self.wd,
                    grad_dtype=wt.WT_DT_BF16 if self.dtype["grad"] == torch.bfloat16 else wt.WT_DT_F32)

    def read(self, name):
        raw = self.buf[name].cpu()
        size = torch.empty(0, dtype=self.dtype[name]).element_size()
        off = self.GUARD + self.shift * size
        count = R.blocks(self.n) if name.endswith("scale") else self.n
        assert bool((raw[:off] == 0xA5).all()) and bool((raw[off + count * size:] == 0xA5).all()), name + ": guard bytes"
        x = raw[off:off + count * size].clone()
        if self.dtype[name] == torch.bfloat16:
            return x.view(torch.int16).numpy().view(np.uint16).copy()
        return x.view(self.dtype[name]).numpy().copy()

    def snapshot(self):
        return {k: self.read(k) for k in self.buf}


def hyper(wt, **kw):
    h = wt.wt_adamw_hyper_init()
    for k, v in dict(HYPER, **kw).items():
        setattr(h, k, v)
    return h


def values(t, snap):
    """64-bit p, g, m, v of a snapshot."""
    p = snap["master"].astype(np.float64) if "master" in snap else R.bf16_value(snap["param"])
    g = R.bf16_value(snap["grad"]) if snap["grad"].dtype == np.uint16 else snap["grad"].astype(np.float64)
    if t.bits == 32:
        return p, g, snap["m"].astype(np.float64), snap["v"].astype(np.float64)
    m = R.E4M3[snap["m"]] * R.per_block(snap["m_scale"].astype(np.float64), t.n)
    r = R.E4M3[snap["v"]] * R.per_block(snap["v_scale"].astype(np.float64), t.n)
    return p, g, m, r * r


def check(t, before, after, block0, h, clip=1.0, what=""):
    p, g, m, v = values(t, before)
    with np.errstate(all="ignore"):
        pn, mn, vn, ep, em, ev, eroot = R.step(
            p, g, m, v, lr=h.lr * t.lr_mul, beta1=h.beta1, beta2=h.beta2, eps=h.eps, wd=t.wd, gs=h.grad_scale * clip,
            t=h.step)
    w = R.words(h.seed, h.step, block0, t.n)
    fine = np.isfinite(pn) & (np.abs(pn) < 3e38)
    assert np.array_equal(before["grad"].view(np.uint8), after["grad"].view(np.uint8)), what + ": the gradient changed"
    if "master" in after:
        got = after["master"].astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(pn)), what + ": master NaN"
        bad = fine & (np.abs(got - pn) > ep)
        assert not bad.any(), f"{what}: master off at {np.argmax(bad)}: {got[bad][0]} want {pn[bad][0]} +- {ep[bad][0]}"
        if "param" in after:
            want = torch.from_numpy(after["master"]).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
            ok = ~np.isnan(got)
            assert np.array_equal(after["param"][ok], want[ok]), what + ": param is not the rounded master"
            assert np.isnan(R.bf16_value(after["param"][~ok])).all()
    else:
        rho = (((w * np.uint64(0x9E3779B9)) & R.U32) >> np.uint64(16)).astype(np.float64) / 65536
        got = R.bf16_value(after["param"])
        assert np.array_equal(np.isnan(got), np.isnan(pn)), what + ": param NaN"
        a = np.where(fine, np.abs(pn), 0)
        lo, hi = R.bf16_up(np.maximum(a - ep, 0), rho), R.bf16_up(a + ep, rho)
        bad = fine & ~((np.abs(got) >= lo) & (np.abs(got) <= hi))
        assert not bad.any(), f"{what}: param off at {np.argmax(bad)}: {got[bad][0]} want {lo[bad][0]}..{hi[bad][0]}"
        sure = fine & (np.abs(pn) > ep) & (got != 0)
        assert np.array_equal(np.sign(got[sure]), np.sign(pn[sure]))
    if t.bits == 32:
        for name, x, e in (("m", mn, em), ("v", vn, ev)):
            got = after[name].astype(np.float64)
            assert np.array_equal(np.isnan(got), np.isnan(x)), f"{what}: {name} NaN"
            ok = np.isfinite(x) & (np.abs(x) < 3e38)
            assert np.all(np.abs(got[ok] - x[ok]) <= e[ok]), f"{what}: {name}"
    else:
        rho = (w & np.uint64(0xFFFF)).astype(np.float64) / 65536
        R.check_codes(after["m"], after["m_scale"].astype(np.float64), mn, em, rho, False, what + ": m")
        rho = (w >> np.uint64(16)).astype(np.float64) / 65536
        with np.errstate(all="ignore"):
            R.check_codes(after["v"], after["v_scale"].astype(np.float64), np.sqrt(vn), eroot, rho, True, what + ": v")


def run(wt, tensors, h, bits, stream=None):
    before = [t.snapshot() for t in tensors]
    s = stream or torch.cuda.current_stream()
    with wt.AdamW([t.entry(wt) for t in tensors], bits) as a:
        a.step(h, s.cuda_stream)
        s.synchronize()
    return before, [t.snapshot() for t in tensors]


def check_all(tensors, before, after, h, clip=1.0):
    b0 = 0
    for k, t in enumerate(tensors):
        check(t, before[k], after[k], b0, h, clip, what=f"tensor {k} (n={t.n})")
        b0 += R.blocks(t.n)


def exact_norm(tensors, snaps, grad_scale):
    return grad_scale * math.sqrt(sum(float((values(t, s)[1] ** 2).sum()) for t, s in zip(tensors, snaps)))


SIZES = [1, 2, 3, 5, 63, 127, 128, 129, 255, 896, 2047, 4095, 4096, 4097, 8192 + 64, 10007]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("master,param", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("shift", [0, 1])
def test_one_step(wt, bits, grad, master, param, shift):
    h = hyper(wt)
    ts = [Tensor(n, bits, grad, master, param, shift, seed=100 * i + bits, wd=0.1 * (i % 3), lr_mul=1.0 - 0.25 * (i % 2))
          for i, n in enumerate(SIZES)]
    before, after = run(wt, ts, h, bits)
    check_all(ts, before, after, h)


def test_mixed_table_and_empty_tensors(wt):
    # gradient types, masters and alignments mixed in one table; tensors without elements take no block
    h = hyper(wt, beta1=0.0, beta2=0.999, step=1)
    ts = [Tensor(300, 8, "bf16", True, True, 0, 1), Tensor(4096, 8, "fp32", False, True, 3, 2),
          Tensor(4096, 8, "bf16", True, False, 0, 3), Tensor(777, 8, "fp32", True, True, 2, 4)]
    table = [ts[0].entry(wt), {"n": 0}, ts[1].entry(wt), ts[2].entry(wt), {"n": 0}, ts[3].entry(wt)]
    before = [t.snapshot() for t in ts]
    with wt.AdamW(table, 8) as a:
        assert a.info()["n_tensors"] == 4 and a.info()["n_vector_tensors"] == 2
        a.step(h, 0)
        torch.cuda.synchronize()
    check_all(ts, before, [t.snapshot() for t in ts], h)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [0.01, 1e6])
def test_clipping_by_the_global_norm(wt, bits, max_norm):
    norm = torch.full((3,), -1.0, device="cuda")
    h = hyper(wt, max_norm=max_norm, norm_out=norm.data_ptr() + 4, grad_scale=-2.0)
    ts = [Tensor(n, bits, "bf16" if i % 2 else "fp32", True, True, i % 2, seed=i) for i, n in enumerate(SIZES * 3)]
    before, after = run(wt, ts, h, bits)
    want = exact_norm(ts, before, 2.0)
    got = norm.tolist()
    assert got[0] == got[2] == -1.0
    # 16 squares in fp32 per partial sum (17 roundings), the rest in 64 bits, one rounding of the root
    assert abs(got[1] - want) <= 12 * R.EPS32 * want
    check_all(ts, before, after, h, min(1.0, max_norm / (want + 1e-6)))


def test_norm_alone_and_over_many_items(wt):
    # more items than the norm kernel has workgroups; no clipping asked for
    norm = torch.zeros(1, device="cuda")
    h = hyper(wt, norm_out=norm.data_ptr(), grad_scale=1.0, lr=0.0)
    n = 1500 * 4096 + 77
    t = Tensor(n, 32, "bf16", True, True, seed=3, spread=0.1)
    before, _ = run(wt, [t], h, 32)
    want = exact_norm([t], [before[0]], 1.0)
    assert abs(float(norm) - want) <= 12 * R.EPS32 * want
    with wt.AdamW([{"n": 0}]) as a:  # no elements: the norm of nothing
        norm.fill_(5)
        a.step(h, 0)
        assert float(norm) == 0.0


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("value", [1e-18, 3e18, 4.7e18, 6.6e18, 1.8e19])
def test_norm_up_to_the_greatest_square(wt, bits, grad, shift, value):
    # every gradient as large as a square allows: only each square, not a sum of them, has to fit fp32
    norm = torch.zeros(1, device="cuda")
    ts = [Tensor(n, bits, grad, True, True, shift, seed=n) for n in (5000, 37)]
    for t in ts:
        t.set("grad", torch.where(torch.arange(t.n) % 3 == 1, -value, value).to(t.dtype["grad"]))
    h = hyper(wt, max_norm=1.0, norm_out=norm.data_ptr(), grad_scale=0.5)
    before, after = run(wt, ts, h, bits)
    want = exact_norm(ts, before, 0.5)
    # a square rounded once, halved by the root, and the norm rounded once
    assert abs(float(norm) - want) <= 2 * R.EPS32 * want
    check_all(ts, before, after, h, min(1.0, 1.0 / (want + 1e-6)))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite(wt, bits, value):
    ts = [Tensor(n, bits, "fp32", True, True, seed=n) for n in (500, 4096)]
    g = torch.from_numpy(ts[1].read("grad"))
    for at in (0, 1000, 4095):
        g[at] = value
    ts[1].set("grad", g)
    # with the norm computed, the step changes nothing
    norm = torch.zeros(1, device="cuda")
    before, after = run(wt, ts, hyper(wt, max_norm=1.0, norm_out=norm.data_ptr()), bits)
    assert not math.isfinite(float(norm))
    for b, a in zip(before, after):
        for k in b:
            assert np.array_equal(b[k].view(np.uint8), a[k].view(np.uint8)), k
    # without it, what is not finite stays with its element
    h = hyper(wt)
    before, after = run(wt, ts, h, bits)
    check_all(ts, before, after, h)
    assert np.isnan(after[1]["master"]).sum() == 3 and not np.isnan(after[0]["master"]).any()
    # and stays there in the next step, with a finite gradient again
    g[torch.tensor([0, 1000, 4095])] = 0.01
    ts[1].set("grad", g)
    before, after = run(wt, ts, hyper(wt, step=8), bits)
    bad = np.isnan(after[1]["master"])
    assert bad.sum() == 3 and bad[[0, 1000, 4095]].all()


def test_range_of_8_bit_states(wt):
    # blocks of zeros, of values too small to hold, of one large value among tiny ones, of large values
    n = 128 * 8
    t = Tensor(n, 8, "fp32", True, True, seed=5)
    g = np.zeros(n, dtype=np.float32)
    g[128:256] = 1e-33
    g[256:384] = 1e-9
    g[256] = 3.0
    g[384:512] = 1e8
    g[512:640] = np.exp2(np.linspace(-40, 0, 128)).astype(np.float32)
    g[640:768] = -1e-18
    g[768:] = 1.0
    t.set("grad", torch.from_numpy(g))
    for k in ("m", "v"):
        t.set(k, torch.zeros(n, dtype=torch.uint8))
        t.set(k + "_scale", torch.ones(8))
    h = hyper(wt, step=1, grad_scale=1.0)
    before, after = run(wt, [t], h, 8)
    check_all([t], before, after, h)
    a = after[0]
    assert (a["m"][:256] == 0).all() and (a["v"][:128] == 0).all()
    assert (a["m_scale"][:2] == 1).all() and a["v_scale"][0] == 1
    assert (a["v"][257:384] == 1).all()  # the smallest code, never zero
    # the first step's update is close to lr * sign(g) wherever the gradient is well above eps
    _, gg, _, _ = values(t, before[0])
    p0, p1 = before[0]["master"].astype(np.float64), a["master"].astype(np.float64)
    big = np.abs(gg) > 1e-5
    moved = (p1 - p0 * (1 - h.lr * t.wd))[big]
    assert np.all(np.abs(moved + h.lr * np.sign(gg[big])) <= h.lr * 2e-3 + 4 * R.EPS32)


def test_random_rounding_keeps_the_mean(wt):
    # the same step with 400 seeds: the mean of what is stored is within 5.5
    # standard errors of the exact value (a sum of 400 independent two-point
    # variables of spread at most one unit)
    n, runs = 512, 400
    src = Tensor(n, 8, "fp32", False, True, seed=9, spread=0.0)
    first = src.snapshot()
    p, g, m, v = values(src, first)
    h = hyper(wt)
    pn, mn, vn, *_ = R.step(p, g, m, v, lr=h.lr, beta1=h.beta1, beta2=h.beta2, eps=h.eps, wd=src.wd, gs=h.grad_scale, t=h.step)
    sums = {"m": np.zeros(n), "v": np.zeros(n), "param": np.zeros(n)}
    start = {k: b.clone() for k, b in src.buf.items()}
    with wt.AdamW([src.entry(wt)], 8) as a:
        for k in range(runs):
            for name, b in src.buf.items():
                b.copy_(start[name])
            a.step(hyper(wt, seed=1000 + k), 0)
            s = src.snapshot()
            _, _, ms, _ = values(src, s)
            sums["m"] += ms
            sums["v"] += R.E4M3[s["v"]] * R.per_block(s["v_scale"].astype(np.float64), n)
            sums["param"] += R.bf16_value(s["param"])
    for name, x in (("m", mn), ("v", np.sqrt(vn)), ("param", pn)):
        a = np.abs(x)
        if name == "param":
            unit = np.exp2(np.floor(np.log2(a)) - 7)
        else:
            sc = R.per_block(R.block_amax(x) / 448, n)
            unit = np.exp2(np.floor(np.log2(np.maximum(a / sc, 2.0 ** -6))) - 3) * sc
        low = a < 2.0 ** -9 * (sc if name == "v" else 0)  # held up by the smallest code
        frac = a / unit - np.floor(a / unit)
        se = unit * np.sqrt(frac * (1 - frac) / runs) + 1e-5 * unit
        z = (np.abs(sums[name] / runs) - a) / se
        z = z[~low]
        log(f"  {name}: largest |z| {np.abs(z).max():.2f}, mean z {z.mean():.3f}")
        assert np.abs(z).max() < 5.5 and abs(z.mean()) < 5.5 / math.sqrt(z.size)


def test_same_seed_repeats_and_another_differs(wt):
    def go(seed):
        t = Tensor(9000, 8, "bf16", False, True, seed=2)
        _, after = run(wt, [t], hyper(wt, seed=seed, max_norm=0.1), 8)
        return after[0]

    a, b, c = go(1), go(1), go(2)
    assert all(np.array_equal(a[k].view(np.uint8), b[k].view(np.uint8)) for k in a)
    assert (a["m"] != c["m"]).any() and (a["param"] != c["param"]).any()


@pytest.mark.parametrize("bits", [32, 8])
def test_many_steps(wt, bits):
    # twenty steps with a new gradient each, every step checked from the state before it
    ts = [Tensor(n, bits, "bf16", True, True, seed=n) for n in (129, 5000)]
    for t in ts:
        for k in ("m", "v"):
            t.set(k, torch.zeros(t.n, dtype=torch.uint8 if bits == 8 else torch.float32))
            if bits == 8:
                t.set(k + "_scale", torch.ones(R.blocks(t.n)))
    gen = torch.Generator().manual_seed(4)
    b0 = [0, R.blocks(129)]
    for step in range(1, 21):
        for t in ts:
            t.set("grad", (torch.randn(t.n, generator=gen) * 0.01).to(torch.bfloat16))
        h = hyper(wt, step=step, beta2=0.999)
        before, after = run(wt, ts, h, bits)
        for t, b, a, k in zip(ts, before, after, b0):
            check(t, b, a, k, h, what=f"step {step}")


@pytest.mark.parametrize("bits", [32, 8])
def test_capture_and_replay(wt, bits):
    # a captured clipped step, replayed with the step's number and learning rate read on the device, between
    # eager steps of another handle; each replay against the eager step from the same state
    def fresh():
        return [Tensor(n, bits, "bf16", True, True, seed=n) for n in (5000, 4096, 77)]

    ts, es = fresh(), fresh()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.zeros(1, device="cuda")
    norm, enorm = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    a, e = wt.AdamW([t.entry(wt) for t in ts], bits), wt.AdamW([t.entry(wt) for t in es], bits)
    start = [{k: b.clone() for k, b in t.buf.items()} for t in ts]
    s = torch.cuda.Stream()
    h = hyper(wt, max_norm=0.05, step=0, step_dev=step.data_ptr(), lr_dev=lr.data_ptr(), norm_out=norm.data_ptr())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        a.step(h, s.cuda_stream)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            a.step(h, s.cuda_stream)
    for t, b in zip(ts, start):
        for k in b:
            t.buf[k].copy_(b[k])
    torch.cuda.synchronize()
    for k in range(1, 6):
        rate = float(np.float32(1e-3 * k))
        step.fill_(k)
        lr.fill_(rate)
        for t, q in zip(ts, es):
            x = torch.full_like(t.buf["grad"], 0)
            x.copy_(t.buf["grad"])
            q.buf["grad"].copy_(x)
        g.replay()
        e.step(hyper(wt, max_norm=0.05, step=k, lr=rate, norm_out=enorm.data_ptr()), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert float(norm) == float(enorm) > 0
        for t, q in zip(ts, es):
            x, y = t.snapshot(), q.snapshot()
            for name in x:
                assert np.array_equal(x[name].view(np.uint8), y[name].view(np.uint8)), (k, name)
    del g
    a.close()
    e.close()


def test_on_another_stream_behind_its_work(wt):
    t = Tensor(300000, 8, "fp32", True, True, seed=1)
    s = torch.cuda.Stream()
    before = t.snapshot()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with wt.AdamW([t.entry(wt)], 8) as a:
        with torch.cuda.stream(s):
            for _ in range(5):
                big = big @ big * 1e-3
            raw = t.buf["grad"]
            raw[64:64 + 4 * t.n].view(torch.float32).mul_(2.0)
            a.step(hyper(wt), s.cuda_stream)
        s.synchronize()
    after = [t.snapshot()]
    before["grad"] = before["grad"] * 2
    check_all([t], [before], after, hyper(wt))


def test_offsets_past_32_bits(wt):
    # 1.1e9 elements: fp32 and BF16 byte offsets past 2^32
    n = (1 << 30) + 4096 * 5 + 321
    nb = R.blocks(n)
    g = torch.Generator(device="cuda").manual_seed(1)
    master = torch.empty(n, device="cuda").normal_(generator=g).mul_(0.02)
    grad = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    param = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(n, dtype=torch.uint8, device="cuda")
    v = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.ones(nb, device="cuda"), torch.ones(nb, device="cuda")
    at = (nb - 40) * 128
    before = master[at:].cpu().numpy().astype(np.float64)
    h = hyper(wt, step=1)
    with wt.AdamW([dict(param=param.data_ptr(), master=master.data_ptr(), grad=grad.data_ptr(), grad_dtype=1, n=n,
                        m=m.data_ptr(), v=v.data_ptr(), m_scale=ms.data_ptr(), v_scale=vs.data_ptr(),
                        weight_decay=0.1)], 8) as a:
        a.step(h, 0)
        torch.cuda.synchronize()
    gg = grad[at:].float().cpu().numpy().astype(np.float64)
    z = np.zeros_like(gg)
    pn, mn, vn, ep, em, ev, er = R.step(before, gg, z, z, lr=h.lr, beta1=h.beta1, beta2=h.beta2, eps=h.eps, wd=0.1,
                                        gs=h.grad_scale, t=1)
    got = master[at:].cpu().numpy()
    assert np.all(np.abs(got - pn) <= ep)
    assert torch.equal(param[at:].cpu(), torch.from_numpy(got).to(torch.bfloat16))
    w = R.words(h.seed, 1, 0, n - at, first=at)
    R.check_codes(m[at:].cpu().numpy(), ms[nb - 40:].cpu().numpy().astype(np.float64), mn, em,
                  (w & np.uint64(0xFFFF)) / 65536.0, False, "m")
    R.check_codes(v[at:].cpu().numpy(), vs[nb - 40:].cpu().numpy().astype(np.float64), np.sqrt(vn), er,
                  (w >> np.uint64(16)) / 65536.0, True, "v")


def test_handle_refuses_memory_it_cannot_use(wt):
    t = Tensor(256, 32, "fp32", True, True)
    host = torch.zeros(256)
    for name, ptr, status in (("grad", host.data_ptr(), wt.WT_E_INVAL),):
        with pytest.raises(wt.WtError) as e:
            wt.AdamW([dict(t.entry(wt), **{name: ptr})])
        assert e.value.status == status and name in str(e.value)
    with pytest.raises(wt.WtError) as e:
        wt.AdamW([t.entry(wt)], device=64)
    assert e.value.status == wt.WT_E_INVAL


def test_hyper_values_refused(wt):
    t = Tensor(256, 8, "fp32", True, True)
    before = t.snapshot()
    with wt.AdamW([t.entry(wt)], 8) as a:
        for k, x in (("lr", -1.0), ("lr", math.nan), ("lr", 2e6), ("beta1", 1.0), ("beta1", -0.1), ("beta2", 1.0),
                     ("beta2", math.nan), ("eps", 0.0), ("eps", math.inf), ("grad_scale", math.inf),
                     ("grad_scale", math.nan), ("max_norm", -1.0), ("max_norm", math.inf), ("step", 0)):
            with pytest.raises(wt.WtError) as e:
                a.step(hyper(wt, **{k: x}), 0)
            assert e.value.status == wt.WT_E_INVAL and k.split("_")[0].rstrip("12") in str(e.value), str(e.value)
        for k in ("step_dev", "lr_dev", "norm_out"):
            with pytest.raises(wt.WtError) as e:
                a.step(hyper(wt, **{k: 0x1002}), 0)
            assert e.value.status == wt.WT_E_ALIGN
        with pytest.raises(wt.WtError) as e:
            wt.wt_adamw_step(0, hyper(wt), 0)
        assert e.value.status == wt.WT_E_INVAL
    torch.cuda.synchronize()
    after = t.snapshot()
    assert all(np.array_equal(before[k].view(np.uint8), after[k].view(np.uint8)) for k in before)


@pytest.mark.parametrize("bits", [32, 8])
def test_step_then_prepare_of_the_same_shards(wt, bits):
    # what a training step and the transfer behind it do: update the shards in place, prepare them on the same
    # stream; the destination is the oracle's image of the updated shards
    wl = W.custom([(256, 384), (130, 384), (64, 384)], n_shards=3, fused=True, device="cuda")
    shards = [s for o in wl.outputs for p in o.parts for s, r in zip(p.shards, p.shard_rows) if r]
    old = [s.clone() for s in shards]
    gen = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(s.shape, generator=gen, device="cuda") for s in shards]
    dst = torch.full((wl.dst_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream()
    with wt.AdamW.for_workload(wl, grads, state_bits=bits, weight_decay=0.1) as opt, wt.Plan(wl, dst) as plan:
        for step in (1, 2, 3):
            opt.step(hyper(wt, step=step, max_norm=1.0), s.cuda_stream)
            plan.prepare(s.cuda_stream)
        s.synchronize()
    assert all((a != b).float().mean() > 0.5 for a, b in zip(old, shards))
    assert_images_equal(dst.cpu().numpy(), oracle_image_threaded(wl), wl)


@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("exponent", [-20, 0, 16])
def test_stored_states_equal_separate_fp32_operations(wt, grad, exponent):
    # codes and scales bit for bit: every product, sum, root and quotient rounded by itself, as numpy's fp32 does
    n = 128 * 700 + 55
    t = Tensor(n, 8, grad, True, True, seed=21 + exponent, spread=2.0)
    f = np.float32
    for k, up in (("grad", 1), ("m_scale", 1), ("v_scale", 1)):
        x = torch.from_numpy(t.read(k).view(np.int16) if t.dtype[k] == torch.bfloat16 else t.read(k))
        x = x.view(torch.bfloat16) if t.dtype[k] == torch.bfloat16 else x
        t.set(k, x * 2.0 ** exponent)
    h = hyper(wt, seed=99)
    before, after = run(wt, [t], h, 8)
    b, a = before[0], after[0]
    g = (R.bf16_value(b["grad"]).astype(f) if grad == "bf16" else b["grad"]) * f(h.grad_scale)
    m = R.E4M3[b["m"]].astype(f) * R.per_block(b["m_scale"], n)
    r = R.E4M3[b["v"]].astype(f) * R.per_block(b["v_scale"], n)
    m = f(h.beta1) * m + f(1 - h.beta1) * g
    root = np.sqrt(f(h.beta2) * (r * r) + f(1 - h.beta2) * (g * g))
    assert m.dtype == root.dtype == f
    w = R.words(h.seed, h.step, 0, n)
    for name, x, bits in (("m", m, w & np.uint64(0xFFFF)), ("v", root, w >> np.uint64(16))):
        amax = R.block_amax(x.astype(np.float64)).astype(f)
        assert np.array_equal(a[name + "_scale"], amax / f(448)), name
        y = np.abs(x * R.per_block(f(448) / amax, n))
        if name == "v":
            y = np.where(x > 0, np.maximum(y, f(2.0 ** -9)), y)
        want = R.e4m3_up(np.minimum(y, f(448)).astype(np.float64), bits.astype(np.float64) / 65536)
        assert np.array_equal(np.abs(R.E4M3[a[name]]), want), name
