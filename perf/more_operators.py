"""Speed cases of the experts' feed-forward operators: the gated block (both
projections, the activation and the product) with its backward pass, the
products that go with it, and microscaled 4-bit floating point (MXFP4), its
quantisation and its products. Rows are grouped by expert as the row map of a
dispatch leaves them; a dense layer is one expert.

`own = False` computes each operator in its plain form from elementary torch
operations; `own = True` calls the library (bf16_fp8_weight_amd.wt).
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
MX = 32  # elements that share one scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a dense layer of hidden size 1024: the latency of a call
        dict(name="gated_token", op="gated", rows=1, experts=1, hidden=1024, inter=2816, align=1, act="silu",
             pre=False),
        # a decode step's token copies over one GPU's share of a large MoE layer: two or three rows an expert
        dict(name="gated_decode", op="gated", rows=256, experts=96, hidden=7168, inter=2048, align=1, act="silu",
             pre=False),
        # a training batch over a quarter of these experts, gathered from its tokens, pre-activations kept
        dict(name="gated_batch", op="gated", rows=16384, experts=24, hidden=7168, inter=2048, align=128, act="silu",
             pre=True),
        # the projection back: of the decode step, and of a 7B-shaped dense layer
        dict(name="down_decode", op="product", rows=256, experts=96, k=2048, n=7168, align=1, out="bf16"),
        dict(name="down_batch", op="product", rows=8191, experts=1, k=11008, n=4096, align=1, out="fp32"),
        # gradients of an odd little block, and of a batch over 12 experts
        dict(name="grad_ragged", op="grad", rows=1003, experts=5, hidden=1000, inter=1368, align=1, act="gelu"),
        dict(name="grad_batch", op="grad", rows=8192, experts=12, hidden=7168, inter=2048, align=128, act="silu"),
        # rounding to MXFP4 and the values that it stands for: tokens sent to their experts, a layer's gate_up weights
        dict(name="mx_tokens", op="mx_round", rows=1024, tokens=128, cols=7168, dtype="bf16"),
        dict(name="mx_weights", op="mx_round", rows=22016, tokens=0, cols=4096, dtype="bf16"),
        # MXFP4 weights: one token of a dense layer, the decode step, a prefill batch (rows quantised in the pass)
        dict(name="mx_down_token", op="mx", rows=1, experts=1, k=2816, n=1024, align=1, gated=False, act="silu"),
        dict(name="mx_gated_decode", op="mx", rows=256, experts=96, k=7168, n=2048, align=1, gated=True, act="silu"),
        dict(name="mx_gated_batch", op="mx", rows=16384, experts=24, k=7168, n=2048, align=128, gated=True,
             act="silu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A row length: mostly whole 128-byte lines, now and then any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.2 else max(64, n // 64 * 64) if rng.random() < 0.7 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["gated", "gated", "product", "grad", "mx_round", "mx", "mx"])
    if op == "mx_round":
        cols = _size(rng, 64, 8192)
        rows = _log(rng, 1, 22016 * 4096 // max(cols, 4096))
        return dict(op=op, rows=rows, tokens=rng.choice([0, max(1, rows // 8)]), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    experts = rng.choice([1, 1, _log(rng, 2, 96)])
    rows = _log(rng, 1, 8192 if op == "grad" else 16384)
    a, b = _size(rng, 64, 7168), _size(rng, 64, 4096)
    while a * b * experts > 96 * 7168 * 2048 or (op == "grad" and a * b * experts > 12 * 7168 * 2048) \
            or rows * a * b > 8192 * 7168 * 2048:
        experts, rows, b = max(1, experts // 2), max(1, rows * 2 // 3), max(64, b // 2)
    c = dict(op=op, rows=rows, experts=experts, align=rng.choice([1, 16, 128]) if experts > 1 else 1)
    act = rng.choice(["silu", "silu", "gelu"])
    if op == "product":
        return dict(c, k=a, n=b, out=rng.choice(["bf16", "fp32"]))
    if op == "mx":
        return dict(c, k=a, n=b, gated=rng.random() < 0.6, act=act)
    c.update(hidden=a, inter=b, act=act)
    return dict(c, pre=rng.random() < 0.5) if op == "gated" else c


# ------------------------------------------------------------------ prepare
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    """Matrix by matrix, so that no 32-bit copy of a whole stack of weights is held."""
    if len(shape) == 2:
        return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(dtype)
    return torch.stack([_normal(g, *shape[1:], std=std, dtype=dtype) for _ in range(shape[0])])


def _rows(case, seed):
    """Rows of each expert as a row map has them: uneven counts, first rows at multiples of `align`."""
    E, R, align = case["experts"], case["rows"], case["align"]
    s = dict(case=case, n_rows=R, n_experts=E, offsets=None, counts=None, row_token=None)
    if E == 1:
        s.update(slots=torch.arange(R, device=DEV)[None, :])
        return s
    r = random.Random(seed)
    popular = [math.exp(r.gauss(0.0, 0.5)) for _ in range(E)]
    counts = [0] * E
    for e in r.choices(range(E), popular, k=R):
        counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + -(-c // align) * align)
    n_rows = R + min(E, R) * (align - 1)
    g = _gen(seed + 1)
    s.update(n_rows=n_rows, offsets=torch.tensor(offsets, dtype=torch.int32, device=DEV),
             counts=torch.tensor(counts, dtype=torch.int32, device=DEV))
    # the rows of each expert side by side, padded to the longest (n_rows: none)
    at = torch.arange(max(counts), device=DEV)[None, :]
    s["slots"] = torch.where(at < s["counts"][:, None], s["offsets"][:-1, None] + at, n_rows).long()
    s["tokens"] = max(1, R // 8)
    token = torch.full((n_rows + 1,), -1, dtype=torch.int32, device=DEV)
    picked = torch.randint(0, s["tokens"], (n_rows + 1,), generator=g, device=DEV, dtype=torch.int32)
    live = s["slots"].reshape(-1)
    token[live] = picked[live]
    token[n_rows] = -1
    s["row_token"] = token[:-1].contiguous()
    return s


def prepare(case, seed):
    return {"gated": _prepare_gated, "product": _prepare_product, "grad": _prepare_grad, "mx_round": _prepare_round,
            "mx": _prepare_mx}[case["op"]](case, seed)


def _hidden_states(s, g, n):
    """What the rows are taken from: the batch's tokens, or the rows themselves in a dense layer."""
    return _normal(g, s["tokens"] if s["row_token"] is not None else s["n_rows"], n)


def _desc(s, wt, form, n, k, a, b, out, act="silu", gather=False, m=0):
    d = wt.wt_product_desc_init()
    d.n_rows, d.n_experts, d.form, d.m, d.n, d.k = s["n_rows"], s["n_experts"], form, m, n, k
    d.act = wt.WT_ACT_GELU if act == "gelu" else wt.WT_ACT_SILU
    if s["offsets"] is not None:
        d.offsets, d.counts = s["offsets"].data_ptr(), s["counts"].data_ptr()
        if gather:
            d.row_index, d.n_index_rows = s["row_token"].data_ptr(), s["tokens"]
    d.a, d.a_stride = a.data_ptr(), a.stride(0)
    d.b, d.b_stride = b.data_ptr(), b.stride(-2)
    d.out, d.out_stride = out.data_ptr(), out.stride(-2)
    d.out_dtype = wt.WT_DT_F32 if out.dtype == torch.float32 else wt.WT_DT_BF16
    if b.dim() == 3:
        d.b_expert_stride = b.stride(0)
    if out.dim() == 3:
        d.out_expert_stride = out.stride(0)
    return d


def _prepare_gated(case, seed):
    s, g = _rows(case, seed), _gen(seed)
    H, N = case["hidden"], case["inter"]
    s.update(x=_hidden_states(s, g, H), w=_normal(g, s["n_experts"], 2 * N, H, std=H ** -0.5),
             h=torch.zeros(s["n_rows"], N, dtype=torch.bfloat16, device=DEV),
             pre=torch.zeros(s["n_rows"], 2 * N, dtype=torch.bfloat16, device=DEV) if case["pre"] else None)
    if own:
        from bf16_fp8_weight_amd import wt

        s["desc"] = _desc(s, wt, wt.WT_PRODUCT_NT, N, H, s["x"], s["w"], s["h"], act=case["act"], gather=True)
    return s


def _prepare_product(case, seed):
    s, g = _rows(case, seed), _gen(seed)
    s.update(x=_normal(g, s["n_rows"], case["k"]), w=_normal(g, s["n_experts"], case["n"], case["k"],
                                                             std=case["k"] ** -0.5),
             out=torch.zeros(s["n_rows"], case["n"], dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16,
                             device=DEV))
    if own:
        from bf16_fp8_weight_amd import wt

        s["desc"] = _desc(s, wt, wt.WT_PRODUCT_NT, case["n"], case["k"], s["x"], s["w"], s["out"])
    return s


def _prepare_grad(case, seed):
    s, g = _rows(case, seed), _gen(seed)
    E, R, H, N = s["n_experts"], s["n_rows"], case["hidden"], case["inter"]
    s.update(x=_hidden_states(s, g, H), w=_normal(g, E, 2 * N, H, std=H ** -0.5),
             down=_normal(g, E, H, N, std=N ** -0.5), dy=_normal(g, R, H, std=0.01),
             pre=torch.zeros(R, 2 * N, dtype=torch.bfloat16, device=DEV),
             h=torch.zeros(R, N, dtype=torch.bfloat16, device=DEV), dx=torch.zeros(R, H, dtype=torch.bfloat16, device=DEV),
             dw=torch.zeros(E, 2 * N, H, dtype=torch.bfloat16, device=DEV),
             ddown=torch.zeros(E, H, N, dtype=torch.bfloat16, device=DEV))
    f = _plain_gated(s)  # what the forward pass left
    s["pre"].copy_(f["pre"])
    s["h"].copy_(f["h"])
    if own:
        from bf16_fp8_weight_amd import wt

        s["dpre"] = torch.zeros(R, 2 * N, dtype=torch.bfloat16, device=DEV)
        nn, tn = wt.WT_PRODUCT_NN, wt.WT_PRODUCT_TN
        s["d_gated"] = _desc(s, wt, nn, N, H, s["dy"], s["down"], s["dpre"], act=case["act"])
        s["d_x"] = _desc(s, wt, nn, H, 2 * N, s["dpre"], s["w"], s["dx"])
        s["d_w"] = _desc(s, wt, tn, H, 0, s["dpre"], s["x"], s["dw"], gather=True, m=2 * N)
        s["d_down"] = _desc(s, wt, tn, N, 0, s["dy"], s["h"], s["ddown"], m=H)
    return s


def _prepare_round(case, seed):
    g = _gen(seed)
    R, K, T = case["rows"], case["cols"], case["tokens"]
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    # a few channels much larger than the others, as hidden states have them
    wide = torch.exp(torch.randn(K, generator=g, device=DEV) * 0.7)
    x = (torch.randn(T or R, K, generator=g, device=DEV) * wide).to(dtype)
    index = torch.randint(0, T, (R,), generator=g, device=DEV, dtype=torch.int32) if T else None
    nb = -(-K // MX)
    return dict(case=case, x=x, index=index, codes=torch.zeros(R, 16 * nb, dtype=torch.uint8, device=DEV),
                scales=torch.zeros(R, -(-nb // 4) * 4, dtype=torch.uint8, device=DEV),
                values=torch.zeros(R, K, dtype=dtype, device=DEV))


def _prepare_mx(case, seed):
    s, g = _rows(case, seed), _gen(seed)
    E, N, K = s["n_experts"], case["n"] * (2 if case["gated"] else 1), case["k"]
    nb = -(-K // MX)
    codes = torch.zeros(E, N, 16 * nb, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(E, N, -(-nb // 4) * 4, dtype=torch.uint8, device=DEV)
    for e in range(E):  # weights are quantised once, when they are loaded
        q, b = _round_mx(_normal(g, N, K, std=K ** -0.5).float())
        codes[e], scales[e] = _pack(q), b
    s.update(x=_hidden_states(s, g, K), codes=codes, scales=scales,
             a_codes=torch.zeros(s["n_rows"], 16 * nb, dtype=torch.uint8, device=DEV),
             a_scales=torch.zeros(s["n_rows"], scales.shape[2], dtype=torch.uint8, device=DEV),
             out=torch.zeros(s["n_rows"], case["n"], dtype=torch.bfloat16, device=DEV))
    if own:
        from bf16_fp8_weight_amd import wt

        d = s["desc"] = wt.wt_mxfp4_product_desc_init()
        d.n_rows, d.n_experts, d.n, d.k, d.gated = s["n_rows"], E, case["n"], K, int(case["gated"])
        d.act = wt.WT_ACT_GELU if case["act"] == "gelu" else wt.WT_ACT_SILU
        if s["offsets"] is not None:
            d.offsets, d.counts = s["offsets"].data_ptr(), s["counts"].data_ptr()
        d.a, d.a_stride = s["a_codes"].data_ptr(), s["a_codes"].stride(0)
        d.a_scales, d.a_scale_stride = s["a_scales"].data_ptr(), s["a_scales"].stride(0)
        d.b, d.b_stride, d.b_expert_stride = codes.data_ptr(), codes.stride(1), codes.stride(0)
        d.b_scales, d.b_scale_stride, d.b_scale_expert_stride = scales.data_ptr(), scales.stride(1), scales.stride(0)
        d.out, d.out_stride, d.out_dtype = s["out"].data_ptr(), case["n"], wt.WT_DT_BF16
    return s


# ---------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if op == "gated":
        return _own_gated(state) if own else _plain_gated(state)
    if op == "product":
        return _own_product(state) if own else _plain_product(state)
    if op == "grad":
        return _own_grad(state) if own else _plain_grad(state)
    if op == "mx_round":
        return _own_round(state) if own else _plain_round(state)
    return _own_mx(state) if own else _plain_mx(state)


def _own_gated(s):
    from bf16_fp8_weight_amd import wt

    stream = torch.cuda.current_stream().cuda_stream
    if s["pre"] is None:
        wt.wt_gated_forward(s["desc"], 0, 0, stream)
        return {"h": s["h"]}
    wt.wt_gated_forward(s["desc"], s["pre"].data_ptr(), s["pre"].stride(0), stream)
    return {"h": s["h"], "pre": s["pre"]}


def _own_product(s):
    from bf16_fp8_weight_amd import wt

    wt.wt_expert_product(s["desc"], torch.cuda.current_stream().cuda_stream)
    return {"out": s["out"]}


def _own_grad(s):
    from bf16_fp8_weight_amd import wt

    stream = torch.cuda.current_stream().cuda_stream
    wt.wt_gated_backward(s["d_gated"], s["pre"].data_ptr(), s["pre"].stride(0), stream)
    wt.wt_expert_product(s["d_x"], stream)
    wt.wt_expert_product(s["d_w"], stream)
    wt.wt_expert_product(s["d_down"], stream)
    return {"dx": s["dx"], "dw_gate_up": s["dw"], "dw_down": s["ddown"]}


def _own_quantize(wt, x, index, n_out, cols, codes, scales, stream):
    wt.wt_mxfp4_quantize(x.data_ptr(), wt.WT_DT_F32 if x.dtype == torch.float32 else wt.WT_DT_BF16, x.shape[0], cols,
                         x.stride(0), index.data_ptr() if index is not None else 0, n_out, codes.data_ptr(),
                         codes.stride(0), scales.data_ptr(), scales.stride(0), stream)


def _own_round(s):
    from bf16_fp8_weight_amd import wt

    stream = torch.cuda.current_stream().cuda_stream
    R, K, v = s["case"]["rows"], s["case"]["cols"], s["values"]
    _own_quantize(wt, s["x"], s["index"], R, K, s["codes"], s["scales"], stream)
    wt.wt_mxfp4_dequantize(s["codes"].data_ptr(), s["codes"].stride(0), s["scales"].data_ptr(), s["scales"].stride(0),
                           R, K, v.data_ptr(), wt.WT_DT_F32 if v.dtype == torch.float32 else wt.WT_DT_BF16,
                           v.stride(0), stream)
    return {"values": v, "scales": s["scales"]}


def _own_mx(s):
    from bf16_fp8_weight_amd import wt

    stream = torch.cuda.current_stream().cuda_stream
    _own_quantize(wt, s["x"], s["row_token"], s["n_rows"], s["case"]["k"], s["a_codes"], s["a_scales"], stream)
    wt.wt_mxfp4_product(s["desc"], stream)
    return {"out": s["out"]}


# ------------------------------------------------------------- plain forms
def _take(s, x, gather=False):
    """[experts, longest, columns] in 32 bits: each expert's rows, zeros behind them."""
    rows = s["slots"]
    live = rows < s["n_rows"]
    at = rows.clamp(max=s["n_rows"] - 1)
    if gather and s["row_token"] is not None:
        at = s["row_token"].long()[at].clamp(min=0)
    return torch.where(live[:, :, None], x[at].float(), torch.zeros((), device=DEV))


def _put(s, y, dtype):
    """The rows back in their places; rows of no expert stay zero."""
    out = torch.zeros(s["n_rows"] + 1, y.shape[2], dtype=dtype, device=DEV)
    out[s["slots"]] = y.to(dtype)
    return out[:-1]


def _activation(kind, x):
    if kind == "silu":
        return x / (1 + torch.exp(-x))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _slope(kind, x):
    if kind == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def _plain_gated(s):
    n = s["case"]["inter"]
    y = _take(s, s["x"], gather=True) @ s["w"].float().transpose(1, 2)
    h = _put(s, _activation(s["case"]["act"], y[:, :, :n]) * y[:, :, n:], torch.bfloat16)
    return {"h": h} if s["pre"] is None else {"h": h, "pre": _put(s, y, torch.bfloat16)}


def _plain_product(s):
    return {"out": _put(s, _take(s, s["x"]) @ s["w"].float().transpose(1, 2), s["out"].dtype)}


def _plain_grad(s):
    n, act = s["case"]["inter"], s["case"]["act"]
    dy, pre, w = _take(s, s["dy"]), _take(s, s["pre"]), s["w"].float()
    dh = dy @ s["down"].float()
    gate, up = pre[:, :, :n], pre[:, :, n:]
    dpre = torch.cat([dh * up * _slope(act, gate), dh * _activation(act, gate)], dim=2)
    dw = dpre.transpose(1, 2) @ _take(s, s["x"], gather=True)
    ddown = dy.transpose(1, 2) @ _take(s, s["h"])
    return {"dx": _put(s, dpre @ w, torch.bfloat16), "dw_gate_up": dw.to(torch.bfloat16),
            "dw_down": ddown.to(torch.bfloat16)}


def _round_mx(x):
    """Codes (0 .. 15, one to an element, rows padded to whole blocks) and biased scale exponents of 32-bit rows."""
    R, K = x.shape
    nb = -(-K // MX)
    x = torch.nn.functional.pad(x, (0, nb * MX - K)).view(R, nb, MX)
    amax = x.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax).exponent - 3).clamp(min=-127), torch.zeros_like(amax, dtype=torch.int32))
    a = torch.ldexp(x.abs(), -e)
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / unit) * unit).clamp(max=6.0)
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    scales = torch.zeros(R, -(-nb // 4) * 4, dtype=torch.uint8, device=DEV)
    scales[:, :nb] = (e[:, :, 0] + 127).to(torch.uint8)
    return (code | (torch.signbit(x).to(torch.uint8) << 3)).view(R, nb * MX), scales


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _values(codes, scales):
    """What packed codes [..., bytes] and their scales stand for, in 32 bits."""
    v = torch.tensor([s * m for s in (1.0, -1.0) for m in E2M1], device=DEV)
    pairs = torch.stack([v.repeat(16), v.repeat_interleave(16)], dim=1)
    y = pairs[codes.int()].view(*codes.shape[:-1], codes.shape[-1] // 16, MX)
    size = torch.ldexp(torch.ones(256, device=DEV), torch.arange(256, device=DEV) - 127)
    return (y * size[scales[..., : y.shape[-2]].int()][..., None]).flatten(-2)


def _plain_round(s):
    x = s["x"].float() if s["index"] is None else s["x"].float()[s["index"].long()]
    code, scales = _round_mx(x)
    return {"values": _values(_pack(code), scales)[:, : s["case"]["cols"]].to(s["x"].dtype), "scales": scales}


def _plain_mx(s):
    n, k = s["case"]["n"], s["case"]["k"]
    code, scales = _round_mx(s["x"].float())
    a = _take(s, _values(_pack(code), scales)[:, :k], gather=True)
    y = a @ _values(s["codes"], s["scales"])[:, :, :k].transpose(1, 2)
    if s["case"]["gated"]:
        y = _activation(s["case"]["act"], y[:, :, :n]) * y[:, :, n:]
    return {"out": _put(s, y, torch.bfloat16)}


# --------------------------------------------------------------------- work
def work(case):
    R = case["rows"]
    if case["op"] == "mx_round":
        size, K, nb = 4 if case["dtype"] == "fp32" else 2, case["cols"], -(-case["cols"] // MX)
        return {"bytes": size * K * ((case["tokens"] or R) + R) + R * (16 * nb + nb + 4 * (case["tokens"] > 0)),
                "flops": 4 * R * K}
    # with fewer rows than experts some experts have nothing to read
    E = min(case["experts"], R)
    sent = 8 if case["experts"] > 1 else 1  # copies of a token
    if case["op"] == "product":
        k, n = case["k"], case["n"]
        return {"bytes": 2 * E * k * n + 2 * R * k + (4 if case["out"] == "fp32" else 2) * R * n, "flops": 2 * R * k * n}
    if case["op"] == "mx":
        k, n = case["k"], case["n"] * (2 if case["gated"] else 1)
        return {"bytes": E * k * n * (16 + 1) // 32 + 2 * R * k // sent + 2 * R * case["n"], "flops": 2 * R * k * n}
    H, N = case["hidden"], case["inter"]
    if case["op"] == "gated":
        return {"bytes": 2 * E * 2 * N * H + 2 * R * H // sent + 2 * R * N * (3 if case["pre"] else 1),
                "flops": 4 * R * H * N}
    E = case["experts"]  # gradients of experts without rows are written too
    return {"bytes": 2 * (2 * E * 3 * N * H + R * H // sent + R * (2 * H + 3 * N)), "flops": 12 * R * H * N}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits, expert by expert."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "mx_round":
        x = s["x"].double() if s["index"] is None else s["x"].double().index_select(0, s["index"].long())
        return {"values": _exact_mx(x), "scales": None}
    if op == "mx":
        y = s["x"].double()
        s["exact_x"] = _exact_mx(y)
    E, dev = s["n_experts"], dict(dtype=torch.float64, device=DEV)
    first = [0] if s["offsets"] is None else s["offsets"].tolist()
    count = [s["n_rows"]] if s["counts"] is None else s["counts"].tolist()
    out = {}

    def into(name, a, part):
        if name not in out:
            out[name] = torch.zeros(s["n_rows"], part.shape[1], **dev)
        out[name][a:a + part.shape[0]] = part

    for e in range(E):
        a, b = first[e], first[e] + count[e]
        tokens = torch.arange(a, b, device=DEV) if s["row_token"] is None else s["row_token"][a:b].long()
        if op == "product":
            into("out", a, torch.mm(s["x"][a:b].double(), s["w"][e].double().t()))
        elif op == "mx":
            w = _exact_values(s["codes"][e], s["scales"][e])[:, : case["k"]]
            y = torch.mm(s["exact_x"].index_select(0, tokens), w.t())
            into("out", a, _exact_gate(case, y) if case["gated"] else y)
        elif op == "gated":
            y = torch.mm(s["x"].index_select(0, tokens).double(), s["w"][e].double().t())
            into("h", a, _exact_gate(case, y))
            if case["pre"]:
                into("pre", a, y)
        else:
            dy, x, n = s["dy"][a:b].double(), s["x"].index_select(0, tokens).double(), case["inter"]
            y = s["pre"][a:b].double().requires_grad_()
            _exact_gate(case, y).backward(torch.mm(dy, s["down"][e].double()))
            into("dx", a, torch.mm(y.grad, s["w"][e].double()))
            out.setdefault("dw_gate_up", torch.zeros(E, 2 * n, case["hidden"], **dev))[e] = torch.mm(y.grad.t(), x)
            out.setdefault("dw_down", torch.zeros(E, case["hidden"], n, **dev))[e] = torch.mm(dy.t(), s["h"][a:b].double())
    return out


def _exact_gate(case, y):
    gate, up = y.chunk(2, dim=1)
    if case["act"] == "silu":
        return gate * torch.sigmoid(gate) * up
    return torch.nn.functional.gelu(gate, approximate="tanh") * up


def _exact_mx(x):
    """The nearest of the sixteen values times the block's power of two; of two equally near ones the even code."""
    R, K = x.shape
    blocks = torch.zeros(R, -(-K // MX) * MX, dtype=torch.float64, device=DEV)
    blocks[:, :K] = x
    blocks = blocks.reshape(-1, MX)
    top = blocks.abs().max(dim=1, keepdim=True).values
    size = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    middle = (grid[1:] + grid[:-1]) / 2
    y = blocks.abs() / size
    low, high = torch.searchsorted(middle, y), torch.searchsorted(middle, y, right=True)
    code = torch.where(low % 2 == 0, low, high)
    return (torch.sign(blocks) * grid[code] * size).view(R, -1)[:, :K]


def _exact_values(codes, scales):
    codes = torch.stack([codes % 16, codes // 16], dim=2).flatten(1)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    y = grid[(codes % 8).long()] * (1 - 2 * (codes // 8).double())
    size = torch.exp2(scales.double() - 127).repeat_interleave(MX, dim=1)
    return y * size[:, : y.shape[1]]
