"""Speed cases of the training-step operators that run next to a weight
transfer: the AdamW step over many parameter shards (states in 32 or 8 bits),
the expert router with its balance loss and per-expert counts (forward and
backward), and the row map that groups token copies by expert.

`own = False` computes each operator in its plain form from elementary torch
operations; `own = True` calls the library (bf16_fp8_weight_amd.wt).
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128  # elements that share one scale in an 8-bit state
M32 = 0xFFFFFFFF
M64 = (1 << 64) - 1


# ------------------------------------------------------------------- cases
def listed():
    return [
        # norm and bias vectors of a few layers, 8 row shards each: the step's latency over many tiny tensors
        dict(name="adamw32_vectors", op="adamw", bits=32, tensors=96, elements=896, ragged=False, grad="fp32",
             master=True, max_norm=0.0),
        # one rank's experts (24 shards each), the usual mixed-precision step: fp32 master, BF16 gradient and shard
        dict(name="adamw32_experts", op="adamw", bits=32, tensors=96, elements=1835008, ragged=False, grad="bf16",
             master=True, max_norm=0.0),
        # one dense layer of hidden size 1024 in its row shards, 8-bit states, clipped by the global norm
        dict(name="adamw8_layer", op="adamw", bits=8, tensors=24, elements=720896, ragged=False, grad="bf16",
             master=True, max_norm=1.0),
        # the experts again with 8-bit states
        dict(name="adamw8_experts", op="adamw", bits=8, tensors=96, elements=1835008, ragged=False, grad="bf16",
             master=True, max_norm=0.0),
        # odd sizes, no master copy (BF16 is the only copy of the weights), fp32 gradients, clipped
        dict(name="adamw8_ragged", op="adamw", bits=8, tensors=301, elements=300007, ragged=True, grad="fp32",
             master=False, max_norm=1.0),
        # one decode step's tokens: sigmoid scores with a selection bias
        dict(name="router_decode", op="router", tokens=128, experts=384, topk=8, score="sigmoid", normalize=True,
             bias=True, logits="fp32", seqs=1, masked=0),
        # a packed training batch
        dict(name="router_batch", op="router", tokens=16384, experts=384, topk=8, score="sigmoid", normalize=True,
             bias=True, logits="fp32", seqs=13, masked=0),
        # an odd batch, softmax scores from BF16 logits, some experts switched off
        dict(name="router_softmax", op="router", tokens=5003, experts=160, topk=6, score="softmax", normalize=False,
             bias=False, logits="bf16", seqs=3, masked=5),
        # the gradients of the two batches
        dict(name="router_grad_batch", op="router_grad", tokens=16384, experts=384, topk=8, score="sigmoid",
             normalize=True, bias=True, logits="fp32", seqs=13, masked=0),
        dict(name="router_grad_softmax", op="router_grad", tokens=5003, experts=160, topk=6, score="softmax",
             normalize=False, bias=False, logits="bf16", seqs=3, masked=5),
        # token copies grouped by expert for a dispatch: one decode step, and a batch padded to whole row tiles
        dict(name="rows_decode", op="rows", tokens=128, experts=384, topk=8, align=1),
        dict(name="rows_batch", op="rows", tokens=16384, experts=384, topk=8, align=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "router", "router_grad", "rows"])
    if op == "adamw":
        tensors = _log(rng, 1, 400)
        return dict(op=op, bits=rng.choice([32, 8]), tensors=tensors,
                    elements=_log(rng, 100, min(8_000_000, 170_000_000 // tensors)), ragged=rng.random() < 0.7,
                    grad=rng.choice(["bf16", "fp32"]), master=rng.random() < 0.6,
                    max_norm=rng.choice([0.0, 1.0]))
    experts = _log(rng, 8, 512)
    tokens = _log(rng, 1, 16384 * 384 // max(experts, 384))
    topk = rng.randint(1, min(12, experts // 2))
    if op == "rows":
        return dict(op=op, tokens=min(tokens, 16384 * 8 // topk), experts=experts, topk=topk,
                    align=rng.choice([1, 16, 128]))
    return dict(op=op, tokens=tokens, experts=experts, topk=topk, score=rng.choice(["sigmoid", "softmax"]),
                normalize=rng.random() < 0.5, bias=rng.random() < 0.5, logits=rng.choice(["fp32", "bf16"]),
                seqs=rng.randint(1, min(64, tokens)), masked=rng.choice([0, 0, 1, experts // 4]))


def _sizes(c):
    """Elements of each parameter shard of a step."""
    n, e = c["tensors"], c["elements"]
    if not c["ragged"]:
        # every second tensor of a layer is a smaller projection
        return [e if (i % 2 or e % 11) else max(1, 4 * e // 11) for i in range(n)]
    return [max(1, e * (1 + (37 * i) % n) // n - i % 7) for i in range(n)]


# ------------------------------------------------------------------ prepare
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    return {"adamw": _prepare_adamw, "router": _prepare_router, "router_grad": _prepare_router,
            "rows": _prepare_rows}[case["op"]](case, seed)


def _prepare_adamw(case, seed):
    """Flat buffers that hold every shard of a rank, each shard starting at a
    multiple of 128 elements (the padding between shards stays zero)."""
    g = _gen(seed)
    sizes = _sizes(case)
    blocks = [-(-n // BLOCK) for n in sizes]
    nb = sum(blocks)
    total = nb * BLOCK
    n_of = torch.tensor(sizes, device=DEV)
    b_of = torch.tensor(blocks, device=DEV)
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), b_of)
    first = torch.cumsum(b_of, 0) - b_of
    left = n_of[tensor] - (torch.arange(nb, device=DEV) - first[tensor]) * BLOCK
    live = torch.arange(BLOCK, device=DEV)[None, :] < left[:, None]
    block_std = torch.exp(torch.randn(nb, 1, generator=g, device=DEV))
    grad = torch.randn(nb, BLOCK, generator=g, device=DEV).mul_(block_std * 1e-3).mul_(live)
    first_moment = torch.randn(nb, BLOCK, generator=g, device=DEV).mul_(block_std * 3e-4).mul_(live)
    root = torch.randn(nb, BLOCK, generator=g, device=DEV).mul_(0.5).exp_().mul_(block_std * 1e-3).mul_(live)
    weights = torch.randn(nb, BLOCK, generator=g, device=DEV).mul_(0.02).mul_(live)
    decay = torch.tensor([0.0 if i % 5 == 4 else 0.1 for i in range(len(sizes))], device=DEV)
    s = dict(case=case, sizes=sizes, blocks=blocks, total=total, step=1000, seed=seed & 0xFFFFFF,
             lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, grad_scale=1.0, max_norm=case["max_norm"],
             decay=decay[tensor][:, None], decays=decay.tolist(),
             grad=grad.to(torch.bfloat16 if case["grad"] == "bf16" else torch.float32).reshape(-1),
             param=weights.to(torch.bfloat16).reshape(-1),
             master=weights.reshape(-1) if case["master"] else None,
             norm=torch.zeros(1, device=DEV))
    if case["bits"] == 32:
        s.update(m=first_moment.reshape(-1), v=root.square_().reshape(-1))
    else:
        for name, x in (("m", first_moment), ("v", root)):
            scale = x.abs().amax(1) / 448.0
            scale = torch.where(scale > 0, scale, torch.ones_like(scale))
            s[name] = (x / scale[:, None]).to(torch.float8_e4m3fn).reshape(-1)
            s[name + "_scale"] = scale
    if own:
        from bf16_fp8_weight_amd import wt

        tensors, at = [], 0
        for i, (n, b) in enumerate(zip(sizes, blocks)):
            t = dict(param=s["param"].data_ptr() + 2 * at, n=n, lr_mul=1.0, weight_decay=s["decays"][i],
                     grad=s["grad"].data_ptr() + s["grad"].element_size() * at,
                     grad_dtype=wt.WT_DT_BF16 if case["grad"] == "bf16" else wt.WT_DT_F32,
                     m=s["m"].data_ptr() + s["m"].element_size() * at,
                     v=s["v"].data_ptr() + s["v"].element_size() * at)
            if case["master"]:
                t["master"] = s["master"].data_ptr() + 4 * at
            if case["bits"] == 8:
                t["m_scale"] = s["m_scale"].data_ptr() + 4 * (at // BLOCK)
                t["v_scale"] = s["v_scale"].data_ptr() + 4 * (at // BLOCK)
            tensors.append(t)
            at += b * BLOCK
        s["plan"] = wt.AdamW(tensors, state_bits=case["bits"])
        s["hyper"] = wt.wt_adamw_hyper_init()
        s["hyper"].lr, s["hyper"].beta1, s["hyper"].beta2, s["hyper"].eps = s["lr"], s["beta1"], s["beta2"], s["eps"]
        s["hyper"].grad_scale, s["hyper"].max_norm, s["hyper"].seed = s["grad_scale"], s["max_norm"], s["seed"]
        if case["max_norm"] > 0:
            s["hyper"].norm_out = s["norm"].data_ptr()
    return s


def _logits(case, g):
    T, E = case["tokens"], case["experts"]
    x = torch.randn(T, E, generator=g, device=DEV)
    x += 0.5 * torch.randn(1, E, generator=g, device=DEV)  # some experts are more popular than others
    if case["masked"]:
        x[:, torch.randperm(E, generator=g, device=DEV)[: case["masked"]]] = -math.inf
    return x.to(torch.bfloat16 if case["logits"] == "bf16" else torch.float32)


def _prepare_router(case, seed):
    g = _gen(seed)
    T, E, K, S = case["tokens"], case["experts"], case["topk"], case["seqs"]
    # sequences of different lengths back to back; a batch of several ends in a few rows of padding
    cuts = torch.sort(torch.randperm(T, generator=g, device=DEV)[: S - 1]).values if S > 1 else \
        torch.zeros(0, dtype=torch.int64, device=DEV)
    end = T - (T // 50 if S > 1 else 0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cuts.clamp(max=end),
                         torch.tensor([end], device=DEV)]).to(torch.int32)
    s = dict(case=case, logits=_logits(case, g), offsets=offsets, scale=2.5, coef=0.001,
             bias=0.02 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None,
             index=torch.empty(T, K, dtype=torch.int32, device=DEV),
             weight=torch.empty(T, K, device=DEV), counts=torch.empty(E, dtype=torch.int32, device=DEV),
             seq_counts=torch.empty(S, E, dtype=torch.int32, device=DEV), loss=torch.empty(1, device=DEV))
    if case["op"] == "router_grad":
        f = _plain_router(s)
        s.update(index=f["index"], seq_counts=f["seq_counts"],
                 dweight=torch.randn(T, K, generator=g, device=DEV) * 0.01,
                 dloss=torch.rand(1, generator=g, device=DEV) + 0.5, dlogits=torch.empty_like(s["logits"]))
    if own:
        from bf16_fp8_weight_amd import wt

        s["router"] = wt.wt_router_desc_init()
        d = s["router"]
        d.n_tokens, d.n_experts, d.top_k, d.n_seqs = T, E, K, S
        d.logits, d.logits_stride = s["logits"].data_ptr(), E
        d.logits_dtype = wt.WT_DT_BF16 if case["logits"] == "bf16" else wt.WT_DT_F32
        d.score = wt.WT_SCORE_SIGMOID if case["score"] == "sigmoid" else wt.WT_SCORE_SOFTMAX
        d.normalize, d.scale, d.balance_coef = int(case["normalize"]), s["scale"], s["coef"]
        d.bias = s["bias"].data_ptr() if s["bias"] is not None else None
        d.seq_offsets = offsets.data_ptr()
        s["workspace"] = torch.empty(wt.wt_router_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    return s


def _rows_capacity(case):
    return case["tokens"] * case["topk"] + min(case["experts"], case["tokens"] * case["topk"]) * (case["align"] - 1)


def _prepare_rows(case, seed):
    g = _gen(seed)
    T, E, K = case["tokens"], case["experts"], case["topk"]
    popular = 0.5 * torch.randn(1, E, generator=g, device=DEV)
    index = (torch.randn(T, E, generator=g, device=DEV) + popular).topk(K, dim=1).indices.to(torch.int32)
    index[torch.rand(T, generator=g, device=DEV) < 0.02] = -1  # padding rows of the batch
    n_rows = _rows_capacity(case)
    s = dict(case=case, index=index, n_rows=n_rows, row_token=torch.empty(n_rows, dtype=torch.int32, device=DEV),
             pair_row=torch.empty(T, K, dtype=torch.int32, device=DEV),
             offsets=torch.empty(E + 1, dtype=torch.int32, device=DEV),
             counts=torch.empty(E, dtype=torch.int32, device=DEV))
    if own:
        from bf16_fp8_weight_amd import wt

        s["workspace"] = torch.empty(max(1, wt.wt_dispatch_workspace_bytes(T, K, E)), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if op == "adamw":
        return _run_adamw(state)
    if op == "router":
        return _own_router(state) if own else _plain_router(state)
    if op == "router_grad":
        return _own_router_grad(state) if own else _plain_router_grad(state)
    return _own_rows(state) if own else _plain_rows(state)


def _run_adamw(s):
    s["step"] += 1
    if own:
        from bf16_fp8_weight_amd import wt

        s["hyper"].step = s["step"]
        wt.wt_adamw_step(s["plan"].handle, s["hyper"], torch.cuda.current_stream().cuda_stream)
    else:
        _plain_adamw(s)
    names = ["param", "m", "v"] + (["master"] if s["case"]["master"] else []) + \
        (["m_scale", "v_scale"] if s["case"]["bits"] == 8 else []) + (["norm"] if s["max_norm"] > 0 else [])
    return {k: s[k] for k in names}


def _own_router(s):
    from bf16_fp8_weight_amd import wt

    wt.wt_router_forward(s["router"], s["index"].data_ptr(), s["weight"].data_ptr(), s["counts"].data_ptr(),
                         s["seq_counts"].data_ptr(), s["loss"].data_ptr(), s["workspace"].data_ptr(),
                         s["workspace"].numel(), torch.cuda.current_stream().cuda_stream)
    return {k: s[k] for k in ("index", "weight", "counts", "seq_counts", "loss")}


def _own_router_grad(s):
    from bf16_fp8_weight_amd import wt

    wt.wt_router_backward(s["router"], s["index"].data_ptr(), s["seq_counts"].data_ptr(), s["dweight"].data_ptr(),
                          s["dloss"].data_ptr(), s["dlogits"].data_ptr(), s["dlogits"].stride(0),
                          torch.cuda.current_stream().cuda_stream)
    return {"dlogits": s["dlogits"]}


def _own_rows(s):
    from bf16_fp8_weight_amd import wt

    c = s["case"]
    wt.wt_dispatch_rows(s["index"].data_ptr(), c["tokens"], c["topk"], c["experts"], c["align"], s["n_rows"],
                        s["row_token"].data_ptr(), s["pair_row"].data_ptr(), s["offsets"].data_ptr(),
                        s["counts"].data_ptr(), s["workspace"].data_ptr(), s["workspace"].numel(),
                        torch.cuda.current_stream().cuda_stream)
    return {k: s[k] for k in ("row_token", "pair_row", "offsets", "counts")}


# ------------------------------------------------------------- plain forms
def _mix(x):
    """A 32-bit mixing function (xor-shifts and odd multipliers) on int64 tensors."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & M32
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & M32
    return x ^ (x >> 16)


def _keys(seed, step):
    z = (seed + step * 0x9E3779B97F4A7C15) & M64
    z ^= z >> 32
    z = (z * 0x6A09E667F3BCC909) & M64
    z ^= z >> 29
    z = (z * 0xBB67AE8584CAA73B) & M64
    z ^= z >> 32
    return z & M32, z >> 32


def _random_words(s):
    """One 32-bit word per element, from the step's keys and the element's place."""
    k0, k1 = _keys(s["seed"], s["step"])
    block = (_mix(torch.arange(s["total"] // BLOCK, device=DEV) ^ k0) + k1) & M32
    j = (torch.arange(BLOCK, device=DEV) * 0x9E3779B9) & M32
    return _mix((block[:, None] + j) & M32)


def _plain_state8(x, floor, rho):
    """8-bit E4M3 codes and block scales of x, rounded up with the probability rho says."""
    amax = x.abs().amax(1, keepdim=True)
    live = amax >= 2.0 ** -100
    scale = torch.where(live, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    y = torch.where(live, x * (torch.full_like(amax, 448.0) / amax), torch.zeros_like(x))
    a = y.abs().clamp(max=448.0)
    if floor:
        a = torch.where(a > 0, a.clamp(min=2.0 ** -9), a)
    e = torch.frexp(a).exponent.sub(1).clamp(min=-6)
    q = torch.ldexp(torch.floor(torch.ldexp(a, 3 - e) + rho), e - 3)
    return torch.copysign(q, y).to(torch.float8_e4m3fn), scale


def _plain_bf16(x, rho):
    """fp32 to BF16, rounded away from zero with the probability rho / 65536 says."""
    b = x.view(torch.int32).to(torch.int64) + rho
    return (b & ~0xFFFF).to(torch.int32).view(torch.float32).to(torch.bfloat16)


def _plain_adamw(s):
    c, t = s["case"], s["step"]
    grad = s["grad"].float().view(-1, BLOCK)
    gs = s["grad_scale"]
    if s["max_norm"] > 0:
        norm = grad.double().square().sum().sqrt().mul(gs)
        s["norm"].copy_(norm.reshape(1))
        gs = gs * (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    grad = grad * gs
    if c["bits"] == 8:
        m = s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).square()
        words = _random_words(s)
    else:
        m, v = s["m"].view(-1, BLOCK), s["v"].view(-1, BLOCK)
        words = None if c["master"] else _random_words(s)
    m = m * s["beta1"] + grad * (1 - s["beta1"])
    v = v * s["beta2"] + grad.square() * (1 - s["beta2"])
    root = v.sqrt()
    bias1, bias2 = 1 - s["beta1"] ** t, 1 - s["beta2"] ** t
    update = m / (root * (1 / math.sqrt(bias2)) + s["eps"])
    p = (s["master"] if c["master"] else s["param"].float()).view(-1, BLOCK)
    p = p * (1 - s["lr"] * s["decay"]) - update * (s["lr"] / bias1)
    if c["master"]:
        s["master"].copy_(p.reshape(-1))
        s["param"].copy_(p.reshape(-1))
    else:
        s["param"].copy_(_plain_bf16(p, ((words * 0x9E3779B9) & M32) >> 16).reshape(-1))
    if c["bits"] == 32:
        s["m"].copy_(m.reshape(-1))
        s["v"].copy_(v.reshape(-1))
    else:
        q, scale = _plain_state8(m, False, (words & 0xFFFF) * 2.0 ** -16)
        s["m"].copy_(q.reshape(-1))
        s["m_scale"].copy_(scale.reshape(-1))
        q, scale = _plain_state8(root, True, (words >> 16) * 2.0 ** -16)
        s["v"].copy_(q.reshape(-1))
        s["v_scale"].copy_(scale.reshape(-1))


def _scores(x, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=torch.finfo(x.dtype).min))
    z = e.sum(1, keepdim=True)
    return torch.where(z > 0, e / z, torch.zeros_like(e))


def _member(s):
    """[sequences, tokens]: which token belongs to which sequence."""
    t = torch.arange(s["case"]["tokens"], device=DEV)
    return (t >= s["offsets"][:-1, None]) & (t < s["offsets"][1:, None])


def _plain_router(s):
    c = s["case"]
    E, K, S = c["experts"], c["topk"], c["seqs"]
    x = s["logits"].float()
    score = _scores(x, c["score"])
    # what decides the selection in 64 bits: two experts may be closer than 32 bits tell apart
    key = x.double() if s["bias"] is None else _scores(x.double(), c["score"]) + s["bias"].double()
    key = torch.where(torch.isneginf(x) | torch.isnan(x), torch.full_like(key, -math.inf), key)
    top = torch.sort(key, dim=1, descending=True, stable=True)
    member = _member(s)
    live = member.any(0)[:, None]
    index = torch.where(live & ~torch.isneginf(top.values[:, :K]), top.indices[:, :K], -1)
    chosen = index.clamp(min=0)
    w = torch.where(index >= 0, score.gather(1, chosen), torch.zeros_like(score[:, :K]))
    if c["normalize"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    picked = torch.zeros_like(score, dtype=torch.float64).scatter_add_(1, chosen, (index >= 0).double())
    member = member.double()
    seq_counts = member @ picked
    p = score if c["score"] == "softmax" else score / (score.sum(1, keepdim=True) + 1e-20)
    n = member.sum(1, keepdim=True).clamp(min=1)
    loss = (seq_counts * (E / K) / n * ((member @ p.double()) / n)).sum() * (s["coef"] / S)
    return {"index": index.to(torch.int32), "weight": w * s["scale"], "counts": seq_counts.sum(0).to(torch.int32),
            "seq_counts": seq_counts.to(torch.int32), "loss": loss.float().reshape(1)}


def _plain_router_grad(s):
    c = s["case"]
    E, K, S = c["experts"], c["topk"], c["seqs"]
    score = _scores(s["logits"].float(), c["score"])
    member = _member(s)
    n = member.sum(1, keepdim=True).clamp(min=1).float()
    # of the balance loss with respect to each token's probabilities
    row = s["dloss"] * (s["coef"] / S) * (E / K) * s["seq_counts"].float() / (n * n)
    balance = member.float().t() @ row
    index = s["index"].long()
    chosen, there = index.clamp(min=0), index >= 0
    picked = torch.where(there, score.gather(1, chosen), torch.zeros_like(s["dweight"]))
    dw = torch.where(there, s["dweight"], torch.zeros_like(s["dweight"])) * s["scale"]
    if c["normalize"]:
        z = picked.sum(1, keepdim=True) + 1e-20
        dw = torch.where(there, (dw - (dw * picked).sum(1, keepdim=True) / z) / z, torch.zeros_like(dw))
    direct = torch.zeros_like(score).scatter_add_(1, chosen, dw)
    if c["score"] == "softmax":
        total = balance + direct
        dx = score * (total - (total * score).sum(1, keepdim=True))
    else:
        z = score.sum(1, keepdim=True) + 1e-20
        through = (balance - (balance * score).sum(1, keepdim=True) / z) / z
        dx = (through + direct) * score * (1 - score)
    return {"dlogits": torch.where(member.any(0)[:, None], dx, torch.zeros_like(dx)).to(s["logits"].dtype)}


def _plain_rows(s):
    c = s["case"]
    E, K, align = c["experts"], c["topk"], c["align"]
    e = s["index"].long().reshape(-1)
    e = torch.where((e >= 0) & (e < E), e, torch.full_like(e, E))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, e, torch.ones_like(e))
    padded = (counts[:E] + align - 1) // align * align
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), padded.cumsum(0)])
    order = torch.sort(e, stable=True)
    rank = torch.arange(e.numel(), device=DEV) - (counts.cumsum(0) - counts)[order.values]
    dropped = order.values == E
    row = torch.where(dropped, torch.full_like(rank, s["n_rows"]), offsets[order.values.clamp(max=E)] + rank)
    row_token = torch.full((s["n_rows"] + 1,), -1, dtype=torch.int32, device=DEV)
    row_token[row] = torch.where(dropped, -1, order.indices // K).to(torch.int32)
    pair_row = torch.empty_like(e, dtype=torch.int32)
    pair_row[order.indices] = torch.where(dropped, -1, row).to(torch.int32)
    return {"row_token": row_token[:-1], "pair_row": pair_row.view(-1, K), "offsets": offsets.to(torch.int32),
            "counts": counts[:E].to(torch.int32)}


# --------------------------------------------------------------------- work
def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        per = (2 if case["grad"] == "bf16" else 4) + (8 + 2 if case["master"] else 4) + \
            (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        return {"bytes": per * n, "flops": 20 * n}
    T, K, E = case["tokens"], case["topk"], case["experts"]
    if case["op"] == "rows":
        return {"bytes": 8 * T * K + 4 * _rows_capacity(case) + 8 * E + 4, "flops": T * K}
    S, size = case["seqs"], 2 if case["logits"] == "bf16" else 4
    if case["op"] == "router":
        return {"bytes": T * E * size + 8 * T * K + 4 * E * (S + 1 + case["bias"]) + 4 * S + 8, "flops": 8 * T * E}
    return {"bytes": 2 * T * E * size + 8 * T * K + 4 * E * S + 4 * S + 8, "flops": 12 * T * E}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits, tensor by tensor and sequence by sequence."""
    if case["op"] == "rows":
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_router(s)


def _exact_word(step_keys, block, n):
    """The random word of each of a tensor's n elements, its first block being number `block`."""
    def scramble(w):
        for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
            w = ((w ^ (w >> shift)) * factor) % (1 << 32)
        return w ^ (w >> 16)

    i = torch.arange(n, dtype=torch.int64, device=DEV)
    return scramble((scramble((block + i // BLOCK) ^ step_keys[0]) + step_keys[1] + (i % BLOCK) * 0x9E3779B9) % (1 << 32))


def _exact_codes(x, rho, never_zero):
    """(values of the codes, scales) of one tensor's state."""
    n = x.numel()
    rows = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64, device=DEV)
    rows[:n] = x
    top = rows.view(-1, BLOCK).abs().max(dim=1).values
    scale = torch.where(top < 2.0 ** -100, torch.ones_like(top), top / 448)
    y = x / scale.repeat_interleave(BLOCK)[:n]
    a = y.abs()
    if never_zero:
        a = torch.where(x > 0, torch.maximum(a, torch.full_like(a, 2.0 ** -9)), a)
    unit = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * unit * torch.floor(a / unit + rho), scale


def _exact_adamw(s):
    c, t = s["case"], s["step"] + 1
    keys = _keys(s["seed"], t)
    out = {k: [] for k in ("param", "m", "v", "master", "m_scale", "v_scale")}
    spans, at = [], 0
    for n, b in zip(s["sizes"], s["blocks"]):
        spans.append((at, n, b * BLOCK - n))
        at += b * BLOCK
    factor, norm = s["grad_scale"], None
    if s["max_norm"] > 0:
        norm = s["grad_scale"] * math.sqrt(sum(float((s["grad"][a:a + n].double() ** 2).sum()) for a, n, _ in spans))
        factor *= min(1.0, s["max_norm"] / (norm + 1e-6))
    for k, (a, n, pad) in enumerate(spans):
        def part(name):
            return s[name][a:a + n].double()

        g = part("grad") * factor
        m, v, words = part("m"), part("v"), None
        if c["bits"] == 8:
            at_block = slice(a // BLOCK, (a + n + pad) // BLOCK)
            m = m * s["m_scale"][at_block].double().repeat_interleave(BLOCK)[:n]
            v = (v * s["v_scale"][at_block].double().repeat_interleave(BLOCK)[:n]) ** 2
        if c["bits"] == 8 or not c["master"]:
            words = _exact_word(keys, a // BLOCK, n)
        m = s["beta1"] * m + (1 - s["beta1"]) * g
        v = s["beta2"] * v + (1 - s["beta2"]) * g * g
        hat = (m / (1 - s["beta1"] ** t)) / (torch.sqrt(v / (1 - s["beta2"] ** t)) + s["eps"])
        p = part("master" if c["master"] else "param")
        p = p - s["lr"] * (s["decays"][k] * p + hat)
        zeros = torch.zeros(pad, dtype=torch.float64, device=DEV)
        if c["master"]:
            out["master"] += [p, zeros]
            out["param"] += [p.to(torch.bfloat16).double(), zeros]
        else:
            rho = ((words * 0x9E3779B9) % (1 << 32) >> 16).double() / 65536
            unit = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
            out["param"] += [torch.sign(p) * unit * torch.floor(p.abs() / unit + rho), zeros]
        if c["bits"] == 32:
            out["m"] += [m, zeros]
            out["v"] += [v, zeros]
        else:
            for name, x, rho in (("m", m, words % 65536), ("v", torch.sqrt(v), words >> 16)):
                q, scale = _exact_codes(x, rho.double() / 65536, name == "v")
                out[name] += [q, zeros]
                out[name + "_scale"].append(scale)
    got = {k: torch.cat(v) for k, v in out.items() if v}
    if norm is not None:
        got["norm"] = torch.tensor([norm], dtype=torch.float64)
    return got


def _exact_router(s):
    c = s["case"]
    T, E, K, S = c["tokens"], c["experts"], c["topk"], c["seqs"]
    x = s["logits"].double()
    if c["score"] == "sigmoid":
        score = torch.sigmoid(x)
        prob = score / score.sum(1, keepdim=True)
    else:
        score = prob = torch.softmax(x, dim=1)
    bounds = s["offsets"].tolist()
    if c["op"] == "router_grad":
        grad = torch.zeros(T, E, dtype=torch.float64, device=DEV)
        there = s["index"] >= 0
        for q in range(S):
            a, b = bounds[q], bounds[q + 1]
            if a == b:
                continue
            at, ok = s["index"][a:b].long().clamp(min=0), there[a:b].double()
            sel = score[a:b].gather(1, at) * ok
            up = s["dweight"][a:b].double() * ok * s["scale"]
            if c["normalize"]:
                mass = sel.sum(1, keepdim=True)
                up = ok * (up * mass - (up * sel).sum(1, keepdim=True)) / mass ** 2
            dscore = torch.zeros(b - a, E, dtype=torch.float64, device=DEV).scatter_add_(1, at, up)
            f = E / (K * (b - a)) * s["seq_counts"][q].double()
            dprob = float(s["dloss"]) * s["coef"] / S * f / (b - a)
            centred = dprob - (prob[a:b] * dprob).sum(1, keepdim=True)
            if c["score"] == "softmax":
                grad[a:b] = score[a:b] * (centred + dscore - (score[a:b] * dscore).sum(1, keepdim=True))
            else:
                grad[a:b] = (centred / score[a:b].sum(1, keepdim=True) + dscore) * score[a:b] * (1 - score[a:b])
        return {"dlogits": grad}
    key = x if s["bias"] is None else score + s["bias"].double()
    key = key.masked_fill(x == -math.inf, -math.inf)
    at = torch.argsort(-key, dim=1, stable=True)[:, :K]
    ok = key.gather(1, at) > -math.inf
    ok[: bounds[0]] = False
    ok[bounds[-1]:] = False
    w = score.gather(1, at) * ok
    if c["normalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    loss = 0.0
    for q in range(S):
        a, b = bounds[q], bounds[q + 1]
        if b > a:
            f = torch.bincount(at[a:b][ok[a:b]], minlength=E).double() * E / (K * (b - a))
            loss += float((f * prob[a:b].mean(0)).sum())
    return {"index": None, "weight": w * s["scale"], "counts": None, "seq_counts": None,
            "loss": torch.tensor([s["coef"] * loss / S], dtype=torch.float64)}
