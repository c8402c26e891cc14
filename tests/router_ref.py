"""The expert router and the dispatch's row map in 64 bits and whole numbers
(numpy, token by token). Shares no code with the library."""
import numpy as np


def score64(x, kind):
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = np.max(np.where(np.isnan(x), -np.inf, x))
        e = np.exp(x - (top if top > -np.inf else 0.0))
        z = e.sum()
        return e / z if z != 0 else e


def forward(x, *, kind, top_k, normalize, scale, bias, offsets, coef):
    """x: [T, E] float64. Returns index, weight, seq_counts, loss and the scores."""
    T, E = x.shape
    S = len(offsets) - 1
    index = np.full((T, top_k), -1, dtype=np.int32)
    weight = np.zeros((T, top_k))
    seq_counts = np.zeros((S, E), dtype=np.int64)
    loss = 0.0
    for q in range(S):
        a, b = offsets[q], offsets[q + 1]
        p_sum = np.zeros(E)
        for t in range(a, b):
            s = score64(x[t], kind)
            key = x[t] if bias is None else s + bias
            order = [e for e in np.argsort(-np.where(np.isnan(key), -np.inf, key), kind="stable")
                     if x[t, e] > -np.inf and key[e] > -np.inf][:top_k]
            index[t, :len(order)] = order
            w = s[order]
            weight[t, :len(order)] = scale * (w / (w.sum() + 1e-20) if normalize else w)
            seq_counts[q, order] += 1
            p_sum += s if kind == "softmax" else s / (s.sum() + 1e-20)
        if b > a:
            loss += float((E * seq_counts[q] / (top_k * (b - a)) * p_sum / (b - a)).sum())
    return index, weight, seq_counts, coef / S * loss


def value(x, index, seq_counts, dweight, dloss, *, kind, top_k, normalize, scale, offsets, coef):
    """<dweight, weight> + dloss * loss for fixed selections, a function of the
    logits whose gradient is what the backward pass returns. x: torch float64."""
    import torch

    E = x.shape[1]
    S = len(offsets) - 1
    total = x.new_zeros(())
    # a token whose experts are all switched off has no scores
    none = (x == -float("inf")).all(1, keepdim=True)
    y = torch.where(none, torch.zeros_like(x), x)
    s = (torch.sigmoid(y) if kind == "sigmoid" else torch.softmax(y, dim=1)) * ~none
    p = s / (s.sum(1, keepdim=True) + 1e-20) if kind == "sigmoid" else s
    for q in range(S):
        a, b = offsets[q], offsets[q + 1]
        if a == b:
            continue
        if dweight is not None:
            ok = (index[a:b] >= 0) & (index[a:b] < E)
            w = s[a:b].gather(1, index[a:b].clamp(0, E - 1).long()) * ok
            if normalize:
                w = w / (w.sum(1, keepdim=True) + 1e-20)
            total = total + (dweight[a:b] * w * ok).sum() * scale
        if dloss is not None:
            f = E * seq_counts[q].double() / (top_k * (b - a))
            total = total + dloss * coef / S * (f * p[a:b].mean(0)).sum()
    return total


def rows(index, n_experts, align, n_rows):
    T, K = index.shape
    copies = [[] for _ in range(n_experts)]
    for t in range(T):
        for k in range(K):
            if 0 <= index[t, k] < n_experts:
                copies[index[t, k]].append((t, k))
    offsets = np.zeros(n_experts + 1, dtype=np.int64)
    for e in range(n_experts):
        offsets[e + 1] = offsets[e] + -(-len(copies[e]) // align) * align
    row_token = np.full(n_rows, -1, dtype=np.int32)
    pair_row = np.full((T, K), -1, dtype=np.int32)
    for e in range(n_experts):
        for i, (t, k) in enumerate(copies[e]):
            r = offsets[e] + i
            if r < n_rows:
                row_token[r] = t
                pair_row[t, k] = r
    return row_token, pair_row, offsets, np.array([len(c) for c in copies])
