"""Definitions of the experts' products, the gated block and MXFP4 in 64 bits,
with the bounds that the kernels' arithmetic allows, for small sizes on the CPU.
Nothing here calls the library."""
import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
NT, NN, TN = range(3)
SILU, GELU = range(2)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def act(kind, x):
    if kind == SILU:
        return x * torch.sigmoid(x)
    return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))


def slope(kind, x):
    if kind == SILU:
        s = torch.sigmoid(x)
        return s * (1 + x * (1 - s))
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (x + 0.044715 * x ** 3))
    return s + x * s * (1 - s) * c * (1 + 3 * 0.044715 * x ** 2)


# Sums of n products of two BF16 (or E2M1) values: the products are exact in fp32, each of the n additions is off by at
# most 2^-23 of a partial sum (twice a rounding: a matrix instruction may cut), and no partial sum exceeds the sum of
# magnitudes.
def sum_bound(n, magnitudes):
    return n * 2.0 ** -23 * magnitudes


# Relative error of the activations: exp2's argument is off by 4 roundings of 2^-24 of at most |y| log2(e), so the
# exponential by 4 * 2^-24 |y| (ln 2 and log2(e) cancel) and a last place; the reciprocal, the sum and two products add a last place each. |y| stays
# below 60 in these tests (inputs below 10 in magnitude; y of GELU grows with the cube).
ACT = (4 * 60 + 8) * 2.0 ** -24


class Layout:
    """Rows of each expert: counts, first rows at multiples of `align` from `lead` on, `tail` rows behind the last."""

    def __init__(self, counts, align=1, lead=0, tail=0):
        self.counts, first, at = list(counts), [], lead
        for c in counts:
            first.append(at)
            at += -(-c // align) * align
        self.first, self.n_rows = first, at + tail
        self.offsets = torch.tensor(first + [at], dtype=torch.int32)
        self.counts_t = torch.tensor(self.counts, dtype=torch.int32)

    def spans(self):
        return [(e, f, f + c) for e, (f, c) in enumerate(zip(self.first, self.counts))]

    def owned(self):
        m = torch.zeros(self.n_rows, dtype=torch.bool)
        for _, a, b in self.spans():
            m[a:b] = True
        return m


def gather(x, index):
    if index is None:
        return x
    i = index.long()
    ok = (i >= 0) & (i < x.shape[0])
    if x.shape[0] == 0:
        return torch.zeros(len(i), x.shape[1], dtype=x.dtype)
    return torch.where(ok[:, None], x[i.clamp(0, x.shape[0] - 1)], torch.zeros((), dtype=x.dtype))


def product(form, lay, a, b, index=None):
    """(result, sum of magnitudes, terms) in 64 bits; rows of no expert are NaN in the result."""
    a, b = a.double(), b.double()
    if form == TN:
        b = gather(b, index)
        out = torch.stack([a[s:t].t() @ b[s:t] for _, s, t in lay.spans()])
        mag = torch.stack([a[s:t].abs().t() @ b[s:t].abs() for _, s, t in lay.spans()])
        return out, mag, torch.tensor(lay.counts, dtype=torch.float64)[:, None, None]
    a = gather(a, index)
    n = b.shape[1] if form == NT else b.shape[2]
    out = torch.full((lay.n_rows, n), math.nan, dtype=torch.float64)
    mag = torch.zeros(lay.n_rows, n, dtype=torch.float64)
    for e, s, t in lay.spans():
        w = b[e].t() if form == NT else b[e]
        out[s:t], mag[s:t] = a[s:t] @ w, a[s:t].abs() @ w.abs()
    return out, mag, a.shape[1]


def bound(out, mag, terms, dtype):
    return sum_bound(terms, mag) + half_step(dtype) * (out.abs() + sum_bound(terms, mag))


def gated(lay, x, w, kind, index=None):
    """{name: (result, bound)} of h and pre."""
    y, mag, k = product(NT, lay, x, w, index)
    n = y.shape[1] // 2
    off = sum_bound(k, mag)
    g, u, dg, du = y[:, :n], y[:, n:], off[:, :n], off[:, n:]
    h = act(kind, g) * u
    # both activations have slopes below 1.2 in magnitude
    err = 1.2 * dg * (u.abs() + du) + act(kind, g).abs() * du + ACT * h.abs()
    hs = half_step(torch.bfloat16)
    return {"h": (h, err + hs * (h.abs() + err) + 2.0 ** -133), "pre": (y, off + hs * (y.abs() + off))}


def gated_back(lay, dy, down, pre, kind):
    """(dpre, bound): [rows, 2n]."""
    dh, mag, k = product(NN, lay, dy, down)
    n = dh.shape[1]
    g, u, off = pre[:, :n].double(), pre[:, n:].double(), sum_bound(k, mag)
    out = torch.cat([dh * u * slope(kind, g), dh * act(kind, g)], 1)
    # slope = s + x s (1 - s) y': each factor within ACT of itself except 1 - s, which is off by 2^-23 absolutely; x y' s stays
    # below 60 where it counts
    sl = 2 * ACT * (1 + slope(kind, g).abs()) + 60 * 2.0 ** -23
    err = torch.cat([off * u.abs() * 1.2 + (dh.abs() + off) * u.abs() * sl,
                     off * act(kind, g).abs() + ACT * (dh.abs() + off) * act(kind, g).abs()], 1)
    return out, err + half_step(torch.bfloat16) * (out.abs() + err) + 2.0 ** -133


# --------------------------------------------------------------------- MXFP4
def mx_round(x):
    """(codes, one to an element and padded to whole blocks; scale bytes) of rows, value by value from the definition."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    y = torch.zeros(rows, nb * 32, dtype=torch.float64)
    y[:, :cols] = x.double()
    neg = torch.zeros(rows, nb * 32, dtype=torch.bool)
    neg[:, :cols] = torch.signbit(x)
    y, neg = y.view(rows, nb, 32), neg.view(rows, nb, 32)
    amax = y.abs().amax(2)
    bad = ~torch.isfinite(amax)
    safe = torch.where(bad | (amax == 0), torch.ones_like(amax), amax)
    c = (torch.frexp(safe).exponent - 1 - 2).clamp(-127, 125) + 127
    c = torch.where(amax == 0, 127, torch.where(bad, 255, c))
    z = y.abs() * torch.exp2(127.0 - c.double())[:, :, None]
    grid = torch.tensor(E2M1, dtype=torch.float64)
    dist = (z.clamp(max=6.0)[..., None] - grid).abs()
    best = dist.amin(-1, keepdim=True)
    near = dist == best
    # of two equally near codes the even one
    odd = torch.arange(8) % 2 == 1
    code = torch.where(near, torch.where(odd, 1, 0), 2).argmin(-1)
    code = torch.where(bad[:, :, None], 0, code + 8 * neg.int())
    return code.view(rows, -1).to(torch.uint8), c.to(torch.uint8)


def mx_pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def mx_values(packed, scales):
    """Values in 64 bits of packed codes [rows, 16 nb] and scale bytes [rows, nb]."""
    code = torch.stack([packed & 15, packed >> 4], 2).flatten(1)
    v = torch.tensor(E2M1, dtype=torch.float64)[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0)
    size = torch.where(scales == 255, torch.tensor(math.nan, dtype=torch.float64), torch.exp2(scales.double() - 127))
    return v * size.repeat_interleave(32, dim=1)
