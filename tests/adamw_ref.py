"""The AdamW step's definition in 64 bits (numpy), for one tensor, with bounds
on how far a computation in fp32 may be from it. Shares no code with the
library. eps32 is half a step of fp32 relative to the value."""
import numpy as np

EPS32 = 2.0 ** -24
U32 = np.uint64(0xFFFFFFFF)


def keys(seed, step):
    m = (1 << 64) - 1
    z = (seed + step * 0x9E3779B97F4A7C15) & m
    z ^= z >> 32
    z = z * 0x6A09E667F3BCC909 & m
    z ^= z >> 29
    z = z * 0xBB67AE8584CAA73B & m
    z ^= z >> 32
    return z & 0xFFFFFFFF, z >> 32


def _mix(x):
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x6A09E667)) & U32
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xBB67AE85)) & U32
    return x ^ (x >> np.uint64(16))


def words(seed, step, block0, n, first=0):
    """Random words of elements first .. first + n of a tensor."""
    k0, k1 = keys(seed, step)
    i = np.arange(first, first + n, dtype=np.uint64)
    b = (np.uint64(block0) + i // np.uint64(128)) & U32
    return _mix((_mix(b ^ np.uint64(k0)) + np.uint64(k1) + (i % np.uint64(128)) * np.uint64(0x9E3779B9)) & U32)


E4M3 = np.array([np.nan if (b & 0x7F) == 0x7F else (-1.0 if b & 0x80 else 1.0) *
                 ((b & 7) * 2.0 ** -9 if not b & 0x78 else (1 + (b & 7) / 8) * 2.0 ** (((b >> 3) & 15) - 7))
                 for b in range(256)])


def e4m3_up(a, rho):
    """floor(a + rho in units of the format), a >= 0."""
    unit = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return unit * np.floor(a / unit + rho)


def bf16_up(a, rho):
    unit = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -126))) - 7)
    return unit * np.floor(a / unit + rho)


def bf16_value(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def step(p, g, m, v, *, lr, beta1, beta2, eps, wd, gs, t):
    """(p', m', v' and the bounds of each in fp32) from 64-bit inputs; m, v as
    the state stands for (v the second moment)."""
    g = g * gs
    mn = beta1 * m + (1 - beta1) * g
    vn = beta2 * v + (1 - beta2) * g * g
    # g is scaled and rounded once (gs itself is rounded to fp32), the factors are rounded, each product and sum once
    em = 4 * EPS32 * (np.abs(beta1 * m) + np.abs((1 - beta1) * g)) + 2.0 ** -148
    ev = 8 * EPS32 * vn + 2.0 ** -125
    d = np.sqrt(vn / (1 - beta2 ** t)) + eps
    u = mn / (1 - beta1 ** t) / d
    # the root halves a relative error; quotient, factors and sums add a few roundings
    eroot = np.minimum(np.sqrt(ev), ev / np.maximum(np.sqrt(vn), 1e-300)) + 2 * EPS32 * np.sqrt(vn)
    ed = eroot / np.sqrt(1 - beta2 ** t) + 4 * EPS32 * d
    with np.errstate(all="ignore"):
        eu = em / (1 - beta1 ** t) / np.maximum(d - ed, 1e-300) + np.abs(u) * (ed / np.maximum(d - ed, 1e-300) + 4 * EPS32)
    pn = p - lr * (wd * p + u)
    ep = 4 * EPS32 * (np.abs(p) + np.abs(pn)) + lr * eu + 4 * EPS32 * lr * np.abs(u) + 2.0 ** -148
    return pn, mn, vn, ep, em, ev, eroot


def blocks(n):
    return -(-n // 128)


def per_block(x, n):
    return np.repeat(x, 128)[:n]


def block_amax(x):
    """amax over the finite values of each 128-element block."""
    n = x.size
    pad = np.zeros(blocks(n) * 128)
    pad[:n] = np.where(np.isfinite(x), np.abs(x), 0.0)
    return pad.reshape(-1, 128).max(1)


def check_codes(codes, scale, x, ex, rho, root, what):
    """codes (uint8) and scales of a state whose exact value is x +- ex."""
    n = x.size
    amax, eamax = block_amax(x), block_amax(ex)
    live = amax >= 2.0 ** -100 * 1.001
    dead = amax < 2.0 ** -100 * 0.999
    want = np.where(live, amax / 448, 1.0)
    tol = (eamax / 448 + 4 * EPS32 * want)
    assert np.all(np.abs(scale - want)[live] <= tol[live]), what + ": scale"
    assert np.all(scale[dead] == 1.0), what + ": scale of an empty block"
    got = E4M3[codes]
    fine = np.isfinite(x)
    assert np.array_equal(np.isnan(got), ~fine), what + ": NaN codes"
    s = per_block(want, n)
    rel = per_block(np.where(live, tol / np.where(live, want, 1), 0.0), n)
    with np.errstate(all="ignore"):
        y = np.abs(x) / s
        ey = ex / s + y * (rel + 4 * EPS32)
    y, ey = np.where(fine, y, 0), np.where(fine, ey, 0)
    lo, hi = np.clip(y - ey, 0, 448), np.clip(y + ey, 0, 448)
    if root:
        lo, hi = np.where(x > 0, np.maximum(lo, 2.0 ** -9), lo), np.where(x > 0, np.maximum(hi, 2.0 ** -9), hi)
    in_dead = per_block(dead, n)
    lo, hi = np.where(in_dead, 0, lo), np.where(in_dead, 0, hi)
    lo, hi = e4m3_up(np.where(fine, lo, 0), rho), np.minimum(e4m3_up(np.where(fine, hi, 0), rho), 448)
    a = np.abs(got)
    bad = fine & ~((a >= lo) & (a <= hi))
    assert not bad.any(), f"{what}: {bad.sum()} codes off, first at {np.argmax(bad)}: got {a[bad][0]}, want " \
                          f"[{lo[bad][0]}, {hi[bad][0]}]"
    sign = fine & (a > 0) & (np.abs(x) > ex)
    assert np.array_equal(np.sign(got[sign]), np.sign(x[sign])), what + ": sign"
    # the two bounds are nearly always the same code: the check is on the exact value
    assert np.mean(lo == hi) > 0.99 or n < 2000 or dead.any(), what + ": bounds too wide to say anything"
