"""Plain definitions in 64 bits of the layer norm, the low-rank adapters and their gradients, the AdamW
step in the single fp32 operations that define it, and the error bounds that the kernels' arithmetic
keeps (U = 2^-24, half a step of fp32; the last rounding is _block.check's)."""
import numpy as np
import torch

from _block import U, f64

# Additions that one term of a row's sum goes through: at most 128 in a lane, 6 exchanges between
# lanes, 16 waves.
SUM = 150


def norm_rows(M, groups):
    """Group of each row, -1 outside all."""
    if groups is None:
        return np.zeros(M, int)
    g = np.searchsorted(groups, np.arange(M), side="right") - 1
    return np.where((g < 0) | (g >= len(groups) - 1), -1, g)


def norm_forward(x, w, b, scale, shift, group, eps):
    """y, stats and their bounds; rows of no group are meaningless."""
    mean = x.mean(1, keepdims=True)
    d = x - mean
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    n = d * r
    # the distances are taken from a mean that is SUM U off, and from their own mean, whose sum is as exact
    far = SUM * U * np.abs(x).mean(1, keepdims=True)
    e = (SUM + 4) * U * (np.abs(d).mean(1, keepdims=True) + far)
    br = (SUM / 2 + 6) * U + 2 * (SUM * U) * far * r  # relative: half the squares' error, root and reciprocal
    bn = (np.abs(d) * 2 * U + far * 2 * U + e) * r + np.abs(n) * (br + 2 * U)
    s = 1 + scale[group] if scale is not None else np.ones_like(x)
    h = shift[group] if shift is not None else np.zeros_like(x)
    v = n * w + b
    y = v * s + h
    by = (bn * np.abs(w) + 2 * U * (np.abs(n * w) + np.abs(b))) * np.abs(s) + 2 * U * (np.abs(v * s) + np.abs(h))
    return y, np.concatenate([mean, r], 1), 1.01 * by, np.concatenate([U * np.abs(mean) + e, br * r], 1)


def norm_backward(x, stats, w, b, scale, group, G, dy):
    """dx, the sums dw, db, dscale, dshift, and the bounds of all; rows of no group count in no sum."""
    D = x.shape[1]
    r = stats[:, 1:]
    n = (x - stats[:, :1]) * r
    s = 1 + scale[group] if scale is not None else np.ones_like(x)
    t = dy * s * w
    c0, c1 = t.mean(1, keepdims=True), (t * n).mean(1, keepdims=True)
    dx = r * (t - c0 - n * c1)
    a0, a1 = np.abs(t).mean(1, keepdims=True), np.abs(t * n).mean(1, keepdims=True)
    bx = r * U * (10 * np.abs(t) + (SUM + 8) * a0 + (SUM + 14) * np.abs(n) * a1)
    live = (group >= 0)[:, None]
    # 32 rows in fp32, then double; n holds two roundings; the sums round once where they leave
    S0, S1 = np.zeros((G, D)), np.zeros((G, D))
    A0, A1 = np.zeros((G, D)), np.zeros((G, D))
    for g in range(G):
        m = group == g
        S0[g], S1[g] = dy[m].sum(0), (dy[m] * n[m]).sum(0)
        A0[g], A1[g] = 32 * U * np.abs(dy[m]).sum(0), 36 * U * np.abs(dy[m] * n[m]).sum(0)
    k = 1 + scale if scale is not None else np.ones((G, D))
    sums = dict(dweight=(k * S1).sum(0), dbias=(k * S0).sum(0), dscale=w * S1 + b * S0, dshift=S0)
    bounds = dict(dweight=(np.abs(k) * A1).sum(0), dbias=(np.abs(k) * A0).sum(0), dscale=np.abs(w) * A1 + np.abs(b) * A0, dshift=A0)
    return np.where(live, dx, 0), sums, np.where(live, bx, 0), bounds


# T enters the second product in two bf16 parts, the second rounded by half of its 2^-8 steps where the
# first leaves up to 2^-7: 2^-16.  The gradients' sums take three, which hold all of fp32's digits.
PARTS = 2.0 ** -16


def adapters_forward(x, la, lb, alpha, ids, y0):
    """y, t and their bounds.  A product of K terms adds K exact products in fp32, two roundings' worth
    each, and up to 64 sums of splits: 2 (K + 64) U of the sum of magnitudes."""
    M, K, R = x.shape[0], x.shape[1], lb.shape[1]
    t, bt, y = np.zeros((M, R)), np.zeros((M, R)), y0.copy()
    by = np.zeros_like(y)
    for a in range(len(la)):
        m = ids == a
        t[m] = x[m] @ lb[a].T
        bt[m] = 2 * (K + 64) * U * (np.abs(x[m]) @ np.abs(lb[a]).T)
        s = abs(alpha[a])
        y[m] += alpha[a] * (t[m] @ la[a].T)
        by[m] = s * ((bt[m] + (PARTS + 2 * U + 4 * (R + 32) * U) * (np.abs(t[m]) + bt[m])) @ np.abs(la[a]).T)
    return y, t, by + U * (np.abs(y) + by), bt


def adapters_backward(x, la, lb, alpha, ids, t, dy, dx0):
    """(dx, dla, dlb) and their bounds."""
    N, R = dy.shape[1], lb.shape[1]
    dx, bx = dx0.copy(), np.zeros_like(dx0)
    dla, dlb, ba, bb = (np.zeros_like(v) for v in (la, lb, la, lb))
    for a in range(len(la)):
        m, s = ids == a, alpha[a]
        n = int(m.sum()) + 320  # rows, filled up in each share
        dt = s * (dy[m] @ la[a])
        bt = 2 * (N + 66) * U * abs(s) * (np.abs(dy[m]) @ np.abs(la[a]))
        dx[m] += dt @ lb[a]
        bx[m] = (bt + (PARTS + 4 * (R + 32) * U) * (np.abs(dt) + bt)) @ np.abs(lb[a])
        dlb[a], dla[a] = dt.T @ x[m], s * (dy[m].T @ t[m])
        off = 6 * n * U
        bb[a] = (bt + off * (np.abs(dt) + bt)).T @ np.abs(x[m])
        ba[a] = off * abs(s) * (np.abs(dy[m]).T @ np.abs(t[m]))
    return (dx, dla, dlb), (bx + U * (np.abs(dx) + bx), ba, bb)


# ---------------------------------------------------------------- AdamW

F = np.float32
BLOCK = 256


def e4m3_values():
    """The 127 values from 0 to 448 in the order of their codes."""
    c = np.arange(127)
    e, f = c >> 3, c & 7
    return np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))


def to_e4m3(x):
    """The nearest E4M3 value of fp32 values up to 448, ties to the even code."""
    v = e4m3_values()
    a = np.abs(x).astype(np.float64)
    hi = np.clip(np.searchsorted(v, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = (v[hi] - a < a - v[lo]) | ((v[hi] - a == a - v[lo]) & (hi % 2 == 0))
    return np.copysign(np.where(up, v[hi], v[lo]), x).astype(F)


def blocks(x):
    return np.pad(x, (0, -len(x) % BLOCK)).reshape(-1, BLOCK)


def encode(x, root):
    """E4M3 values and scales of x [n] fp32."""
    b = blocks(x)
    most = np.abs(b).max(1, keepdims=True)
    with np.errstate(divide="ignore", over="ignore"):
        inverse = F(448) / most
    inverse = np.where(np.isfinite(inverse), inverse, F(0))
    s = b * inverse
    if root:
        s = np.where(b > 0, np.maximum(s, F(2.0 ** -9)), s)
    return to_e4m3(s).reshape(-1)[:len(x)], (most / F(448)).reshape(-1)


def decode(codes, scales):
    return codes * np.repeat(scales, BLOCK)[:len(codes)]


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, clip=None, scales=None):
    """p, m, v (with `scales`, of m and of the root: the codes' values and scales) after a step, each line
    one fp32 operation."""
    c1, b2, c2 = F(1 - beta1), F(beta2), F(1 - beta2)
    m_up, u_up = F(1 / (1 - beta1 ** step)), F(1 / np.sqrt(1 - beta2 ** step))
    g = g if clip is None else g * F(clip)
    if scales is not None:
        m = decode(m, scales[0])
        u = decode(v, scales[1])
        v = u * u
    d = g - m
    m = m + d * c1
    keep, add = v * b2, g * g
    add = add * c2
    v = keep + add
    u = np.sqrt(v)
    den = u * u_up
    den = den + F(eps)
    s = m * m_up
    s = s / den
    t = p * F(decay)
    t = s + t
    p = p - t * F(lr)
    if scales is None:
        return p, m, v
    return p, encode(m, False), encode(u, True)


def rnd(seed, *shape, std=1.0, dtype=torch.bfloat16, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).cuda()


__all__ = [n for n in dir() if not n.startswith("__")] + ["f64"]
