"""Plain definitions in 64 bits of the rotary positions, the head norms and the gated block,
and the error bounds that the kernels' arithmetic keeps (u = 2^-24, half a step of fp32; the
last rounding costs half a step of the output's type)."""
import numpy as np
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def angles(pos, dims, theta):
    """[M, pairs] in radians."""
    parts = [pos[:, a:a + 1] * theta ** (-2.0 * np.arange(d // 2) / d) for a, d in enumerate(dims)]
    return np.concatenate(parts, axis=1)


def pair_index(n, pairs):
    """Channels of each pair's first and second value."""
    p = np.arange(n)
    return (2 * p, 2 * p + 1) if pairs == 0 else (p, p + n)


def rotate(x, phi, pairs, sign=1.0):
    a, b = pair_index(phi.shape[1], pairs)
    c, s = np.cos(phi)[:, None], sign * np.sin(phi)[:, None]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def pair_sum(x, n, pairs):
    """|x0| + |x1| of each channel's pair; |x| of a channel that is not turned."""
    a, b = pair_index(n, pairs)
    y = np.abs(x)
    y[..., a], y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b]), np.abs(x[..., a]) + np.abs(x[..., b])
    return y


# A turned value x0 c - x1 s: the reduced angle is within 2^-25 revolutions (two roundings of at
# most 2^-26: 3.2 u radians), cos and sin within 2.2 u of it, each product and the difference
# rounds once: 8 u of |x0| + |x1|.
TURN = 8 * U

# A normed value x r w: 8 squares per lane and up to 5 exchanges sum within 14 u, the mean, eps,
# root and reciprocal add 5 u (half of the sum's error and theirs enter r: 12 u), two products
# 2 u: 14 u of it, then the turn on values that far off.
NORM = 14 * U


def qk_forward(x, w, phi, pairs, eps):
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r * w
    return rotate(n, phi, pairs), (NORM + TURN) * pair_sum(n, phi.shape[1], pairs)


def qk_backward(x, w, phi, pairs, eps, dy):
    """dx, dw and their bounds.  Each of dx's two terms carries the turn (8 u), r (12 u), the sum
    of w t x (14 u and 3 products) and under ten roundings more: 64 u of their magnitudes.  dw
    adds terms within 24 u, at most 16 per group and item chunk and 64 groups in fp32, then in
    double: 128 u of the sum of magnitudes."""
    D, n = x.shape[-1], phi.shape[1]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    t, ta = rotate(dy, phi, pairs, -1.0), pair_sum(dy, n, pairs)
    wt, wta = t * w, ta * np.abs(w)
    dx = r * wt - x * r ** 3 * (wt * x).mean(-1, keepdims=True)
    bx = 64 * U * (r * wta + np.abs(x) * r ** 3 * (wta * np.abs(x)).mean(-1, keepdims=True))
    return dx, (t * x * r).sum((0, 1)), bx, 128 * U * (ta * np.abs(x) * r).sum((0, 1))


def erf(x):
    return torch.erf(torch.from_numpy(x)).numpy()


def act(g, kind):
    """value and slope; kind 0 SiLU, 1 GELU."""
    if kind == 0:
        with np.errstate(over="ignore"):  # exp(-g) = inf leaves p = 0
            p = 1 / (1 + np.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    p = 0.5 * (1 + erf(g / np.sqrt(2)))
    return g * p, p + g * np.exp(-g * g / 2) / np.sqrt(2 * np.pi)


def act_bound(g):
    """Error of the kernels' act(g) and act'(g): exp of an argument rounded to fp32 is within
    (2 |g| + 4) u, the rest a few roundings; GELU's Phi is within 5 u in absolute terms
    (Abramowitz and Stegun 7.1.26 halved, 1.3 u, and its roundings), times |g|; the slope's
    g exp(-g^2 / 2) is below 1."""
    return (8 + 4 * np.abs(g)) * U * (1 + np.abs(g))


def glu_forward(x, wg, wu, kind, dtype=torch.bfloat16):
    """y, g, u and the bounds before the last rounding.  A product of K terms adds K exact
    products in fp32, two roundings' worth each: 2 K u of the sum of magnitudes."""
    K = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    bg, bu = 2 * K * U * (np.abs(x) @ np.abs(wg).T), 2 * K * U * (np.abs(x) @ np.abs(wu).T)
    v, _ = act(g, kind)
    by = (1.13 * bg + act_bound(g)) * (np.abs(u) + bu) + np.abs(v) * bu + 2 * U * np.abs(v * u)
    return v * u, g, u, by, bg, bu


def glu_backward(x, wg, wu, g, u, dy, kind, elements=None):
    """dx, dwg, dwu and their bounds (`elements`: of G in the call, where g holds some of its
    rows): dG and dU round once to bf16 (2^-8 of each; up to 2^14
    elements twice, 2^-16) after an activation within act_bound; the products add as in
    glu_forward, twice as many where they run over both roundings."""
    v, s = act(g, kind)
    dg, du = dy * u * s, dy * v
    b = act_bound(g)
    few = (elements or g.size) <= 2 ** 14
    step = 2.0 ** -16 if few else 2.0 ** -8
    eg = np.abs(dg) * (step + 4 * U) + 1.01 * np.abs(dy * u) * b
    eu = np.abs(du) * (step + 4 * U) + 1.01 * np.abs(dy) * b
    dx, dwg, dwu = dg @ wg + du @ wu, dg.T @ x, du.T @ x
    H, M = (2 if few else 1) * (g.shape[1] + 64), (2 if few else 1) * (g.shape[0] + 64)  # padded with zeros
    ag, au = np.abs(dg) + eg, np.abs(du) + eu
    bx = eg @ np.abs(wg) + eu @ np.abs(wu) + 4 * H * U * (ag @ np.abs(wg) + au @ np.abs(wu))
    bwg = eg.T @ np.abs(x) + 2 * M * U * (ag.T @ np.abs(x))
    bwu = eu.T @ np.abs(x) + 2 * M * U * (au.T @ np.abs(x))
    return (dx, dwg, dwu), (bx, bwg, bwu)


def check(got, want, bound, dtype, name):
    got = f64(got)
    assert got.shape == want.shape, name
    assert np.isfinite(got).all(), f"{name}: not finite"
    # half a step of a value that lies within `bound` of the exact one; the type's smallest
    # normal covers results below it
    room = bound + half(dtype) * (np.abs(want) + bound) + torch.finfo(dtype).tiny
    off = np.abs(got - want)
    worst = np.max(off / room) if off.size else 0.0
    print(f"  {name}: max error {off.max():.3e}, {worst:.3f} of its bound", flush=True)
    assert worst <= 1, f"{name}: {worst} times the bound at {np.unravel_index(np.argmax(off / room), off.shape)}"
