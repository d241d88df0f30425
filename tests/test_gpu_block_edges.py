"""GPU tests of the block operators where their arithmetic leaves the ordinary: infinities, values
at the ends of the types' ranges, tensors of no heads, and long sums."""
import numpy as np
import pytest
import torch

import _block as B
from _gpu import Guarded

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
BF, F32 = torch.bfloat16, torch.float32


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rnd(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def same_nonfinite(got, want, name):
    """The same elements NaN, and the same infinite with the same sign."""
    got = B.f64(got)
    for what, a, b in (("NaN", np.isnan(got), np.isnan(want)), ("+inf", got == np.inf, want == np.inf),
                       ("-inf", got == -np.inf, want == -np.inf)):
        assert (a == b).all(), f"{name}: {what} at {np.argwhere(a)[:4]}, expected at {np.argwhere(b)[:4]}"


def check_glu_gradient(args, kind, same=True):
    """The gradient's outputs: infinite and NaN where the definition's are, the others within its
    bounds (which the infinite operands do not enter: a finite element meets none of them)."""
    got = rtl.rtl_glu_backward(*args, act=kind)
    with np.errstate(invalid="ignore", over="ignore"):
        want, _ = B.glu_backward(*map(B.f64, args), kind)
        _, bounds = B.glu_backward(*(np.nan_to_num(B.f64(t), nan=0.0, posinf=0.0, neginf=0.0) for t in args), kind)
    for t, w, b, name in zip(got, want, bounds, ("dX", "dWg", "dWu")):
        same_nonfinite(t, w, name)
        fine = np.isfinite(w)
        B.check(torch.where(torch.isfinite(t), t, torch.zeros_like(t)), np.where(fine, w, 0.0), b, BF, name)


# 2^14 elements of G at most (the gradient's two-part form), and more
@pytest.mark.parametrize("M,H", ((1, 64), (3, 72), (40, 100), (200, 130)))
@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
@pytest.mark.parametrize("where", ("dY", "U", "Wg", "Wu", "X"))
def test_gradient_of_infinities(where, kind, M, H):
    K = 128
    args = [rnd(1, M, K), rnd(2, H, K, std=K ** -0.5), rnd(3, H, K, std=K ** -0.5), rnd(4, M, H, std=1.5),
            rnd(5, M, H), rnd(6, M, H, std=0.1)]
    m, h = M - 1, H // 2
    # dG of 1/2 or 1 exactly, and dU of 0: what is left of them after one rounding is 0
    args[3][:, 3], args[4][:, 3], args[5][:, 3] = 0.0, 1.0, 1.0
    args[3][:, h], args[4][:, h] = 0.75, 1.25  # no zero meets an infinity
    at = {"dY": (5, m, h), "U": (4, m, h), "Wg": (1, h, 7), "Wu": (2, h, 70), "X": (0, m, 9)}[where]
    args[at[0]][at[1], at[2]] = float("-inf") if M == 3 else float("inf")
    if where == "Wg":
        args[1][3, 8] = float("inf")
    check_glu_gradient(args, kind)


# the streamed kernel, small tiles, large tiles
@pytest.mark.parametrize("M,K,H", ((2, 128, 70), (150, 192, 700), (1100, 640, 4003)))
@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
@pytest.mark.parametrize("where", ("X", "Wg", "Wu"))
def test_forward_of_infinities(where, kind, M, K, H):
    """An infinite token or weight gives infinities and NaN in its own row or column, as defined."""
    args = dict(X=rnd(1, M, K), Wg=rnd(2, H, K, std=K ** -0.5), Wu=rnd(3, H, K, std=K ** -0.5))
    fine = B.glu_forward(*map(B.f64, args.values()), kind)
    args[where][1, 5] = float("inf")
    G, U = torch.empty(M, H, dtype=BF, device="cuda"), torch.empty(M, H, dtype=BF, device="cuda")
    Y = rtl.rtl_glu_fused(**args, act=kind, G=G, U=U)
    with np.errstate(invalid="ignore"):
        want = B.glu_forward(*map(B.f64, args.values()), kind)[:3]
    for t, w, b, name in zip((Y, G, U), want, fine[3:], "YGU"):
        same_nonfinite(t, w, name)
        B.check(torch.where(torch.isfinite(t), t, torch.zeros_like(t)), np.where(np.isfinite(w), w, 0.0), b, BF, name)


@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
def test_gradient_past_bf16(kind):
    """dU above the largest bf16 value but within fp32's, in the two-part form: its products with
    small weights and tokens are finite."""
    M, K, H = 3, 64, 40
    X, Wg, Wu = rnd(1, M, K, std=2.0 ** -20), rnd(2, H, K, std=2.0 ** -20), rnd(3, H, K, std=2.0 ** -20)
    G, U, dY = rnd(4, M, H, std=1.5), rnd(5, M, H, std=2.0 ** -30), rnd(6, M, H, std=0.1)
    # a G whose activation times a dY of bf16 falls between the two types' ends
    steps = torch.arange(1 << 14, dtype=torch.int32)
    g = ((0x3F80 + steps[:256]).to(torch.int16)).view(BF).double().numpy()  # 1 to 4
    d = ((0x7E80 + steps[:256]).to(torch.int16)).view(BF).double().numpy()  # 2^126 up to the largest
    v = B.act(g, kind)[0][:, None] * d[None]
    i, j = np.unravel_index(np.argmin(np.abs(v - 3.399e38)), v.shape)
    assert 3.3965e38 < v[i, j] < 3.402e38
    G[1, 7], dY[1, 7], U[1, 7] = float(g[i]), float(d[j]), 2.0 ** -30
    check_glu_gradient([X, Wg, Wu, G, U, dY], kind)


# eps and the heads' size: zero heads with a root of their eps, sizes whose cube leaves fp32
RANGES = [(2.0 ** -126, 0.0, F32), (1e-30, 0.0, BF), (1e-30, 2.0 ** -45, F32), (2.0 ** -126, 2.0 ** -61, BF),
          (1e-6, 2.0 ** 45, F32), (1e-6, 2.0 ** 45, BF), (1e-6, 2.0 ** 55, F32), (1e-6, 2.0 ** 55, BF), (1.0, 2.0 ** 58, F32)]


@pytest.mark.parametrize("eps,size,dt", RANGES)
@pytest.mark.parametrize("D", (32, 256))
def test_head_norm_range(eps, size, dt, D):
    """Norm and gradient wherever the squares lie in fp32's range."""
    M, H, dims = 9, 3, (8, 16)
    Q, w, dY, pos = rnd(1, M, H, D, std=size, dtype=dt), rnd(2, D, dtype=dt) + 1, rnd(3, M, H, D, dtype=dt), rnd(4, M, 2, dtype=F32)
    Q[2] = 0
    phi, e = B.angles(B.f64(pos), dims, 10000.0), float(np.float32(eps))
    Qo, _ = rtl.rtl_qk_norm_rope(Q, None, w, None, pos, dims, eps=eps)
    B.check(Qo, *B.qk_forward(B.f64(Q), B.f64(w), phi, 0, e), dt, "Qo")
    dQ, _, dqw, _ = rtl.rtl_qk_norm_rope_backward(Q, None, w, None, pos, dims, dY, None, eps=eps)
    dx, dw, bx, bw = B.qk_backward(B.f64(Q), B.f64(w), phi, 0, e, B.f64(dY))
    B.check(dQ, dx, bx, dt, "dQ")
    B.check(dqw, dw, bw, F32, "dqw")


def test_head_norm_gradient_of_large_gradients():
    """Large heads under a large gradient: their product leaves fp32's range, the gradient does not."""
    M, H, D = 9, 3, 64
    Q, w, dY = rnd(1, M, H, D, std=2.0 ** 58, dtype=F32), rnd(2, D, dtype=F32) + 1, rnd(3, M, H, D, std=2.0 ** 75, dtype=F32)
    dQ, _, dqw, _ = rtl.rtl_qk_norm_rope_backward(Q, None, w, None, None, (), dY, None)
    dx, dw, bx, bw = B.qk_backward(B.f64(Q), B.f64(w), np.zeros((M, 0)), 0, 1e-6, B.f64(dY))
    B.check(dQ, dx, bx, F32, "dQ")
    B.check(dqw, dw, bw, F32, "dqw")


@pytest.mark.parametrize("given", (False, True))
def test_no_key_heads(given):
    """Keys of no heads: their outputs are empty, the gradient of their weights is an empty sum."""
    M, H, D = 5, 2, 64
    Q, K, w, dY, dK = rnd(1, M, H, D), rnd(2, M, 0, D), rnd(3, D), rnd(4, M, H, D), rnd(5, M, 0, D)
    Qo, Ko = rtl.rtl_qk_norm_rope(Q, K, w, w, None, ())
    assert Ko.shape == (M, 0, D) and torch.equal(Qo, rtl.rtl_qk_norm_rope(Q, None, w, None, None, ())[0])
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        held = torch.full((D,), 7.0, device="cuda")
        if not given:  # the next allocation of its size is that memory
            torch.cuda.synchronize()
            del held
        how = dict(dkw=held) if given else {}
        want = rtl.rtl_qk_norm_rope_backward(Q, None, w, None, None, (), dY, None)
        dQ, dKs, dqw, dkw = rtl.rtl_qk_norm_rope_backward(Q, K, w, w, None, (), dY, dK, stream=stream, **how)
        torch.cuda.synchronize()
        assert dKs.shape == (M, 0, D) and torch.equal(dQ, want[0]) and torch.equal(dqw, want[2])
        assert bool((dkw == 0).all())


@pytest.mark.parametrize("dt", (BF, F32))
def test_long_sums(dt):
    """Norm weights' gradients over 14 million heads of one sign, most of which one lane adds one
    after another: all heads alike, so that every addition to a sum rounds the same way."""
    M, H, D = 40_000, 350, 256
    x, dy, w = rnd(1, D, dtype=dt).abs() + 0.25, rnd(2, D, dtype=dt).abs() + 0.25, rnd(3, D, dtype=dt)
    spread = lambda t, n: t.view(1, 1, D).expand(M, n, D)
    dx = torch.empty(M, H, D, dtype=dt, device="cuda")
    _, _, dqw, dkw = rtl.rtl_qk_norm_rope_backward(spread(x, H), spread(x, 1), w, w, None, (), spread(dy, H), spread(dy, 1),
                                                   dQ=dx)
    one = B.f64(dy) * B.f64(x) / np.sqrt((B.f64(x) ** 2).mean() + 1e-6)
    B.check(dqw, one * M * H, 128 * B.U * one * M * H, F32, "dqw")
    B.check(dkw, one * M, 128 * B.U * one * M, F32, "dkw")


# the sizes whose gradients take the larger tiles, parts of a tile's sum, and the few-element form
EXACT = [(1, 1344, 333), (15, 640, 130), (64, 64, 11000), (400, 320, 6000), (100, 1344, 1500), (140, 832, 5000),
         (3100, 4096, 70), (90, 3200, 2049), (257, 320, 516), (1029, 192, 4100), (2050, 768, 3001)]


def label(c):
    return "x".join(map(str, c))


def exact_inputs(M, K, H, gen):
    """Gates of 0 and 64, whose activation is 0 and 64 with slopes 1/2 and 1; all else -1, 0, 1."""
    def three(*shape):
        return torch.randint(-1, 2, shape, generator=gen, device="cuda", dtype=torch.int8).to(BF)

    G = torch.randint(0, 2, (M, H), generator=gen, device="cuda", dtype=torch.int8).to(BF) * 64
    return three(M, K), three(H, K), three(H, K), G, three(M, H), three(M, H)


def exact_parts(G, U, dY):
    return dY.double() * U.double() * torch.where(G == 0, 0.5, 1.0), dY.double() * G.double()


# GELU's Phi(0) is off by its approximation's error, which only the rounding to one part takes away
@pytest.mark.parametrize("kind,c", [(k, c) for k in (0, 1) for c in EXACT if k == 0 or c[0] * c[2] > 2 ** 14],
                         ids=lambda v: label(v) if isinstance(v, tuple) else ("silu", "gelu")[v])
def test_gradient_sums_exact(kind, c):
    """Every term of every sum: inputs whose products and sums are halves of whole numbers below
    2^24, so that each output is its exact value rounded once (a lost or repeated step of a sum
    shows, where a bound on the roundings of all its terms leaves room for it)."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    X, Wg, Wu, G, U, dY = exact_inputs(*c, gen)
    got = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY, act=kind)
    dg, du = (t.cpu() for t in exact_parts(G, U, dY))
    x, wg, wu = (t.double().cpu() for t in (X, Wg, Wu))
    for t, want, name in zip(got, (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x), ("dX", "dWg", "dWu")):
        assert torch.equal(t.cpu(), want.to(BF)), f"{name}: off by {(t.cpu().double() - want).abs().max()}"


@pytest.mark.parametrize("c", [(1_020_000, 2112, 96), (1_020_000, 64, 2112)], ids=label)
def test_gradient_sums_exact_far(c):
    """The same where P, X or dX pass 2^32 bytes, every token with terms of its own: the weights'
    gradients in full, the tokens' at both ends and in the middle."""
    M, K, H = c
    gen = torch.Generator(device="cuda").manual_seed(8)
    X, Wg, Wu, G, U, dY = exact_inputs(M, K, H, gen)
    dX, dWg, dWu = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY)
    want = [torch.zeros(H, K, dtype=torch.float64, device="cuda") for _ in range(2)]
    n = 1 << 16
    for m in range(0, M, n):
        x = X[m:m + n].double()
        for w, p in zip(want, exact_parts(G[m:m + n], U[m:m + n], dY[m:m + n])):
            w += torch.mm(p.t().contiguous(), x)
    assert torch.equal(dWg, want[0].to(BF)) and torch.equal(dWu, want[1].to(BF))
    for m in (0, M // 2, M - 300):
        dg, du = exact_parts(G[m:m + 300], U[m:m + 300], dY[m:m + 300])
        assert torch.equal(dX[m:m + 300], (torch.mm(dg, Wg.double()) + torch.mm(du, Wu.double())).to(BF))
    del X, dX, G, U, dY, x, p
    torch.cuda.empty_cache()


# every bf16 value to 40 in magnitude as a pre-activation: rows of the streamed and of the tiled kernels
@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
@pytest.mark.parametrize("rows", (16, 1 << 15))
def test_activation_sweep(kind, rows):
    """Value and slope of the activation by themselves, through weights of one 1: relative bounds on
    the negative side, where both fall off.

    SiLU: exp(-g) is within (2 |g| + 4) u, a sum, a reciprocal and a product add under 8 u: value
    within (2 |g| + 12) u of itself, slope likewise of p (1 + |g|).  GELU: the published polynomial
    P(t) exp(-x^2) / 2 stands for Phi(-|g|); the argument x^2 = g^2 / 2 is within 7 u of itself, exp within 4 g^2 + 8 u,
    the polynomial (five steps, coefficients up to 1.5, a result of 0.1 or more) within 40 u: (4 g^2
    + 60) u of it, 1 - tail adds u.  The polynomial itself is within 1.5e-7 of erf, and of its tail
    within 6e-5 to g = -3, 5e-4 to -4, 1.1% to -8 and 4% to -13.2; past that exp(-x^2) lies below fp32's normal numbers
    (exp(-87.8) = 7.5e-39 < 2^-126) and may be 0: 2^-126 of it."""
    bits = torch.arange(0x4221, dtype=torch.int32)
    g = torch.cat([bits, bits - 0x8000]).to(torch.int16).view(BF)
    g = g[(g == 0) | (g.abs().float() > 2.0 ** -100)]
    if rows == 16:
        g = g[torch.linspace(0, len(g) - 1, rows).long()]
    M, K, u = len(g), 64, B.U
    X = torch.zeros(M, K, dtype=BF)
    X[:, 0], X[:, 1] = g, 1.0
    Wg, Wu = torch.zeros(1, K, dtype=BF), torch.zeros(1, K, dtype=BF)
    Wg[0, 0], Wu[0, 1] = 1.0, 1.0
    X, Wg, Wu, gd = X.cuda(), Wg.cuda(), Wu.cuda(), g.cuda().view(M, 1)
    one = torch.ones_like(gd)
    G, U = torch.empty_like(gd), torch.empty_like(gd)
    Y = rtl.rtl_glu_fused(X, Wg, Wu, act=kind, G=G, U=U)
    assert torch.equal(G, gd) and torch.equal(U, one)
    dX = rtl.rtl_glu_backward(X, Wg, Wu, gd, one, one, act=kind, need_dw=False)[0]
    x = B.f64(g)
    a = np.abs(x)
    if kind == 0:
        value, slope = B.act(x, 0)
        p = 1 / (1 + np.exp(-x))
        bv, bs = (2 * a + 12) * u * np.abs(value), (2 * a + 12) * u * p * (1 + a)
    else:
        phi = np.exp(-x * x / 2) / np.sqrt(2 * np.pi)
        tail = 0.5 * torch.special.erfc(torch.from_numpy(a / np.sqrt(2))).numpy()
        cut = np.select([a <= 3, a <= 4, a <= 8, a <= 13.2], [6e-5, 5e-4, 1.1e-2, 4e-2], 0.4)
        p = np.where(x < 0, tail, 1 - tail)
        value, slope = x * p, p + x * phi
        end = torch.finfo(F32).tiny
        bp = end + np.minimum(0.75e-7, cut * tail) + (4 * x * x + 60) * u * tail + np.where(x < 0, 0, 2 * u)
        bv = a * bp + 2 * u * np.abs(value)
        bs = bp + a * end + (4 * x * x + 8) * u * a * phi + 2 * u * (p + a * phi)
    few = 2.0 ** -16 if M <= 2 ** 14 else 2.0 ** -8  # the gradient's operands, rounded
    zero = np.zeros_like(x)
    B.check(Y[:, 0], value, bv, BF, "Y")
    B.check(dX[:, 0], slope, bs + few * (np.abs(slope) + bs), BF, "slope")
    B.check(dX[:, 1], value, bv + few * (np.abs(value) + bv), BF, "value in the gradient")
    assert not dX[:, 2:].any()


# one forward tile to a CU, on either side of the K from which its waves are square: rows that end on a
# 128-byte line, inside one, and at an odd address
@pytest.mark.parametrize("c", [(200, 1920, 5001), (200, 1984, 5001), (300, 1984, 4000), (257, 2112, 3844)], ids=label)
@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
def test_one_tile_to_a_cu(c, kind):
    M, K, H = c
    X, Wg, Wu = rnd(1, M, K), rnd(2, H, K, std=K ** -0.5), rnd(3, H, K, std=K ** -0.5)
    outs = [Guarded((M, H), BF) for _ in range(3)]
    rtl.rtl_glu_fused(X, Wg, Wu, act=kind, Y=outs[0].t, G=outs[1].t, U=outs[2].t)
    want = B.glu_forward(B.f64(X), B.f64(Wg), B.f64(Wu), kind)
    for o, w, bound, name in zip(outs, want[:3], want[3:], "YGU"):
        B.check(o.t, w, bound, BF, name)
        o.check(name)


def test_outputs_given_by_the_caller_count_as_changed():
    """Tensors that a call writes in place have a new version, so that torch's autograd refuses to use
    them where it kept them for a backward pass."""
    M, H, D, K = 3, 2, 64, 128
    pos, w = rnd(1, M, 1, dtype=F32), rnd(2, D)
    q, k, dq, dk, y = (rnd(3 + i, M, H, D) for i in range(5))
    x, wg, wu, s, t = rnd(9, M, K), rnd(10, K, K), rnd(11, K, K), rnd(12, M, K), rnd(13, M, K)
    dqw, dkw = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    out = [torch.empty_like(wg) for _ in range(2)] + [torch.empty_like(x) for _ in range(3)]

    def grows(call, *written, kept=()):
        before = [a._version for a in (*written, *kept)]
        call()
        after = [a._version for a in (*written, *kept)]
        n = len(written)
        assert all(b > a for a, b in zip(before[:n], after[:n])) and after[n:] == before[n:]

    grows(lambda: rtl.rtl_rope_axes(y, pos, (D,), Y=y), y, kept=(pos,))
    grows(lambda: rtl.rtl_qk_norm_rope(q, k, w, w, pos, (D,), Qo=q, Ko=k), q, k, kept=(w,))
    grows(lambda: rtl.rtl_qk_norm_rope_backward(q, k, w, w, pos, (D,), dq, dk, dQ=dq, dK=dk, dqw=dqw, dkw=dkw),
          dq, dk, dqw, dkw, kept=(q, k))
    grows(lambda: rtl.rtl_glu_fused(x, wg, wu, Y=out[2], G=s, U=t), out[2], s, t, kept=(x, wg))
    grows(lambda: rtl.rtl_glu_backward(x, wg, wu, s, t, out[2], dX=out[3], dWg=out[0], dWu=out[1]), out[3], out[0], out[1],
          kept=(x, s, t))
    scale = torch.ones(M, H, D, dtype=BF, device="cuda", requires_grad=True)
    loss = (y * scale).sum()  # keeps y
    rtl.rtl_rope_axes(y, pos, (D,), Y=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        z = torch.zeros(M, H, D, dtype=BF, device="cuda")
        assert rtl.rtl_rope_axes(z, pos, (D,), Y=z) is z
