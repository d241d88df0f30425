"""GPU parity of the gated feed-forward block and its gradient against their definitions in 64
bits, and a run of the block's operators together as the layer policy makes them."""
import numpy as np
import pytest
import torch

import _block as B
from _gpu import Guarded

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
BF = torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rnd(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def inputs(M, K, H, seed=1):
    return rnd(seed, M, K), rnd(seed + 1, H, K, std=K ** -0.5), rnd(seed + 2, H, K, std=K ** -0.5)


# M, K, H: one row, the row counts around each kernel's limits, one K step, odd widths, ragged
# tiles in both directions
SHAPES = [
    (1, 64, 16), (1, 1344, 333), (2, 320, 7), (15, 640, 130), (16, 64, 1), (17, 128, 50), (32, 704, 96), (33, 192, 64),
    (48, 512, 31), (64, 256, 200), (65, 64, 65), (130, 448, 1), (200, 1088, 77), (257, 320, 516), (300, 256, 260),
    (700, 128, 1000), (1029, 192, 4100), (3000, 64, 2049),
    (64, 64, 11000), (100, 1344, 1500), (140, 832, 5000), (400, 320, 6000), (3100, 4096, 70), (90, 3200, 2049),  # the gradients' larger tiles
]


# the forward product's larger tiles and its small ones one and two to a CU: rows that end on a
# 128-byte line, inside one, and at an odd address
LARGE = [(300, 640, 4000), (300, 640, 4003), (200, 1408, 5001), (520, 192, 4096), (520, 192, 4099),
         (1700, 768, 4096), (1700, 768, 4100), (1601, 832, 3841), (1030, 1024, 5003)]


def label(c):
    return "x".join(map(str, c))


@pytest.mark.parametrize("c", SHAPES + LARGE, ids=label)
@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
def test_glu_fused(c, kind):
    M, K, H = c
    X, Wg, Wu = inputs(*c)
    outs = [Guarded((M, H), BF) for _ in range(3)]
    rtl.rtl_glu_fused(X, Wg, Wu, act=kind, Y=outs[0].t, G=outs[1].t, U=outs[2].t)
    y, g, u, by, bg, bu = B.glu_forward(B.f64(X), B.f64(Wg), B.f64(Wu), kind)
    for o, want, bound, name in zip(outs, (y, g, u), (by, bg, bu), "YGU"):
        B.check(o.t, want, bound, BF, name)
        o.check(name)
    assert torch.equal(rtl.rtl_glu_fused(X, Wg, Wu, act=kind), outs[0].t)  # kept or not, the same Y


@pytest.mark.parametrize("c", SHAPES, ids=label)
@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
def test_glu_backward(c, kind):
    M, K, H = c
    X, Wg, Wu = inputs(*c)
    G, U, dY = rnd(11, M, H, std=1.5), rnd(12, M, H), rnd(13, M, H, std=0.1)
    outs = [Guarded(s, BF) for s in ((M, K), (H, K), (H, K))]
    rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY, act=kind, dX=outs[0].t, dWg=outs[1].t, dWu=outs[2].t)
    want, bounds = B.glu_backward(*map(B.f64, (X, Wg, Wu, G, U, dY)), kind)
    for o, w, b, name in zip(outs, want, bounds, ("dX", "dWg", "dWu")):
        B.check(o.t, w, b, BF, name)
        o.check(name)
    dX, a, b = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY, act=kind, need_dw=False)
    assert a is None and b is None and torch.equal(dX, outs[0].t)
    n, dWg, dWu = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY, act=kind, need_dx=False)
    assert n is None and torch.equal(dWg, outs[1].t) and torch.equal(dWu, outs[2].t)


@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
def test_gradient_against_differences(kind):
    """Forward and gradient as a training step chains them, against central differences of the
    definition.  G and U are kept in bf16 and dG and dU round again, each 2^-8 relative: the
    product with a direction is within 4 * 2^-8 of the sum of magnitudes, the step's third
    order term far below."""
    M, K, H = 24, 128, 96
    X, Wg, Wu = inputs(M, K, H, seed=20)
    dY = rnd(23, M, H)
    G, U = torch.empty((M, H), dtype=BF, device="cuda"), torch.empty((M, H), dtype=BF, device="cuda")
    rtl.rtl_glu_fused(X, Wg, Wu, act=kind, G=G, U=U)
    grads = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY, act=kind)
    at, dy = [B.f64(t) for t in (X, Wg, Wu)], B.f64(dY)
    f = lambda p: (B.act(p[0] @ p[1].T, kind)[0] * (p[0] @ p[2].T) * dy).sum()
    for i, grad in enumerate(grads):
        v = B.f64(rnd(30 + i, *grad.shape))
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-4 * v, at[i] - 1e-4 * v
        diff = (f(up) - f(down)) / 2e-4
        assert abs((B.f64(grad) * v).sum() - diff) <= 4 * 2.0 ** -8 * np.abs(B.f64(grad) * v).sum()


@pytest.mark.parametrize("kind", (0, 1), ids=("silu", "gelu"))
@pytest.mark.parametrize("M", (3, 200))
def test_far_pre_activations(kind, M):
    """Pre-activations of both signs far out on the activation: no infinity or NaN."""
    K, H = 64, 40
    X, Wg, Wu = rnd(40, M, K, std=30.0), rnd(41, H, K), rnd(42, H, K)
    Y = rtl.rtl_glu_fused(X, Wg, Wu, act=kind)
    y, g, u, by, _, _ = B.glu_forward(B.f64(X), B.f64(Wg), B.f64(Wu), kind)
    assert np.abs(g).max() > 600
    B.check(Y, y, by, BF, "Y")
    G, U, dY = rnd(43, M, H, std=200.0), rnd(44, M, H), rnd(45, M, H)
    got = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY, act=kind)
    for t, w, b, n in zip(got, *B.glu_backward(*map(B.f64, (X, Wg, Wu, G, U, dY)), kind), ("dX", "dWg", "dWu")):
        B.check(t, w, b, BF, n)


@pytest.mark.parametrize("M", (5, 150))
def test_rows_apart(M):
    """A token of NaN stays in its own rows of Y, G, U and dX."""
    K, H = 256, 72
    X, Wg, Wu = inputs(M, K, H)
    want = rtl.rtl_glu_fused(X, Wg, Wu)
    G, U, dY = rnd(51, M, H), rnd(52, M, H), rnd(53, M, H)
    dX = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY, need_dw=False)[0]
    X2, G2 = X.clone(), G.clone()
    X2[3], G2[2] = float("nan"), float("nan")
    got = rtl.rtl_glu_fused(X2, Wg, Wu)
    dX2 = rtl.rtl_glu_backward(X, Wg, Wu, G2, U, dY, need_dw=False)[0]
    rows = torch.arange(M, device="cuda")
    assert torch.equal(got[rows != 3], want[rows != 3]) and bool(torch.isnan(got[3]).all())
    assert torch.equal(dX2[rows != 2], dX[rows != 2]) and bool(torch.isnan(dX2[2]).all())


@pytest.mark.parametrize("M", (1, 40, 300))
def test_streams_graph_replay_and_repeat(M):
    """On another stream, captured and replayed on new inputs between eager calls, and the same
    bits on every run."""
    K, H = 512, 328
    X, Wg, Wu = inputs(M, K, H)
    G, U, dY = rnd(61, M, H), rnd(62, M, H), rnd(63, M, H)
    eager = lambda: (rtl.rtl_glu_fused(X, Wg, Wu), *rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY))
    first = eager()
    assert all(torch.equal(a, b) for a, b in zip(first, eager()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y = rtl.rtl_glu_fused(X, Wg, Wu, stream=side)
    grads = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (Y, *grads)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = eager()
    for k in range(3):
        X.copy_(rnd(70 + k, M, K))
        dY.copy_(rnd(80 + k, M, H))
        want = eager()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
