"""GPU parity of rotary positions over several axes and of the per-head norms of queries and
keys with the rotation, forward and gradient, against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import _block as B

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rnd(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def positions(seed, M, axes, far=0.0):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(-200, 2000, (M, axes), generator=g).float() * 0.75
    p[0] = 0
    return (p + far).cuda()


BF, F32 = torch.bfloat16, torch.float32
# M, H, D, dims, pairs, dtype, far: one token to many, one head to many, every group width,
# heads that do not fill their lanes, channels left unturned, far and fractional positions
SHAPES = [
    (1, 1, 8, (8,), 0, BF, 0), (1, 24, 128, (16, 56, 56), 0, BF, 0), (3, 5, 40, (8, 8, 8), 1, F32, 0),
    (77, 6, 80, (8, 32, 32), 1, F32, 0), (333, 7, 72, (2, 70), 1, BF, 1e5), (130, 3, 96, (16, 24, 24), 0, F32, 1e6),
    (65, 2, 256, (64, 64, 64, 64), 1, BF, 0), (19, 9, 160, (6, 10, 16), 0, BF, 12345.5), (1000, 40, 64, (64,), 1, BF, 0),
    (4099, 24, 128, (44, 42, 42), 0, BF, 0), (2050, 33, 128, (44, 42, 42), 1, F32, 0), (515, 70, 24, (24,), 0, BF, 0),
]


def label(c):
    return "x".join(map(str, c[:3])) + f"-{'halves' if c[4] else 'adjacent'}-{str(c[5])[6:]}"


def strided(M, H, D, dtype, layout):
    """A [M,H,D] tensor of `layout` and the buffer it lies in, filled with 7."""
    if layout == "packed":       # beside two other projections of a row
        buf = torch.full((M, H + 3, D), 7.0, dtype=dtype, device="cuda")
        return buf[:, 2:2 + H], buf
    if layout == "head-major":
        buf = torch.full((H, M, D), 7.0, dtype=dtype, device="cuda")
        return buf.transpose(0, 1), buf
    if layout == "interleaved":  # q, k, v of each head side by side
        buf = torch.full((M, H, 3, D), 7.0, dtype=dtype, device="cuda")
        return buf[:, :, 1], buf
    buf = torch.full((M, H, D), 7.0, dtype=dtype, device="cuda")
    return buf, buf


LAYOUTS = ("contiguous", "packed", "head-major", "interleaved")


@pytest.mark.parametrize("c", SHAPES, ids=label)
@pytest.mark.parametrize("inverse", (False, True))
def test_rope(c, inverse):
    M, H, D, dims, pairs, dt, far = c
    X, pos = rnd(1, M, H, D, dtype=dt), positions(2, M, len(dims), far)
    Y = rtl.rtl_rope_axes(X, pos, dims, theta=10000.0, pairs=pairs, inverse=inverse)
    phi = B.angles(B.f64(pos), dims, 10000.0)
    want = B.rotate(B.f64(X), phi, pairs, -1.0 if inverse else 1.0)
    n = phi.shape[1]
    B.check(Y, want, B.TURN * B.pair_sum(B.f64(X), n, pairs), dt, "Y")
    assert torch.equal(Y[..., 2 * n:], X[..., 2 * n:])  # unturned channels are copied
    assert torch.equal(Y[0], X[0]) if far == 0 else True  # the origin turns nothing


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", (BF, F32))
def test_rope_layouts_and_in_place(layout, dt):
    M, H, D, dims = 37, 6, 72, (8, 32, 24)
    pos = positions(3, M, 3)
    src = rnd(4, M, H, D, dtype=dt)
    plain = rtl.rtl_rope_axes(src, pos, dims, pairs=rtl.RTL_ROPE_HALVES)
    for other in LAYOUTS:
        X, _ = strided(M, H, D, dt, layout)
        X.copy_(src)
        Y, buf = strided(M, H, D, dt, other)
        rtl.rtl_rope_axes(X, pos, dims, pairs=rtl.RTL_ROPE_HALVES, Y=Y)
        assert torch.equal(Y, plain)
        Y.fill_(7.0)
        assert bool((buf == 7.0).all()), "a store beside the output"
    X, buf = strided(M, H, D, dt, layout)
    X.copy_(src)
    assert rtl.rtl_rope_axes(X, pos, dims, pairs=rtl.RTL_ROPE_HALVES, Y=X) is X
    assert torch.equal(X, plain)
    X.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_rope_repeated_input():
    """One head's row repeated over tokens and heads by zero strides."""
    x, pos = rnd(5, 1, 1, 64, dtype=BF), positions(6, 50, 2)
    Y = rtl.rtl_rope_axes(x.expand(50, 4, 64), pos, (32, 32))
    assert torch.equal(Y, rtl.rtl_rope_axes(x.expand(50, 4, 64).contiguous(), pos, (32, 32)))


def qk_inputs(c, Hk, seed=10):
    M, H, D, dims, pairs, dt, far = c
    return (rnd(seed, M, H, D, dtype=dt, std=2.0), rnd(seed + 1, M, Hk, D, dtype=dt, std=0.3),
            rnd(seed + 2, D, dtype=dt) + 1, rnd(seed + 3, D, dtype=dt) + 1, positions(seed + 4, M, len(dims), far))


@pytest.mark.parametrize("c", SHAPES, ids=label)
def test_qk_norm_rope(c):
    M, H, D, dims, pairs, dt, _ = c
    Hk = max(1, H // 3)
    Q, K, qw, kw, pos = qk_inputs(c, Hk)
    Qo, Ko = rtl.rtl_qk_norm_rope(Q, K, qw, kw, pos, dims, theta=256.0, eps=1e-6, pairs=pairs)
    phi = B.angles(B.f64(pos), dims, 256.0)
    for name, x, w, y in (("Qo", Q, qw, Qo), ("Ko", K, kw, Ko)):
        B.check(y, *B.qk_forward(B.f64(x), B.f64(w), phi, pairs, 1e-6), dt, name)


@pytest.mark.parametrize("c", SHAPES, ids=label)
def test_qk_norm_rope_backward(c):
    M, H, D, dims, pairs, dt, _ = c
    Hk = max(1, H // 3)
    Q, K, qw, kw, pos = qk_inputs(c, Hk)
    dQo, dKo = rnd(20, M, H, D, dtype=dt, std=0.1), rnd(21, M, Hk, D, dtype=dt, std=0.1)
    run = lambda: rtl.rtl_qk_norm_rope_backward(Q, K, qw, kw, pos, dims, dQo, dKo, theta=256.0, eps=1e-6, pairs=pairs)
    dQ, dK, dqw, dkw = run()
    phi = B.angles(B.f64(pos), dims, 256.0)
    for name, x, w, dy, dx, dw in (("q", Q, qw, dQo, dQ, dqw), ("k", K, kw, dKo, dK, dkw)):
        rx, rw, bx, bw = B.qk_backward(B.f64(x), B.f64(w), phi, pairs, 1e-6, B.f64(dy))
        B.check(dx, rx, bx, dt, "d" + name)
        B.check(dw, rw, bw, F32, f"d{name}w")
    for a, b in zip((dQ, dK, dqw, dkw), run()):
        assert torch.equal(a, b)  # the same on every run


def test_qk_gradient_against_differences():
    """The gradient's product with a direction against a central difference of the definition
    (third order terms: step 1e-4 leaves about 1e-8 of it) and the kernel's forward."""
    M, H, D, dims = 5, 3, 32, (8, 8, 16)
    Q, qw, pos = rnd(30, M, H, D), rnd(31, D) + 1, positions(32, M, 3)
    dY = rnd(33, M, H, D)
    dQ, _, dqw, _ = rtl.rtl_qk_norm_rope_backward(Q, None, qw, None, pos, dims, dY, None, eps=1e-3)
    phi = B.angles(B.f64(pos), dims, 10000.0)
    q, w, dy = B.f64(Q), B.f64(qw), B.f64(dY)
    f = lambda q_, w_: (B.qk_forward(q_, w_, phi, 0, 1e-3)[0] * dy).sum()
    vq, vw = B.f64(rnd(34, M, H, D)), B.f64(rnd(35, D))
    h = 1e-4
    for got, diff, size in (((B.f64(dQ) * vq).sum(), f(q + h * vq, w) - f(q - h * vq, w), np.abs(B.f64(dQ) * vq).sum()),
                            ((B.f64(dqw) * vw).sum(), f(q, w + h * vw) - f(q, w - h * vw), np.abs(B.f64(dqw) * vw).sum())):
        assert abs(got - diff / (2 * h)) <= 1e-5 * size


def test_qk_views_of_one_projection_in_place():
    """Queries and keys as views of the packed projection, written in place, and their gradients
    written over the gradients from above; the values beside them stay."""
    M, H, Hk, D, dims = 130, 6, 2, 64, (16, 24, 24)
    qkv = rnd(40, M, H + 2 * Hk, D, dtype=BF)
    keep = qkv.clone()
    Q, K = qkv[:, :H], qkv[:, H:H + Hk]
    qw, kw, pos = rnd(41, D, dtype=BF), rnd(42, D, dtype=BF), positions(43, M, 3)
    want = rtl.rtl_qk_norm_rope(Q, K, qw, kw, pos, dims)
    d = rnd(44, M, H + 2 * Hk, D, dtype=BF)
    grads = rtl.rtl_qk_norm_rope_backward(Q, K, qw, kw, pos, dims, d[:, :H], d[:, H:H + Hk])
    dkeep = d.clone()
    got = rtl.rtl_qk_norm_rope_backward(Q, K, qw, kw, pos, dims, d[:, :H], d[:, H:H + Hk], dQ=d[:, :H],
                                        dK=d[:, H:H + Hk])
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert torch.equal(d[:, H + Hk:], dkeep[:, H + Hk:])
    rtl.rtl_qk_norm_rope(Q, K, qw, kw, pos, dims, Qo=Q, Ko=K)
    assert torch.equal(Q, want[0]) and torch.equal(K, want[1])
    assert torch.equal(qkv[:, H + Hk:], keep[:, H + Hk:])


def test_qk_options():
    """No keys, no weights, no rotation; heads of zeros give zeros and finite gradients."""
    M, H, D = 33, 4, 128
    Q, w = rnd(50, M, H, D, dtype=BF), rnd(51, D, dtype=BF)
    pos, dims = positions(52, M, 2), (64, 64)
    Q[3] = 0
    ones = torch.ones(D, dtype=BF, device="cuda")
    a, none = rtl.rtl_qk_norm_rope(Q, None, None, None, pos, dims)
    b, _ = rtl.rtl_qk_norm_rope(Q, Q.clone(), ones, w, pos, dims)
    assert none is None and torch.equal(a, b) and bool((a[3] == 0).all())
    still, _ = rtl.rtl_qk_norm_rope(Q, None, w, None, None, ())
    zero, _ = rtl.rtl_qk_norm_rope(Q, None, w, None, torch.zeros(M, 2, device="cuda"), dims)
    assert torch.equal(still, zero)
    dY = rnd(53, M, H, D, dtype=BF)
    dQ, dK, dqw, dkw = rtl.rtl_qk_norm_rope_backward(Q, None, w, None, None, (), dY, None)
    assert dK is None and dkw is None and bool(torch.isfinite(dQ).all())
    with pytest.raises(ValueError):
        rtl.rtl_qk_norm_rope(Q, None, w, None, pos, dims, Ko=Q)
    with pytest.raises(ValueError):
        rtl.rtl_qk_norm_rope_backward(Q, None, w, None, None, (), dY, None, dkw=torch.zeros(D, device="cuda"))
    x = B.f64(Q)
    rx, rw, bx, bw = B.qk_backward(x, B.f64(w), np.zeros((M, 0)), 0, 1e-6, B.f64(dY))
    B.check(dQ, rx, bx, BF, "dQ")
    B.check(dqw, rw, bw, F32, "dqw")


def test_rows_apart():
    """A row of infinities or NaN, or a position that is not finite, stays in its own outputs."""
    M, H, D, dims = 40, 3, 64, (32, 32)
    Q, w, pos = rnd(60, M, H, D, dtype=F32), rnd(61, D), positions(62, M, 2)
    want = rtl.rtl_qk_norm_rope(Q, None, w, None, pos, dims)[0]
    Q2, pos2 = Q.clone(), pos.clone()
    Q2[7, 1, 5], Q2[9, 2, 0], pos2[20, 1] = float("nan"), float("inf"), float("inf")
    got = rtl.rtl_qk_norm_rope(Q2, None, w, None, pos2, dims)[0]
    same = torch.ones(M, H, dtype=torch.bool, device="cuda")
    same[7, 1] = same[9, 2] = False
    same[20] = False
    assert torch.equal(got[same], want[same])
    assert bool(torch.isnan(got[7, 1]).all())


def test_streams_and_graph_replay():
    """On another stream, and captured and replayed on new inputs between eager calls."""
    M, H, Hk, D, dims = 300, 8, 4, 128, (16, 56, 56)
    c = (M, H, D, dims, 0, BF, 0)
    Q, K, qw, kw, pos = qk_inputs(c, Hk)
    dQo, dKo = rnd(70, M, H, D, dtype=BF), rnd(71, M, Hk, D, dtype=BF)
    side = torch.cuda.Stream()
    eager = lambda: (*rtl.rtl_qk_norm_rope(Q, K, qw, kw, pos, dims), rtl.rtl_rope_axes(Q, pos, dims),
                     *rtl.rtl_qk_norm_rope_backward(Q, K, qw, kw, pos, dims, dQo, dKo))
    first = eager()
    side.wait_stream(torch.cuda.current_stream())
    on_side = rtl.rtl_qk_norm_rope(Q, K, qw, kw, pos, dims, stream=side)
    side.synchronize()
    assert torch.equal(on_side[0], first[0]) and torch.equal(on_side[1], first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = eager()
    for k in range(3):
        Q.copy_(rnd(80 + k, M, H, D, dtype=BF))
        dKo.copy_(rnd(90 + k, M, Hk, D, dtype=BF))
        want = eager()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_python_refusals():
    """Tensors that do not go together are refused before the call."""
    Q, w, pos = rnd(1, 6, 2, 64, dtype=BF), rnd(2, 64, dtype=BF), positions(3, 6, 2)
    ok = dict(Q=Q, K=Q.clone(), qw=w, kw=w, pos=pos, axis_dims=(32, 32))
    for bad, err in ((dict(K=Q.float()), TypeError), (dict(K=Q[:5]), ValueError), (dict(qw=w.float()), TypeError),
                     (dict(kw=w[:32]), ValueError), (dict(pos=pos[:, :1]), ValueError), (dict(pos=pos.double()), TypeError),
                     (dict(pos=positions(3, 6, 4)[:, ::2]), ValueError), (dict(qw=w.cpu()), ValueError),
                     (dict(Q=Q[..., ::2]), ValueError), (dict(axis_dims=(32, -32)), ValueError),
                     (dict(Qo=Q[:, :1]), ValueError), (dict(Q=Q.half()), TypeError)):
        with pytest.raises(err):
            rtl.rtl_qk_norm_rope(**{**ok, **bad})
    with pytest.raises(rtl.RtlError):  # no tokens
        rtl.rtl_rope_axes(Q[:0], pos[:0], (32, 32))
    with pytest.raises(rtl.RtlError):  # one buffer for both outputs
        rtl.rtl_qk_norm_rope(**ok, Qo=ok["Q"], Ko=ok["Q"])
