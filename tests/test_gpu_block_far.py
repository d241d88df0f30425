"""The rotary, head-norm and gated-block operators on tensors whose offsets pass 2^31 elements or
2^32 bytes: the rows at both ends against the definitions in 64 bits."""
import pytest
import torch

import _block as B

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
BF = torch.bfloat16
FAR = 2 ** 31 + 64  # elements


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def rnd(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def ends(t, n=48):
    return torch.cat([t[:n], t[-n:]])


def far(M, H, D, way):
    """[M,H,D] whose tokens, or heads, lie FAR elements apart."""
    row, head = (FAR, D) if way == "tokens" else (D, FAR)
    buf = torch.empty((M - 1) * row + (H - 1) * head + D, dtype=BF, device="cuda")
    return buf.as_strided((M, H, D), (row, head, 1))


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("way", ("tokens", "heads"))
def test_strides(way):
    M, H, D, dims = 3, 3, 64, (16, 40)
    q, k, dq, dk = (rnd(i, M, H, D) for i in range(4))
    w, pos = rnd(5, D), torch.rand(M, 2, device="cuda") * 100
    Q, Y = far(M, H, D, way), far(M, H, D, way)
    Q.copy_(q)
    assert torch.equal(rtl.rtl_rope_axes(Q, pos, dims, Y=Y), rtl.rtl_rope_axes(q, pos, dims))
    same(rtl.rtl_qk_norm_rope(Q, k, w, None, pos, dims, Qo=Y), rtl.rtl_qk_norm_rope(q, k, w, None, pos, dims))
    Y.copy_(dq)
    want = rtl.rtl_qk_norm_rope_backward(q, k, w, None, pos, dims, dq, dk)
    same(rtl.rtl_qk_norm_rope_backward(Q, k, w, None, pos, dims, Y, dk, dQ=Q), want)


def test_many_tokens():
    M, H, D, dims = 270_000, 64, 128, (16, 56, 56)  # 2.2e9 elements
    Q, w = rnd(1, M, H, D), rnd(2, D)
    pos = torch.rand(M, 3, device="cuda") * 1000
    x, p = B.f64(ends(Q)), B.f64(ends(pos))
    phi, wf = B.angles(p, dims, 10000.0), B.f64(w)
    Y = rtl.rtl_rope_axes(Q, pos, dims)
    B.check(ends(Y), B.rotate(x, phi, 0), B.TURN * B.pair_sum(x, phi.shape[1], 0), BF, "rope")
    rtl.rtl_qk_norm_rope(Q, None, w, None, pos, dims, Qo=Y)
    B.check(ends(Y), *B.qk_forward(x, wf, phi, 0, 1e-6), BF, "Qo")
    # a gradient of zeros but for the two ends
    Y.zero_()
    Y[:48].copy_(rnd(3, 48, H, D))
    Y[-48:].copy_(rnd(4, 48, H, D))
    dy = B.f64(ends(Y))
    dQ, _, dqw, _ = rtl.rtl_qk_norm_rope_backward(Q, None, w, None, pos, dims, Y, None, dQ=Y)
    dx, dw, bx, bw = B.qk_backward(x, wf, phi, 0, 1e-6, dy)
    B.check(ends(dQ), dx, bx, BF, "dQ")
    B.check(dqw, dw, bw, torch.float32, "dqw")
    assert not dQ[48:-48].any()


# M, K, H: X past 2^32 bytes; Y, G, U and both P halves; the weights with few rows; rows of X and
# of the weights as far apart as they may lie, for the streamed and the tiled kernels
GLU = [(1_020_000, 2112, 96), (1_020_000, 64, 2112), (3, 64, 34_000_000), (5, 4_194_240, 300), (70, 4_194_240, 520)]


def label(c):
    return "x".join(map(str, c))


def product(a, b):
    """a b^T in 64 bits, on the GPU, a few million columns at a time."""
    n = 1 << 19
    return sum(a[:, i:i + n].double() @ b[:, i:i + n].double().t() for i in range(0, a.shape[1], n)).cpu().numpy()


@pytest.mark.parametrize("c", GLU, ids=label)
def test_glu(c):
    M, K, H = c
    # -1, 0 and 1, the weights scaled by a power of two: every sum is exact
    X, Wg, Wu = (rnd(i, *s).clamp_(-1, 1).round_() for i, s in enumerate(((M, K), (H, K), (H, K))))
    for w in (Wg, Wu):
        w *= 2.0 ** -round(K.bit_length() / 2)
    G, U = torch.empty(M, H, dtype=BF, device="cuda"), torch.empty(M, H, dtype=BF, device="cuda")
    Y = rtl.rtl_glu_fused(X, Wg, Wu, G=G, U=U)
    rows = (lambda t: t) if M <= 96 else ends
    cols = (lambda t: t) if H <= 2112 else (lambda t: ends(t, 1000))
    x, wg, wu = rows(X), cols(Wg), cols(Wu)
    for out, w, name in ((G, wg, "G"), (U, wu, "U")):
        want = product(x, w)
        B.check(cols(rows(out).t()).t(), want, 0 * want, BF, name)
    g, u = B.f64(cols(rows(G).t()).t()), B.f64(cols(rows(U).t()).t())
    v, _ = B.act(g, 0)
    # Y from the accumulators, which G and U hold within their rounding, 2^-8: SiLU's slope is below 1.13
    # and its value below |g|
    off = 2.0 ** -8 * (1.13 * abs(g) * abs(u) + abs(v) * abs(u)) * 1.02 + B.act_bound(g) * abs(u)
    B.check(cols(rows(Y).t()).t(), v * u, off, BF, "Y")


@pytest.mark.parametrize("c", [(1_020_000, 2112, 96), (1_020_000, 64, 2112), (70, 4_194_240, 520)], ids=label)
def test_glu_backward(c):
    M, K, H = c
    X, Wg, Wu = rnd(1, M, K), rnd(2, H, K, std=K ** -0.5), rnd(3, H, K, std=K ** -0.5)
    G, U, dY = rnd(4, M, H, std=1.5), rnd(5, M, H), torch.zeros(M, H, dtype=BF, device="cuda")
    n = min(M // 2, 48)  # a gradient of zeros but for the two ends
    dY[:n].copy_(rnd(6, n, H, std=0.1))
    dY[-n:].copy_(rnd(7, n, H, std=0.1))
    dX, dWg, dWu = rtl.rtl_glu_backward(X, Wg, Wu, G, U, dY)
    cols = (lambda t: t) if K <= 2112 else (lambda t: torch.cat([t[:, :500], t[:, -500:]], dim=1))
    x, wg, wu = cols(ends(X, n)), cols(Wg), cols(Wu)
    want, bounds = B.glu_backward(*map(B.f64, (x, wg, wu, ends(G, n), ends(U, n), ends(dY, n))), 0, elements=M * H)
    for out, w, b, name in zip((cols(ends(dX, n)), cols(dWg), cols(dWu)), want, bounds, ("dX", "dWg", "dWu")):
        B.check(out, w, b, BF, name)
    assert not dX[n:M - n].any()
