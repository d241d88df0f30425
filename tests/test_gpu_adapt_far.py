"""The layer norm, the adapters and the AdamW step on tensors whose offsets pass 2^31 elements or 2^32 bytes, and
on batches past the shares that the chip holds at once: against the same calls on tensors that lie close, which
other tests hold against the definitions, and against the definitions in 64 bits."""
import pytest
import torch

import _adapt as A
from test_gpu_adapters import Case

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
FAR = 2 ** 31 + 64  # elements


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def far(t):
    """t's values in rows that lie FAR elements apart."""
    M, D = t.shape
    return torch.empty((M - 1) * FAR + D, dtype=t.dtype, device="cuda").as_strided((M, D), (FAR, 1)).copy_(t)


def same(got, want):
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("D", (264, 77))
def test_norm_rows_far_apart(D):
    M = 3
    X, dY, w, scale, shift = A.rnd(1, M, D), A.rnd(2, M, D), A.rnd(3, D), A.rnd(4, 2, D), A.rnd(5, 2, D)
    at, stats = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"), torch.empty(M, 2, device="cuda")
    Y = rtl.rtl_layer_norm(X, w, None, scale, shift, at, stats=stats)
    want = rtl.rtl_layer_norm_backward(X, stats, dY, w, None, scale, at)
    x, s, h = far(X), far(scale), far(shift)
    y = rtl.rtl_layer_norm(x, w, None, s, h, at, Y=far(torch.zeros_like(X)))
    same([y, *rtl.rtl_layer_norm_backward(x, stats, far(dY), w, None, s, at, dX=y)], [y, *want])
    assert torch.equal(rtl.rtl_layer_norm(x, w, None, s, h, at, Y=y), Y)


def test_norm_of_many_elements():
    """More than 2^31: rows that repeat every 1024, whole chunks of rows, have results that repeat, and sums of as many
    times as they do."""
    P, D, times = 1024, 5120, 420
    x, dy, scale, shift = A.rnd(1, P, D, mean=0.2), A.rnd(2, P, D, std=0.1), A.rnd(3, 3, D, std=0.3), A.rnd(4, 3, D)
    X, dY, M = x.repeat(times, 1), dy.repeat(times, 1), P * times
    assert X.numel() > 2 ** 31
    cut = torch.tensor([0, P, (times - 2) * P, M], dtype=torch.int32, device="cuda")
    stats, few = torch.empty(M, 2, device="cuda"), torch.tensor([0, P], dtype=torch.int32, device="cuda")
    Y = rtl.rtl_layer_norm(X, None, None, scale, shift, cut, stats=stats)
    dX, _, _, dscale, dshift = rtl.rtl_layer_norm_backward(X, stats, dY, None, None, scale, cut)
    for g, lo, hi in ((0, 0, 1), (1, 1, times - 2), (2, times - 2, times)):
        own = torch.empty(P, 2, device="cuda")
        y = rtl.rtl_layer_norm(x, None, None, scale[g:g + 1], shift[g:g + 1], few, stats=own)
        back = rtl.rtl_layer_norm_backward(x, own, dy, None, None, scale[g:g + 1], few)
        for k in range(lo, hi):
            rows = slice(k * P, (k + 1) * P)
            same((Y[rows], stats[rows], dX[rows]), (y, own, back[0]))
        # 16 or 32 rows of a sum in fp32 and the rest in double; the sums round once where they leave
        n = (x.double() - own[:, :1].double()) * own[:, 1:].double()
        for got, terms in ((dscale[g], dy.double() * n), (dshift[g], dy.double())):
            off = (got.double() - (hi - lo) * terms.sum(0)).abs()
            assert bool((off <= 36 * 2.0 ** -24 * (hi - lo) * terms.abs().sum(0)).all())


def test_adapters_rows_far_apart():
    M, K, N, R, n = 3, 72, 136, 16, 2
    X, dY, Y0, dX0 = A.rnd(1, M, K), A.rnd(2, M, N), A.rnd(3, M, N), A.rnd(4, M, K)
    LA, LB = A.rnd(5, n, N, R), A.rnd(6, n, R, K)
    plan = rtl.rtl_adapters_plan(torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda"), n)
    T = torch.empty(M, R, device="cuda")
    want = [rtl.rtl_adapters(X, LA, LB, plan, Y0=Y0, T=T), *rtl.rtl_adapters_backward(X, LA, LB, plan, T, dY, dX0=dX0)]
    x, y = far(X), far(Y0)
    t = torch.empty_like(T)
    got = [rtl.rtl_adapters(x, LA, LB, plan, Y0=y, Y=y, T=t)]
    same(got + [t], [want[0], T])
    y.copy_(dY)
    dx = far(dX0)
    same(rtl.rtl_adapters_backward(x, LA, LB, plan, T, y, dX0=dx, dX=dx), want[1:])


def test_adapters_with_far_factors():
    """The last of 32 adapters, whose factors begin past 2^30 elements and end past 2^31."""
    M, N, K, R, n = 5, 2 ** 22, 64, 24, 32
    X, dY = A.rnd(1, M, K), torch.randn(M, N, device="cuda").to(BF)
    la, lb = (torch.randn(1, N, R, device="cuda") * R ** -0.5).to(BF), A.rnd(4, 1, R, K, std=K ** -0.5)
    plan = [rtl.rtl_adapters_plan(torch.full((M,), a, dtype=torch.int32, device="cuda"), k) for a, k in ((0, 1), (n - 1, n))]
    T = torch.empty(M, R, device="cuda")
    Y = rtl.rtl_adapters(X, la, lb, plan[0], T=T)
    want = rtl.rtl_adapters_backward(X, la, lb, plan[0], T, dY)
    LA, LB = torch.zeros(n, N, R, dtype=BF, device="cuda"), torch.zeros(n, R, K, dtype=BF, device="cuda")
    LA[-1], LB[-1] = la[0], lb[0]
    assert LA.numel() > 2 ** 31
    t = torch.empty_like(T)
    same((rtl.rtl_adapters(X, LA, LB, plan[1], T=t), t), (Y, T))
    dX, dLA, dLB = rtl.rtl_adapters_backward(X, LA, LB, plan[1], T, dY)
    same((dX, dLA[-1], dLB[-1]), (want[0], want[1][0], want[2][0]))
    assert not bool(dLA[:-1].any()) and not bool(dLB[:-1].any())


@pytest.mark.parametrize("eight", (False, True))
def test_step_of_a_tensor_of_many_elements(eight):
    """One tensor of more than 2^31 elements: what repeats every 2^20 stays alike, and its end is a short tensor's."""
    P, end = 2 ** 20, 300
    n = 2 ** 31 + P + end
    g, p = A.rnd(1, P, std=1e-3), A.rnd(2, P, std=0.02, dtype=F32)
    how = dict(step=1, lr=1e-3, weight_decay=0.1)

    def tensors(n):
        state = E4 if eight else F32
        times = (n + P - 1) // P
        master = p.repeat(times)[:n]
        scales = [torch.zeros((n + 255) // 256, device="cuda") for _ in range(2)] if eight else [None] * 2
        m, v = torch.zeros(n, dtype=state, device="cuda"), torch.zeros(n, dtype=state, device="cuda")
        d = dict(params=[master.to(BF)], grads=[g.repeat(times)[:n]], m=[m], v=[v], masters=[master])
        return {**d, **(dict(m_scales=[scales[0]], v_scales=[scales[1]]) if eight else {})}

    few, many = tensors(P + end), tensors(n)
    for d in (few, many):
        rtl.rtl_adamw(rtl.rtl_adamw_tensors(**d), **how)
    for name in few:
        a, b = (d[name][0] for d in (few, many))
        if a.dtype is E4:
            a, b = a.view(torch.uint8), b.view(torch.uint8)
        whole = P // 256 if name.endswith("scales") else P
        assert torch.equal(b[-(a.numel() - whole):], a[whole:]), name
        rows = b[:b.numel() // whole * whole].view(-1, whole)
        assert all(torch.equal(row, a[:whole]) for row in rows[::61]) and torch.equal(rows[-1], a[:whole]), name


@pytest.mark.parametrize("R", (8, 64, 128))
@pytest.mark.parametrize("kind", ("mixed", "runs"))
def test_shares_of_more_work_than_the_chip_holds(R, kind):
    """Tiles by steps past four times the workgroups that run at once: shares that begin and end inside tiles."""
    c = Case(6000, 2056, 2056, R, 3, kind)
    c.forward(f"{R} {kind}")
    c.backward(f"{R} {kind}")
