"""GPU tests of the low-rank adapters of many requests and their gradient against their definitions in 64
bits: one row to many, adapters with no rows, one, and several tiles and shares of them, rows without an
adapter, odd sizes, strides, and what lies around the outputs."""
import numpy as np
import pytest
import torch

import _adapt as A
import _block as B
from _gpu import Guarded

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
BF, F32 = torch.bfloat16, torch.float32


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ids_of(kind, M, n, seed=0):
    """Each row's adapter: `kind` says how the rows of n adapters lie."""
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full(M, n - 1)
    if kind == "none":
        return np.full(M, -1)
    if kind == "mixed":  # and some without, in both ways of saying so
        return rng.choice(np.r_[np.arange(n), -1, n, -2 ** 31, 2 ** 31 - 1], M)
    if kind == "runs":
        return np.sort(rng.integers(-1, n, M))
    if kind == "few":  # the first and the last adapter, one row of the latter
        i = np.zeros(M, int)
        i[M // 2] = n - 1
        return i
    raise KeyError(kind)


class Case:
    def __init__(self, M, K, N, R, n, kind, seed=1, alpha=True, wide=False):
        self.ids = ids_of(kind, M, n, seed)
        self.X = A.rnd(seed, M, 2 * K if wide else K)[:, :K]
        self.LA, self.LB = A.rnd(seed + 1, n, N, R, std=R ** -0.5), A.rnd(seed + 2, n, R, K, std=K ** -0.5)
        self.alpha = torch.linspace(0.5, -1.5, n, device="cuda") if alpha else None
        self.Y0 = A.rnd(seed + 3, M, 3 * N if wide else N)[:, -N:]
        self.dY, self.dX0 = A.rnd(seed + 4, M, N, std=0.1), A.rnd(seed + 5, M, K, std=0.1)
        self.plan = rtl.rtl_adapters_plan(torch.from_numpy(self.ids.astype(np.int32)).cuda(), n)
        self.M, self.K, self.N, self.R, self.n = M, K, N, R, n

    def host(self):
        a = np.ones(self.n) if self.alpha is None else B.f64(self.alpha)
        return B.f64(self.X), B.f64(self.LA), B.f64(self.LB), a

    def forward(self, name):
        x, la, lb, a = self.host()
        Y, T = Guarded((self.M, self.N), BF), Guarded((self.M, self.R), F32)
        rtl.rtl_adapters(self.X, self.LA, self.LB, self.plan, self.alpha, Y0=self.Y0, Y=Y.t, T=T.t)
        y, t, by, bt = A.adapters_forward(x, la, lb, a, self.ids, B.f64(self.Y0))
        B.check(T.t, t, bt, F32, name + " T")
        B.check(Y.t, y, by, BF, name + " Y")
        bare = torch.from_numpy((self.ids < 0) | (self.ids >= self.n)).cuda()
        assert torch.equal(Y.t[bare], self.Y0[bare]) and not bool(T.t[bare].any())
        Y.check(name)
        T.check(name)
        return Y.t, T.t

    def backward(self, name):
        x, la, lb, a = self.host()
        T = torch.from_numpy(A.adapters_forward(x, la, lb, a, self.ids, B.f64(self.Y0))[1]).float().cuda()
        out = Guarded((self.M, self.K), BF), Guarded(self.LA.shape, F32), Guarded(self.LB.shape, F32)
        got = rtl.rtl_adapters_backward(self.X, self.LA, self.LB, self.plan, T, self.dY, self.alpha, dX0=self.dX0,
                                        dX=out[0].t, dLA=out[1].t, dLB=out[2].t)
        want, bounds = A.adapters_backward(x, la, lb, a, self.ids, B.f64(T), B.f64(self.dY), B.f64(self.dX0))
        for o, t, w, b, what, dt in zip(out, got, want, bounds, ("dX", "dLA", "dLB"), (BF, F32, F32)):
            B.check(t, w, b, dt, f"{name} {what}")
            o.check(name)
        return got


# (M, K, N, R, adapters): a row, a tile and one more, K and N that end inside steps, strips and column tiles,
# every class of ranks; the last ones split K, and the rows into shares
SIZES = [(1, 8, 8, 8, 1), (1, 5120, 72, 64, 3), (2, 64, 40, 16, 4), (5, 72, 1000, 24, 2), (63, 136, 264, 32, 3),
         (64, 200, 128, 40, 3), (65, 328, 72, 64, 2), (129, 1032, 520, 72, 5), (200, 512, 1032, 96, 2), (300, 264, 2056, 128, 3),
         (700, 2056, 136, 8, 70), (1100, 640, 328, 112, 2), (2500, 264, 200, 16, 1)]


@pytest.mark.parametrize("M,K,N,R,n", SIZES)
@pytest.mark.parametrize("kind", ("one", "mixed", "runs"))
def test_forward(M, K, N, R, n, kind):
    Case(M, K, N, R, n, kind).forward(f"{M} x {K} -> {N}, {R}, {kind}")


@pytest.mark.parametrize("M,K,N,R,n", SIZES)
@pytest.mark.parametrize("kind", ("one", "mixed", "runs"))
def test_backward(M, K, N, R, n, kind):
    Case(M, K, N, R, n, kind).backward(f"{M} x {K} -> {N}, {R}, {kind}")


@pytest.mark.parametrize("M", (1, 64, 130, 1000))
@pytest.mark.parametrize("kind", ("none", "few"))
def test_adapters_without_rows(M, kind):
    c = Case(M, 136, 264, 16, 6, kind)
    c.forward(kind)
    _, dla, dlb = c.backward(kind)
    used = {int(i) for i in c.ids if i >= 0}
    for a in range(6):
        assert a in used or not (bool(dla[a].any()) or bool(dlb[a].any()))


def test_many_adapters():
    """A row each of 300, the plan's tables past one workgroup's threads; and the largest number."""
    c = Case(300, 72, 136, 8, 300, "mixed")
    c.ids = np.random.default_rng(5).permutation(300)
    c.plan = rtl.rtl_adapters_plan(torch.from_numpy(c.ids.astype(np.int32)).cuda(), 300)
    c.forward("300")
    c.backward("300")
    Case(700, 8, 8, 8, 4096, "mixed").forward("4096")


def test_plan_keeps_the_order_of_rows():
    """The plan's rows sorted by adapter, in their order, those without one last (its layout is not public:
    the last M words are the order)."""
    for M, n, kind in ((1, 1, "one"), (1000, 7, "mixed"), (5000, 3, "runs"), (70000, 2, "mixed"), (257, 300, "mixed")):
        ids = ids_of(kind, M, n, 3)
        plan = rtl.rtl_adapters_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), n)
        key = np.where((ids < 0) | (ids >= n), n, ids)
        assert np.array_equal(plan.view(torch.int32)[-M:].cpu().numpy(), np.argsort(key, kind="stable"))


def test_strides_in_place_and_without_a_projection():
    c = Case(150, 264, 200, 32, 3, "mixed", wide=True)
    Y, T = c.forward("wide")
    wide = A.rnd(4, 150, 600)  # the same values that Case drew
    y = wide[:, 400:]
    assert torch.equal(y, c.Y0)
    before = wide[:, :400].clone()
    got = rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, Y0=y, Y=y)
    assert got is y and torch.equal(y, Y) and torch.equal(wide[:, :400], before)
    none = rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha)
    zero = rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, Y0=torch.zeros(150, 200, dtype=BF, device="cuda"))
    assert torch.equal(none, zero)
    plain = Case(150, 264, 200, 32, 3, "mixed", alpha=False)
    plain.forward("no alpha")
    plain.backward("no alpha")
    # gradients: dX in its dX0, without one, and each output left out
    want = c.backward("wide")
    d = c.dX0.clone()
    got = rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha, dX0=d, dX=d)
    again = rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha, dX0=c.dX0)
    assert got[0] is d and all(torch.equal(a, b) for a, b in zip(got, again))
    assert torch.equal(d, want[0])
    only = rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha, dX0=c.dX0, need_dw=False)
    assert only[1:] == (None, None) and torch.equal(only[0], d)
    only = rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha, need_dx=False)
    assert only[0] is None and torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])
    none = rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha, need_dw=False)
    zero = rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha, dX0=torch.zeros_like(d), need_dw=False)
    assert torch.equal(none[0], zero[0])


def test_infinities_and_nan_stay_with_their_rows():
    """A bad row of X and dY, a bad factor of one adapter, and rows without an adapter that hold NaN."""
    c = Case(140, 136, 72, 24, 3, "runs")
    bare = torch.from_numpy(c.ids < 0).cuda()
    assert bool(bare.any())
    c.X[bare] = float("nan")
    c.dY[bare] = float("nan")
    c.forward("bare")
    want = c.backward("bare")
    T = torch.zeros(140, 24, device="cuda")
    Y = rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, T=T)
    row = int(np.nonzero(c.ids == 1)[0][3])
    other = torch.from_numpy(c.ids != 1).cuda()
    x, dy = c.X.clone(), c.dY.clone()
    x[row, 5] = float("inf")
    dy[row, 6] = float("inf")
    y = rtl.rtl_adapters(x, c.LA, c.LB, c.plan, c.alpha)
    rest = torch.arange(140, device="cuda") != row
    assert torch.equal(y[rest], Y[rest])
    # T is infinite of either sign there, and Y what the definition makes of that
    with np.errstate(invalid="ignore"):
        want_row = float(c.alpha[1]) * ((B.f64(x)[row] @ B.f64(c.LB)[1].T) @ B.f64(c.LA)[1].T)
    assert np.array_equal(np.isnan(B.f64(y[row])), np.isnan(want_row)) and not np.isfinite(want_row).any()
    t = T.clone()
    t[bare] = float("nan")
    got = rtl.rtl_adapters_backward(x, c.LA, c.LB, c.plan, t, dy, c.alpha, dX0=c.dX0)
    base = rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha, dX0=c.dX0)
    assert torch.equal(got[0][rest], base[0][rest])
    for a, b in zip(got[1:], base[1:]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    # of the adapter's own gradients, only the columns that meet them
    cols = torch.arange(72, device="cuda") != 6
    assert torch.equal(got[1][1][cols], base[1][1][cols]) and bool(torch.isinf(got[1][1][6]).all())
    la = c.LA.clone()
    la[1, 7, 3] = float("inf")
    y = rtl.rtl_adapters(c.X, la, c.LB, c.plan, c.alpha)
    assert torch.equal(y[other], Y[other]) and bool(torch.isinf(y[~other][:, 7]).all())
    assert torch.equal(y[~other][:, 8:], Y[~other][:, 8:])


def test_large_and_small_values():
    """T at both ends of its range: values past bf16's largest keep their digits in two parts."""
    for size in (2.0 ** 60, 2.0 ** -60):
        c = Case(70, 64, 72, 16, 2, "runs")
        c.X = (c.X.float() * size).to(BF)
        c.LA = (c.LA.float() / size).to(BF)
        c.Y0 = torch.zeros_like(c.Y0)
        c.forward(f"{size}")
        c.backward(f"{size}")


def test_gradient_against_differences():
    c = Case(40, 64, 72, 16, 3, "mixed")
    x, la, lb, a = c.host()
    dy = B.f64(c.dY)
    T = torch.empty(40, 16, device="cuda")
    rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, T=T)
    got = rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha)
    rng = np.random.default_rng(2)
    for k, name in enumerate(("X", "LA", "LB")):
        d = rng.standard_normal((x, la, lb)[k].shape)

        def value(s):
            moved = [v + s * d if i == k else v for i, v in enumerate((x, la, lb))]
            return (A.adapters_forward(moved[0], moved[1], moved[2], a, c.ids, np.zeros((40, 72)))[0] * dy).sum()

        slope = (value(0.5) - value(-0.5))  # linear in each argument: exact
        terms = B.f64(got[k]) * d
        # every term within a bf16 rounding, T within its own
        assert abs(slope - terms.sum()) <= 2.0 ** -8 * np.abs(terms).sum(), (name, slope, terms.sum())


def test_captured_and_replayed_on_other_batches():
    """Plan, forward and backward in one graph; two graphs with one workspace, replayed one after the other."""
    M, K, N, R, n = 260, 264, 328, 32, 4
    c = Case(M, K, N, R, n, "mixed")
    ids = torch.from_numpy(np.clip(c.ids, -1, n).astype(np.int32)).cuda()
    ws = torch.empty(max(rtl.rtl_adapters_workspace_bytes(M, N, K, R, n), rtl.rtl_adapters_backward_workspace_bytes(M, N, K, R, n)),
                     dtype=torch.uint8, device="cuda")
    T = torch.empty(M, R, device="cuda")

    def forward():
        rtl.rtl_adapters_plan(ids, n, plan=c.plan)
        return rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, Y0=c.Y0, T=T, workspace=ws)

    def backward():
        return rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha, dX0=c.dX0, workspace=ws)

    forward(), backward()
    graphs, held = [], []
    for f in (forward, backward):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(f())
    for k in range(4):
        c.X.copy_(A.rnd(70 + k, M, K))
        c.dY.copy_(A.rnd(80 + k, M, N, std=0.1))
        ids.copy_(torch.from_numpy(ids_of(("runs", "one", "few", "mixed")[k], M, n, k).clip(-1, n).astype(np.int32)))
        want = forward(), backward()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], want[0]) and all(torch.equal(a, b) for a, b in zip(held[1], want[1]))


def test_same_result_on_every_run():
    c = Case(900, 640, 520, 64, 3, "mixed")
    Y, T = c.forward("a")
    got = [(rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, Y0=c.Y0),
            *rtl.rtl_adapters_backward(c.X, c.LA, c.LB, c.plan, T, c.dY, c.alpha)) for _ in range(3)]
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(g, got[0]))


def test_plan_of_garbage_stays_in_bounds():
    """A plan that was never made: results mean nothing, but nothing outside the outputs changes."""
    c = Case(200, 136, 264, 24, 3, "mixed")
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        words = torch.randint(-2 ** 31, 2 ** 31 - 1, (c.plan.numel() // 4,), generator=g).to(torch.int32).cuda()
        if seed == 2:
            words = words.abs() % 300  # numbers that could be of a larger batch
        plan = words.view(torch.uint8)
        Y, T = Guarded((200, 264), BF), Guarded((200, 24), F32)
        rtl.rtl_adapters(c.X, c.LA, c.LB, plan, c.alpha, Y0=c.Y0, Y=Y.t, T=T.t)
        out = Guarded((200, 136), BF), Guarded(c.LA.shape, F32), Guarded(c.LB.shape, F32)
        rtl.rtl_adapters_backward(c.X, c.LA, c.LB, plan, T.t, c.dY, c.alpha, dX=out[0].t, dLA=out[1].t, dLB=out[2].t)
        for o in (Y, T, *out):
            o.check(f"garbage {seed}")


@pytest.mark.parametrize("M", (1, 2, 15, 16, 17))
@pytest.mark.parametrize("R", (8, 40, 72, 128))
@pytest.mark.parametrize("kind", ("one", "mixed", "none", "few"))
def test_few_rows_in_place(M, R, kind):
    """Single rows of requests, Y in Y0's place: T of every row, zeros without an adapter, whose Y is not touched."""
    K, N, n = 328, 1032, 5
    c = Case(M, K, N, R, n, kind, seed=60 + M)
    x, la, lb, a = c.host()
    y, t, by, bt = A.adapters_forward(x, la, lb, a, c.ids, B.f64(c.Y0))
    Y, T = Guarded((M, N), BF), Guarded((M, R), F32)
    Y.t.copy_(c.Y0)
    rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, Y0=Y.t, Y=Y.t, T=T.t)
    B.check(T.t, t, bt, F32, f"{M} {R} {kind} T")
    B.check(Y.t, y, by, BF, f"{M} {R} {kind} Y")
    bare = torch.from_numpy((c.ids < 0) | (c.ids >= n)).cuda()
    assert torch.equal(Y.t[bare], c.Y0[bare]) and not bool(T.t[bare].any())
    Y.check(kind)
    T.check(kind)
    # the same without T, into a tensor of its own and on top of zeros
    assert torch.equal(rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, Y0=c.Y0), Y.t)
    zeros = torch.zeros_like(c.Y0)
    assert torch.equal(rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha), rtl.rtl_adapters(c.X, c.LA, c.LB, c.plan, c.alpha, Y0=zeros))
