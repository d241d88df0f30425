"""The layer norm, the adapters of a batch's requests and the optimizer's step together, as the layer policy's
objects and the trained fit call them: the norm with each request's scale and shift, a sparse projection with
adapters beside it, both gradients, a step of the factors.  Each stage is held against its definition in 64 bits
on the stage's own input; the whole step, captured and replayed on other batches, against its eager run."""
import threading

import numpy as np
import pytest
import torch

import _adapt as A
import _block as B
import oracle
from _gpu import check_y, f64, to_host

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
from activation_sparse_gemm_amd import calib, policy  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
HOW = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Step:
    """Requests of a batch, each with its scale, shift and one of three adapters or none."""

    def __init__(self, M, K=256, N=320, R=24, A_=3, eight=False):
        self.M = M
        self.norm = policy.AdaptiveNorm(A.rnd(1, K, std=0.2, mean=1.0), A.rnd(2, K, std=0.2))
        shared = policy.Linear(A.rnd(3, N, K, std=K ** -0.5), A.rnd(4, N, 32, std=0.02), A.rnd(5, 32, K, std=0.02))
        self.masters = [A.rnd(6, A_, N, R, std=R ** -0.5, dtype=F32), A.rnd(7, A_, R, K, std=K ** -0.5, dtype=F32)]
        self.lin = policy.AdaptedLinear(shared, *(t.to(BF) for t in self.masters), torch.tensor([0.5, -1.0, 2.0], device="cuda"))
        self.grads = [torch.zeros_like(t) for t in self.masters]
        states = [torch.zeros_like(t, dtype=torch.float8_e4m3fn if eight else F32) for t in self.masters * 2]
        scales = [torch.zeros((t.numel() + 255) // 256, device="cuda") for t in self.masters * 2] if eight else None
        self.state = dict(masters=self.masters, m=states[:2], v=states[2:],
                          **(dict(m_scales=scales[:2], v_scales=scales[2:]) if eight else {}))
        self.tensors = rtl.rtl_adamw_tensors([self.lin.LA, self.lin.LB], self.grads, **self.state)
        self.count = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.ids = torch.zeros(M, dtype=torch.int32, device="cuda")
        self.groups = torch.zeros(5, dtype=torch.int32, device="cuda")
        self.X, self.dY = (torch.zeros(M, n, dtype=BF, device="cuda") for n in (K, N))
        self.parts = torch.zeros(4, 2 * K, dtype=BF, device="cuda")

    def batch(self, seed):
        M, K = self.X.shape
        rng = np.random.default_rng(seed)
        at = np.sort(rng.integers(0, M + 1, 3))
        self.offsets = np.r_[0, at, M].astype(np.int32)
        self.which = rng.choice([-1, 0, 1, 2], 4)
        self.host_ids = np.repeat(self.which, np.diff(self.offsets)).astype(np.int32)
        self.groups.copy_(torch.from_numpy(self.offsets))
        self.ids.copy_(torch.from_numpy(self.host_ids))
        self.X.copy_(A.rnd(seed + 1, M, K, mean=0.2))
        self.parts.copy_(A.rnd(seed + 2, 4, 2 * K, std=0.3))
        self.dY.copy_(A.rnd(seed + 3, *self.dY.shape, std=0.1))

    def __call__(self):
        K = self.X.shape[1]
        self.plan = self.lin.plan(self.ids, getattr(self, "plan", None))
        scale, shift = self.parts[:, K:], self.parts[:, :K]
        stats, T = torch.empty(self.M, 2, device="cuda"), torch.empty(self.M, self.lin.LB.shape[1], device="cuda")
        h = self.norm(self.X, scale, shift, self.groups, stats=stats)
        y = self.lin(h, self.plan, T=T)
        back = rtl.rtl_linear_dense_ref(self.dY, self.lin.linear.W.T.contiguous())  # straight through the selection
        dh, dLA, dLB = self.lin.backward(h, self.plan, T, self.dY, dX0=back)
        sums = self.norm.backward(self.X, stats, dh, scale, self.groups)
        self.grads[0].copy_(dLA)
        self.grads[1].copy_(dLB)
        self.count.add_(1)
        rtl.rtl_adamw(self.tensors, self.count, **HOW)
        return dict(h=h, y=y, stats=stats, T=T, back=back, dh=dh, dLA=dLA, dLB=dLB, dX=sums[0], dw=sums[1], db=sums[2],
                    dscale=sums[3], dshift=sums[4])


@pytest.mark.parametrize("M", (1, 7, 130, 500))
def test_stages(M):
    s = Step(M)
    s.batch(10 + M)
    LA, LB, masters = s.lin.LA.clone(), s.lin.LB.clone(), [to_host(t) for t in s.masters]
    r = s()
    K = s.X.shape[1]
    group = A.norm_rows(M, s.offsets)
    w, b, scale, shift = B.f64(s.norm.weight), B.f64(s.norm.bias), B.f64(s.parts[:, K:]), B.f64(s.parts[:, :K])
    y, st, by, bs = A.norm_forward(B.f64(s.X), w, b, scale, shift, group, float(np.float32(1e-6)))
    B.check(r["h"], y, by, BF, "norm")
    B.check(r["stats"], st, bs, F32, "stats")
    # the projection alone, then the adapters on top of what it gave
    shared = s.lin.linear
    y0 = rtl.rtl_linear_fused(r["h"], shared.W, shared.LA, shared.LB)
    want, _ = oracle.linear(to_host(r["h"]), to_host(shared.W), to_host(shared.LA), to_host(shared.LB))
    check_y(f64(to_host(y0), "bf16"), want, "bf16", "projection")
    alpha = B.f64(s.lin.alpha)
    y, t, by, bt = A.adapters_forward(B.f64(r["h"]), B.f64(LA), B.f64(LB), alpha, s.host_ids, B.f64(y0))
    B.check(r["y"], y, by, BF, "adapted")
    B.check(r["T"], t, bt, F32, "T")
    bare = s.ids < 0
    assert torch.equal(r["y"][bare], y0[bare])
    # back
    want, bounds = A.adapters_backward(B.f64(r["h"]), B.f64(LA), B.f64(LB), alpha, s.host_ids, B.f64(r["T"]), B.f64(s.dY),
                                       B.f64(r["back"]))
    for name, v, e in zip(("dh", "dLA", "dLB"), want, bounds):
        B.check(r[name], v, e, BF if name == "dh" else F32, name)
    dx, sums, bx, bounds = A.norm_backward(B.f64(s.X), B.f64(r["stats"]), w, b, scale, group, 4, B.f64(r["dh"]))
    B.check(r["dX"], dx, bx, BF, "dX")
    for name, key in (("dw", "dweight"), ("db", "dbias"), ("dscale", "dscale"), ("dshift", "dshift")):
        B.check(r[name], sums[key], bounds[key], F32, name)
    # the step, to the bit
    for i, p in enumerate(masters):
        zero = np.zeros(p.size, np.float32)
        want, m, v = A.adamw(p.reshape(-1), to_host(s.grads[i]).reshape(-1), zero, zero, 1, *HOW.values())
        assert np.array_equal(to_host(s.masters[i]).reshape(-1), want)
    assert torch.equal(s.lin.LA, s.masters[0].to(BF)) and torch.equal(s.lin.LB, s.masters[1].to(BF))


@pytest.mark.parametrize("eight", (False, True), ids=("f32", "e4m3"))
def test_step_captured_and_replayed(eight):
    """The whole step in a graph, its batches copied in between replays, with eager work and synchronizations."""
    M = 300
    one, two = Step(M, eight=eight), Step(M, eight=eight)
    one.batch(0)
    one()  # what a first call allocates and plans
    two.batch(0)
    two()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = one()
    for k in range(4):
        one.batch(40 + k)
        two.batch(40 + k)
        graph.replay()
        want = two()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(held[name], want[name]), (k, name)
        for a, b in zip(one.masters + one.state["m"] + one.state["v"], two.masters + two.state["m"] + two.state["v"]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


def test_two_streams_with_one_plan():
    """Two threads, each with its own stream and workspaces, on one plan and one pair of factors."""
    M, K, N, R = 700, 264, 520, 16
    LA, LB = A.rnd(1, 2, N, R, std=R ** -0.5), A.rnd(2, 2, R, K, std=K ** -0.5)
    plan = rtl.rtl_adapters_plan((torch.arange(M, device="cuda") % 3 - 1).int(), 2)
    X, Y0, dY = [A.rnd(5 + i, M, K) for i in range(2)], [A.rnd(7 + i, M, N) for i in range(2)], [A.rnd(9 + i, M, N) for i in range(2)]

    def calls(i, n=1, stream=None):
        for _ in range(n):
            T = torch.empty(M, R, device="cuda")
            Y = rtl.rtl_adapters(X[i], LA, LB, plan, Y0=Y0[i], T=T, stream=stream)
            got = rtl.rtl_adapters_backward(X[i], LA, LB, plan, T, dY[i], stream=stream)
        return Y, T, *got

    want = [calls(i) for i in range(2)]
    torch.cuda.synchronize()
    out, errors, start = [None] * 2, [], threading.Barrier(2)

    def worker(i):
        try:
            s = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(s):
                out[i] = calls(i, 20)
            s.synchronize()
        except Exception as e:
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for got, ref in zip(out, want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_two_graphs_on_one_workspace():
    """Two captured calls that share a workspace, replayed one after the other in both orders."""
    M, K, N, R = 200, 136, 264, 8
    LA, LB = A.rnd(1, 3, N, R, std=R ** -0.5), A.rnd(2, 3, R, K, std=K ** -0.5)
    plans = [rtl.rtl_adapters_plan((torch.arange(M, device="cuda") // d % 3).int(), 3) for d in (1, 50)]
    X, dY = A.rnd(3, M, K), A.rnd(4, M, N)
    T = torch.empty(M, R, device="cuda")
    want = []
    for p in plans:
        Y = rtl.rtl_adapters(X, LA, LB, p, T=T)
        want.append((Y, *rtl.rtl_adapters_backward(X, LA, LB, p, T, dY)))
    need = max(rtl.rtl_adapters_workspace_bytes(M, N, K, R, 3), rtl.rtl_adapters_backward_workspace_bytes(M, N, K, R, 3))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs, held = [], []
    for p in plans:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y = rtl.rtl_adapters(X, LA, LB, p, T=T, workspace=ws)
            held.append((Y, *rtl.rtl_adapters_backward(X, LA, LB, p, T, dY, workspace=ws)))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for i in order:
            ws.fill_(255)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held[i], want[i])), order


def test_calls_while_another_gpu_is_current(monkeypatch):
    """Each call makes its tensors' GPU the current one first (here the current device's number and the
    context that changes it stand in for a second GPU)."""
    M, K, N, R = 9, 64, 40, 8
    X, dY, w = A.rnd(1, M, K), A.rnd(2, M, N), A.rnd(3, K)
    LA, LB = A.rnd(4, 2, N, R), A.rnd(5, 2, R, K)
    ids = (torch.arange(M, device="cuda") % 2).int()
    p, T, stats = torch.zeros(10, device="cuda"), torch.empty(M, R, device="cuda"), torch.empty(M, 2, device="cuda")
    g, m, v = (torch.full_like(p, x) for x in (1.0, 0.0, 0.0))

    def calls():
        for t in (p, m, v):
            t.zero_()
        plan = rtl.rtl_adapters_plan(ids, 2)
        got = [rtl.rtl_adapters(X, LA, LB, plan, T=T), *rtl.rtl_adapters_backward(X, LA, LB, plan, T, dY),
               rtl.rtl_layer_norm(X, w, stats=stats), *rtl.rtl_layer_norm_backward(X, stats, X, w)]
        rtl.rtl_adamw(rtl.rtl_adamw_tensors([p], [g], [m], [v]), 1, 0.1)
        return [t.clone() for t in got + [p, m, v] if t is not None]

    want, here, entered = calls(), X.get_device(), []
    current = [here + 1]

    class There:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)
            current[0] = self.device

        def __exit__(self, *exc):
            current[0] = here + 1

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", There)
    got = calls()
    monkeypatch.undo()
    assert entered and set(entered) == {here} and len(entered) >= 6
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_of_the_fit():
    """Half the gradient of ||E - X (L_A L_B)^T||^2 against its formula, on the difference as it was rounded, and
    against differences of the objective in 64 bits."""
    M, K, N, R = 130, 72, 104, 16
    X, E, LA, LB = A.rnd(1, M, K), A.rnd(2, M, N), A.rnd(3, N, R, std=0.3), A.rnd(4, R, K, std=0.3)
    dLA, dLB = calib.lowrank_gradient(X, E, LA, LB)
    x, e, la, lb = map(B.f64, (X, E, LA, LB))
    off = x @ (la @ lb).T - e
    want = dict(dLA=off.T @ (x @ lb.T), dLB=(off @ la).T @ x)
    # the difference is rounded to bf16 (2^-8 of it at most, and a part of the sums behind it)
    slack = 2.0 ** -8 * np.abs(off) * 1.01 + 1e-5
    bound = dict(dLA=slack.T @ np.abs(x @ lb.T), dLB=(slack @ np.abs(la)).T @ np.abs(x))
    for name, got in (("dLA", dLA), ("dLB", dLB)):
        B.check(got, want[name], bound[name] + 1e-5 * np.abs(want[name]), F32, name)

    def half(a, b):
        return 0.5 * np.square(e - x @ (a @ b).T).sum()

    rng = np.random.default_rng(5)
    da, db = rng.standard_normal(la.shape), rng.standard_normal(lb.shape)
    t = 1e-4
    diff = (half(la + t * da, lb + t * db) - half(la - t * da, lb - t * db)) / (2 * t)
    # the formula's own distance from the difference is of order t^2; the kernels' as above
    exact = (want["dLA"] * da).sum() + (want["dLB"] * db).sum()
    assert abs(diff - exact) <= 1e-6 * (np.abs(want["dLA"] * da).sum() + np.abs(want["dLB"] * db).sum())
    got = (B.f64(dLA) * da).sum() + (B.f64(dLB) * db).sum()
    assert abs(got - diff) <= (bound["dLA"] * np.abs(da)).sum() + (bound["dLB"] * np.abs(db)).sum() + \
        2e-5 * (np.abs(want["dLA"] * da).sum() + np.abs(want["dLB"] * db).sum())


def test_trained_fit_runs():
    X, E = A.rnd(1, 300, 64), A.rnd(2, 300, 48)
    LA, LB = calib.train_lowrank(X, E, 8, steps=5, rows=128)
    assert LA.shape == (48, 8) and LB.shape == (8, 64) and LA.dtype == LB.dtype == F32
    assert bool(torch.isfinite(LA).all()) and bool(torch.isfinite(LB).all()) and bool(LA.any())
    again = calib.train_lowrank(X, E, 8, steps=5, rows=128)
    assert torch.equal(again[0], LA) and torch.equal(again[1], LB)
    # no step leaves the factors that were given
    same = calib.train_lowrank(X, E, 8, steps=0, LA=LA, LB=LB)
    assert torch.equal(same[0], LA) and torch.equal(same[1], LB)
