"""GPU tests at the edges of the layer norm, the adapters, the AdamW step and what is built on them."""
import pytest
import torch

import _adapt as A

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")

from activation_sparse_gemm_amd import calib, policy  # noqa: E402

BF = torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def digits(seed, M):
    """[M, 3] in bf16: a value of 24 digits, eight in each."""
    eight = torch.randint(128, 256, (M, 3), generator=torch.Generator().manual_seed(seed)) / 128
    return (eight * torch.tensor([1.0, 2.0 ** -8, 2.0 ** -16])).to(BF).cuda()


@pytest.mark.parametrize("M", (1, 12, 40, 200))  # joined in up's own launch, a block of rows, a tile, several
@pytest.mark.parametrize("R", (8, 40, 72, 128))
def test_every_digit_of_the_inner_product(M, R):
    """T = (h + m + l, -(h + m)) with 8 digits in each of h, m and l, added up: l to the bit.  All sums on the
    way are whole multiples of 2^-23 below 4, exact in fp32; T in two bf16 parts has 17 digits, which leave none of l."""
    K, N = 72, 136
    v = digits(M + R, M)
    plan = rtl.rtl_adapters_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), 1)
    # forward: three channels of X through two ranks into every column
    X = torch.zeros(M, K, dtype=BF, device="cuda")
    X[:, :3] = v
    LB, LA = torch.zeros(1, R, K, dtype=BF, device="cuda"), torch.zeros(1, N, R, dtype=BF, device="cuda")
    LB[0, 0, :3], LB[0, R - 1, :2], LA[0, :, 0], LA[0, :, R - 1] = 1.0, -1.0, 1.0, 1.0
    assert torch.equal(rtl.rtl_adapters(X, LA, LB, plan), v[:, 2:].expand(M, N))
    # back: three channels of dY through two ranks into every channel of dX
    dY = torch.zeros(M, N, dtype=BF, device="cuda")
    dY[:, :3] = v
    LB, LA = torch.zeros_like(LB), torch.zeros_like(LA)
    LA[0, :3, 0], LA[0, :2, R - 1], LB[0, 0], LB[0, R - 1] = 1.0, -1.0, 1.0, 1.0
    dX = rtl.rtl_adapters_backward(X, LA, LB, plan, None, dY, need_dw=False)[0]
    assert torch.equal(dX, v[:, 2:].expand(M, K))


@pytest.mark.parametrize("M", (128, 255, 256, 300))
def test_trained_fit_walks_the_whole_set(M):
    """The steps of the fit on the batches that its documentation names: the same factors to the bit."""
    K, N, R, rows, lr = 64, 48, 8, 128, 1e-2
    X, E = A.rnd(M, M, K), A.rnd(M + 1, M, N)
    start = [A.rnd(3, N, R, std=0.3, dtype=torch.float32), A.rnd(4, R, K, std=0.3, dtype=torch.float32)]
    got = calib.train_lowrank(X, E, R, steps=5, rows=rows, lr=lr, LA=start[0], LB=start[1])
    masters = [t.clone() for t in start]
    params = [t.to(BF) for t in masters]
    grads, m, v = ([torch.zeros_like(t) for t in masters] for _ in range(3))
    tensors = rtl.rtl_adamw_tensors(params, grads, m, v, masters=masters)
    scale = torch.full((1,), 2.0 / (rows * N), device="cuda")
    for step in range(5):
        at = torch.arange(step * rows, (step + 1) * rows, device="cuda") % M
        for to, t in zip(grads, calib.lowrank_gradient(X[at], E[at], *params)):
            to.copy_(t)
        rtl.rtl_adamw(tensors, step + 1, lr, weight_decay=0.0, grad_scale=scale)
    assert all(torch.equal(a, b) for a, b in zip(got, masters))


@pytest.mark.parametrize("dt", (BF, torch.float32), ids=("bf16", "f32"))
@pytest.mark.parametrize("M,D", ((2, 64), (70, 136), (37, 1153), (1100, 64), (1500, 136), (5, 8191), (2049, 5120)))
@pytest.mark.parametrize("groups", ("early", "void"))
def test_rows_of_no_request_in_new_outputs(M, D, groups, dt, monkeypatch):
    """Rows outside the groups are zeros in outputs that the call allocates, whatever their memory held, and as
    they were in outputs that it is given."""
    g = {"early": [M // 4, M // 2, M - M // 5], "void": [M // 2, M // 2, M // 2]}[groups]
    at = torch.tensor(g, dtype=torch.int32, device="cuda")
    X, dY, parts = A.rnd(1, M, D, dtype=dt), A.rnd(2, M, D, dtype=dt), A.rnd(3, 2, 2 * D, std=0.3, dtype=dt)
    live = torch.from_numpy(A.norm_rows(M, g) >= 0).cuda()
    X[~live] = dY[~live] = float("nan")
    kept, stats = torch.full_like(X, 7.0), torch.zeros(M, 2, device="cuda")
    scale, shift = parts[:, :D], parts[:, D:]
    norm = policy.AdaptiveNorm()

    fresh = rtl._new
    monkeypatch.setattr(rtl, "_new", lambda *of: fresh(*of).view(torch.uint8).fill_(255).view(of[3]))  # NaN in each type
    rtl.rtl_layer_norm(X, None, None, scale, shift, at, Y=kept, stats=stats)
    assert bool((kept[~live] == 7).all())
    Y = norm(X, scale, shift, at)
    assert torch.equal(Y[live], kept[live]) and not bool(Y[~live].any())
    want = rtl.rtl_layer_norm_backward(X, stats, dY, None, None, scale, at, dX=kept.fill_(7.0))
    assert bool((kept[~live] == 7).all())
    got = norm.backward(X, stats, dY, scale, at)
    assert torch.equal(got[0][live], kept[live]) and not bool(got[0][~live].any())
    assert all(torch.equal(a, b) for a, b in zip(got[3:], want[3:]))


@pytest.mark.parametrize("G,D", ((2 ** 24 + 3, 8), (2 ** 20 + 1, 40)))
def test_sums_of_more_groups_than_a_grid_row_takes(G, D):
    """A group of one row here and there among 2^24: each request's own gradients, zeros for the empty ones."""
    M = 7
    group = torch.tensor([0, 1, 2 ** 19, 2 ** 20 - 1, 2 ** 20, G - 2, G - 1]).sort().values  # each row's
    offsets = torch.searchsorted(group, torch.arange(G + 1)).int().cuda()
    X, dY, w = A.rnd(1, M, D), A.rnd(2, M, D, std=0.1), A.rnd(3, D, std=0.2, mean=1.0)
    scale = torch.zeros(1, D, dtype=BF, device="cuda").expand(G, D)
    stats = torch.zeros(M, 2, device="cuda")
    rtl.rtl_layer_norm(X, w, None, scale, scale, offsets, stats=stats)
    dX, dw, db, dscale, dshift = rtl.rtl_layer_norm_backward(X, stats, dY, w, None, scale, offsets)
    some = group.unique(return_inverse=True)[1]
    few = torch.searchsorted(some, torch.arange(int(some.max()) + 2)).int().cuda()
    want = rtl.rtl_layer_norm_backward(X, stats, dY, w, None, scale[:len(few) - 1], few)
    used = group.unique().cuda()
    assert torch.equal(dX, want[0]) and torch.equal(dw, want[1]) and db is None
    assert torch.equal(dscale[used], want[3]) and torch.equal(dshift[used], want[4])
    for t in (dscale, dshift):
        assert int(t.any(dim=1).sum()) == len(used)


@pytest.mark.parametrize("dt", (BF, torch.float32), ids=("bf16", "f32"))
@pytest.mark.parametrize("bad", (float("nan"), float("inf"), float("-inf")))
def test_parameters_of_empty_requests_do_not_enter(dt, bad):
    """Scale and shift of requests without rows, whatever they hold, and weights that are infinite, beside them."""
    M, D = 50, 72
    at = torch.tensor([0, 0, 20, 20, 20, 45, 45], dtype=torch.int32, device="cuda")
    X, dY = A.rnd(1, M, D, dtype=dt), A.rnd(2, M, D, std=0.1, dtype=dt)
    w, b, parts = A.rnd(3, D, dtype=dt), A.rnd(4, D, dtype=dt), A.rnd(5, 6, 2 * D, std=0.3, dtype=dt)
    empty = torch.tensor([True, False, True, True, False, True], device="cuda")
    stats, runs = torch.zeros(M, 2, device="cuda"), []
    for value in (None, bad):
        if value is not None:
            parts[empty] = value
        scale, shift = parts[:, :D], parts[:, D:]
        runs.append((rtl.rtl_layer_norm(X, w, b, scale, shift, at, stats=stats),
                     *rtl.rtl_layer_norm_backward(X, stats, dY, w, b, scale, at)))
    assert all(torch.equal(a, c) for a, c in zip(*runs)) and not bool(runs[0][4][empty].any())
    w[3], b[5] = bad, bad
    dscale, dshift = rtl.rtl_layer_norm_backward(X, stats, dY, w, b, parts[:, :D], at)[3:]
    assert not bool(dscale[empty].any()) and not bool(dshift[empty].any())


def test_layers_on_another_stream_leave_freed_memory_alone():
    """A layer that is dropped while its call waits on another stream: tensors made then hold their values, and the
    call gives what it gives alone.  A layer's calls on two streams do not meet either."""
    M, K, N, R = 130, 256, 320, 24
    X, plan = A.rnd(1, M, K), rtl.rtl_adapters_plan((torch.arange(M, device="cuda") % 3 - 1).int(), 2)

    def layer():
        shared = policy.Linear(W, LA, LB)
        return policy.AdaptedLinear(shared, *factors)

    W, LA, LB = A.rnd(2, N, K, std=K ** -0.5), A.rnd(3, N, 32, std=0.02), A.rnd(4, 32, K, std=0.02)
    factors = A.rnd(5, 2, N, R, std=R ** -0.5), A.rnd(6, 2, R, K, std=K ** -0.5)
    want = layer()(X, plan)
    sizes = rtl.rtl_linear_fused_workspace_bytes(rtl.RTL_BF16, M, N, K, 32), rtl.rtl_adapters_workspace_bytes(M, N, K, R, 2)
    side, Y = torch.cuda.Stream(), torch.empty_like(want)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        lin = layer()
        lin(X, plan, Y=Y, stream=side)
        del lin
        held = [torch.full((n,), 85, dtype=torch.uint8, device="cuda") for n in sizes * 2]
        torch.cuda.synchronize()
        assert all(bool((t == 85).all()) for t in held) and torch.equal(Y, want)
        del held
    lin, other, outs = layer(), torch.cuda.Stream(), []
    spaces = {lin.linear.workspace(M, s).data_ptr() for s in (None, side, other)}
    assert len(spaces) == 3 and lin.linear.workspace(M, side).data_ptr() in spaces
    for s in (side, other) * 8:
        outs.append(lin(X, plan, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in outs)


def test_layers_write_the_gradients_that_an_optimizer_holds():
    """Gradients in given tensors: the same values, and a step's list that is made once, captured with the
    gradients and replayed on other batches."""
    M, K, N, R = 90, 64, 72, 16
    factors = [A.rnd(5, 2, N, R, std=R ** -0.5, dtype=torch.float32), A.rnd(6, 2, R, K, std=K ** -0.5, dtype=torch.float32)]
    norm = policy.AdaptiveNorm(A.rnd(1, K, std=0.2, mean=1.0, dtype=BF), A.rnd(2, K, std=0.2))
    lin = policy.AdaptedLinear(policy.Linear(A.rnd(3, N, K, std=K ** -0.5), sparse=False), *(t.to(BF) for t in factors))
    at, ids = torch.tensor([0, 30, M], dtype=torch.int32, device="cuda"), (torch.arange(M, device="cuda") % 2).int()
    X, dY, parts, plan = A.rnd(7, M, K), A.rnd(8, M, N), A.rnd(9, 2, 2 * K, std=0.3), lin.plan(ids)
    scale, shift = parts[:, :K], parts[:, K:]
    stats, T = torch.empty(M, 2, device="cuda"), torch.empty(M, R, device="cuda")
    masters = [norm.weight.float(), norm.bias.float(), *factors]
    params = [norm.weight, norm.bias, lin.LA, lin.LB]
    grads = [torch.full_like(t, float("nan")) for t in masters]
    m, v = ([torch.zeros_like(t) for t in masters] for _ in range(2))
    tensors = rtl.rtl_adamw_tensors(params, grads, m, v, masters=masters)

    def gradients(given):
        h = norm(X, scale, shift, at, stats=stats)
        lin(h, plan, T=T)
        out = dict(zip(("dLA", "dLB"), grads[2:])) if given else {}
        dh, dLA, dLB = lin.backward(h, plan, T, dY, **out)
        out = dict(zip(("dweight", "dbias"), grads[:2])) if given else {}
        return norm.backward(X, stats, dh, scale, at, **out)[1:3] + (dLA, dLB)

    def step():
        gradients(True)
        rtl.rtl_adamw(tensors, 1, 1e-2)

    want = gradients(False)
    got = gradients(True)
    assert all(a is b for a, b in zip(got, grads)) and all(torch.equal(a, b) for a, b in zip(grads, want))
    dX, ds, dh = torch.empty_like(X), torch.empty(2, K, device="cuda"), torch.empty(2, K, device="cuda")
    out = norm.backward(X, stats, X, scale, at, dX=dX, dscale=ds, dshift=dh)
    assert out[0] is dX and out[3] is ds and out[4] is dh
    out = lin.backward(X, plan, T, dY, dX=dX)
    assert out[0] is dX
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    state = masters + m + v + params
    for k in range(3):
        X.copy_(A.rnd(20 + k, M, K))
        before = [t.clone() for t in state]
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in state + grads]
        for t, b in zip(state, before):
            t.copy_(b)
        step()
        assert all(torch.equal(a, b) for a, b in zip(replayed, state + grads))


def test_layers_while_another_gpu_is_current(monkeypatch):
    """A projection, and one with adapters, makes its tensors' GPU the current one first (here the current device's
    number and the context that changes it stand in for a second GPU)."""
    M, K, N, R = 9, 64, 40, 8
    X, W, ids = A.rnd(1, M, K), A.rnd(2, N, K), (torch.arange(M, device="cuda") % 2).int()
    layers = [policy.Linear(W, sparse=False), policy.Linear(W, A.rnd(3, N, 32, std=0.1), A.rnd(4, 32, K, std=0.1))]
    layers += [policy.AdaptedLinear(layer, A.rnd(5, 2, N, R), A.rnd(6, 2, R, K)) for layer in layers]

    def calls():
        plan = layers[2].plan(ids)
        return [layer(X) for layer in layers[:2]] + [layer(X, plan) for layer in layers[2:]]

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
    assert len(entered) == 7 and set(entered) == {here}  # the plan, four projections, two calls of adapters
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for layer in layers[:2]:
        with pytest.raises(ValueError):
            layer(X.cpu())
