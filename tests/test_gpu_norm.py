"""GPU tests of the layer norm and its gradient against their definitions in 64 bits: widths that fill no
piece, wave or workgroup, groups of rows that are empty, end early or outnumber the rows, strides, odd
addresses, and what lies outside the groups."""
import numpy as np
import pytest
import torch

import _adapt as A
import _block as B
from _gpu import Guarded

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dt", (BF, F32), ids=("bf16", "f32"))


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# offsets for M rows; "early" starts late and ends early, "many" has more groups than a wave has lanes
GROUPS = {
    "none": lambda M: None,
    "one": lambda M: [0, M],
    "even": lambda M: [M * i // 3 for i in range(4)],
    "empty": lambda M: [0, 0, M // 3, M // 3, M // 3, M, M],
    "early": lambda M: [M // 4, M // 2, M - M // 5],
    "void": lambda M: [M // 2, M // 2],
    "many": lambda M: [M * i // 199 for i in range(200)],
    "rows": lambda M: [min(i, M) for i in range(5001)],
}


def case(seed, M, D, dt, groups, affine=True, mean=0.3):
    g = GROUPS[groups](M)
    G = 1 if g is None else len(g) - 1
    x = A.rnd(seed, M, D, dtype=dt, mean=mean)
    w, b = (A.rnd(seed + 1, D, std=0.2, dtype=dt, mean=1.0), A.rnd(seed + 2, D, std=0.2, dtype=dt)) if affine else (None, None)
    wide = A.rnd(seed + 3, G, 3 * D, std=0.3, dtype=dt)  # scale and shift as parts of one projection
    return dict(X=x, weight=w, bias=b, scale=wide[:, D:2 * D], shift=wide[:, :D],
                groups=None if g is None else torch.tensor(g, dtype=torch.int32, device="cuda")), g, G


def host(c):
    D = c["X"].shape[1]
    w = np.ones(D) if c.get("weight") is None else B.f64(c["weight"])
    b = np.zeros(D) if c.get("bias") is None else B.f64(c["bias"])
    scale, shift = (None if c.get(n) is None else B.f64(c[n]) for n in ("scale", "shift"))
    return B.f64(c["X"]), w, b, scale, shift


EPS = 1e-6
E32 = float(np.float32(EPS))


def run(c, g, G, dt, dY, name):
    M, D = c["X"].shape
    group = A.norm_rows(M, g)
    live = group >= 0
    x, w, b, scale, shift = host(c)
    Y, stats = Guarded((M, D), dt), Guarded((M, 2), F32)
    before = Y.t.clone()
    rtl.rtl_layer_norm(**c, eps=EPS, Y=Y.t, stats=stats.t)
    y, st, by, bs = A.norm_forward(x, w, b, scale, shift, group, E32)
    if live.any():
        B.check(Y.t[torch.from_numpy(live).cuda()], y[live], by[live], dt, name + " Y")
        B.check(stats.t[torch.from_numpy(live).cuda()], st[live], bs[live], F32, name + " stats")
    out = torch.from_numpy(~live).cuda()
    assert torch.equal(Y.t[out].view(torch.uint8), before[out].view(torch.uint8))
    Y.check(name)
    stats.check(name)

    dX = Guarded((M, D), dt)
    before = dX.t.clone()
    kept = torch.from_numpy(st).float().cuda()
    args = {k: v for k, v in c.items() if k not in ("X", "shift")}
    got = rtl.rtl_layer_norm_backward(c["X"], kept, dY, **args, dX=dX.t)
    dx, sums, bx, bounds = A.norm_backward(x, B.f64(kept), w, b, scale, group, G, B.f64(dY))
    if live.any():
        B.check(dX.t[torch.from_numpy(live).cuda()], dx[live], bx[live], dt, name + " dX")
    assert torch.equal(dX.t[out].view(torch.uint8), before[out].view(torch.uint8))
    dX.check(name)
    given = dict(dweight=c.get("weight"), dbias=c.get("bias"), dscale=c.get("scale"), dshift=c.get("scale"))
    for (what, of), t in zip(given.items(), got[1:]):
        assert (t is None) == (of is None), what
        if t is not None:
            B.check(t, sums[what], bounds[what], F32, f"{name} {what}")
    return got


@TYPES
@pytest.mark.parametrize("D", (1, 3, 8, 64, 72, 255, 257, 520, 1153, 2048, 2056, 5120, 8191))
def test_widths(D, dt):
    for M in (1, 5):
        c, g, G = case(D, M, D, dt, "none")
        run(c, g, G, dt, A.rnd(D + 9, M, D, std=0.1, dtype=dt), f"{M} x {D}")


@TYPES
@pytest.mark.parametrize("D", (8192, 10240, 13824, 16384, 32768))
def test_wide_rows(D, dt):
    if dt == F32 and D > 16384:
        with pytest.raises(rtl.RtlError):
            rtl.rtl_layer_norm(A.rnd(1, 2, D, dtype=dt))
        return
    c, g, G = case(D, 3, D, dt, "even")
    run(c, g, G, dt, A.rnd(D + 9, 3, D, std=0.1, dtype=dt), f"3 x {D}")


# a wave a row and a workgroup a row (1024 rows and more), chunks of 2 to 32 rows
@TYPES
@pytest.mark.parametrize("M,D", ((37, 320), (300, 1153), (1023, 1280), (1024, 264), (1500, 136), (2049, 5120), (17000, 72)))
@pytest.mark.parametrize("groups", ("none", "empty", "early", "many"))
def test_rows(M, D, groups, dt):
    c, g, G = case(M, M, D, dt, groups)
    run(c, g, G, dt, A.rnd(M + 9, M, D, std=0.1, dtype=dt), f"{M} x {D} {groups}")


@pytest.mark.parametrize("groups", sorted(GROUPS))
@pytest.mark.parametrize("affine", (True, False))
def test_groups(groups, affine):
    for M, D in ((1, 64), (70, 136), (1100, 64)):
        c, g, G = case(M, M, D, BF, groups, affine)
        run(c, g, G, BF, A.rnd(M + 9, M, D, std=0.1), f"{M} x {D} {groups}")


def test_groups_without_scale():
    """Groups alone say which rows are normed; the weights' sums run over them."""
    c, g, G = case(1, 200, 264, BF, "early")
    c["scale"] = c["shift"] = None
    got = run(c, g, G, BF, A.rnd(2, 200, 264, std=0.1), "no scale")
    assert got[3] is None and got[4] is None


@TYPES
def test_strides_and_addresses(dt):
    """Rows of a wider tensor, a tensor that starts at an odd element, and every row the same one."""
    M, D = 90, 264
    c, g, G = case(3, M, D, dt, "even")
    dY = A.rnd(5, M, D, std=0.1, dtype=dt)
    want = run(c, g, G, dt, dY, "plain")
    wide = torch.zeros(M, 3 * D, dtype=dt, device="cuda")
    wide[:, D:2 * D] = c["X"]
    c["X"] = wide[:, D:2 * D]
    assert all(torch.equal(a, b) for a, b in zip(run(c, g, G, dt, dY, "wide"), want))
    odd = torch.zeros(M * (D + 1) + 1, dtype=dt, device="cuda")[1:].view(M, D + 1)[:, :D]
    odd.copy_(c["X"])
    c["X"] = odd
    run(c, g, G, dt, dY, "odd")
    c["X"] = A.rnd(6, 1, D, dtype=dt).expand(M, D)
    run(c, g, G, dt, dY, "one row")


@TYPES
def test_in_place(dt):
    M, D = 33, 520
    c, g, G = case(3, M, D, dt, "early")
    dY = A.rnd(5, M, D, std=0.1, dtype=dt)
    stats = torch.zeros(M, 2, device="cuda")
    x = c.pop("X")
    Y = rtl.rtl_layer_norm(x, **c, Y=x.clone(), stats=stats)
    y = x.clone()
    rtl.rtl_layer_norm(y, **c, Y=y)
    assert torch.equal(y, Y)
    c.pop("shift")
    want = rtl.rtl_layer_norm_backward(x, stats, dY, **c, dX=dY.clone())
    d = dY.clone()
    got = rtl.rtl_layer_norm_backward(x, stats, d, **c, dX=d)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0] is d
    v = x.clone()
    got = rtl.rtl_layer_norm_backward(v, stats, dY, **c, dX=v)
    rows = A.norm_rows(M, g) >= 0
    assert torch.equal(v[torch.from_numpy(rows).cuda()], want[0][torch.from_numpy(rows).cuda()])
    # the same sums on every run, and none when they are not wanted
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    only = rtl.rtl_layer_norm_backward(x, stats, dY, **c, dX=dY.clone(), need_dw=False)
    assert torch.equal(only[0], want[0]) and only[1:] == (None,) * 4


@TYPES
@pytest.mark.parametrize("mean,std", ((0.0, 0.0), (3.0, 0.0), (1000.0, 1.0), (-3e4, 0.5), (0.0, 1e15), (0.0, 1e-15)))
def test_far_and_flat_rows(mean, std, dt):
    """Rows far from 0, of one value, large and small."""
    M, D = 4, 1032
    x = A.rnd(1, M, D, std=std, dtype=dt, mean=mean)
    run(dict(X=x, weight=None, bias=None, scale=None, shift=None, groups=None), None, 1, dt, A.rnd(2, M, D, dtype=dt), f"{mean} {std}")


def test_infinities_stay_in_their_rows():
    M, D = 6, 264
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = A.rnd(1, M, D)
        want = rtl.rtl_layer_norm(x)
        x[2, 7] = bad
        stats = torch.empty(M, 2, device="cuda")
        got = rtl.rtl_layer_norm(x, stats=stats)
        rest = [0, 1, 3, 4, 5]
        assert torch.equal(got[rest], want[rest]) and bool(torch.isnan(got[2]).all())
        assert bool(torch.isfinite(stats[rest]).all())
        # outside the groups: not read
        g = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
        dx, _, _, ds, dh = rtl.rtl_layer_norm_backward(x, stats, x, None, None, torch.zeros(1, D, dtype=BF, device="cuda"), g)
        assert bool(torch.isfinite(ds).all()) and bool(torch.isfinite(dh).all()) and bool(torch.isfinite(dx[:2]).all())


def test_gradient_against_differences():
    """The whole gradient along random directions, in fp32."""
    M, D, h = 24, 72, 1e-2
    c, g, G = case(11, M, D, F32, "empty")
    dY = A.rnd(12, M, D, dtype=F32)
    stats = torch.empty(M, 2, device="cuda")
    rtl.rtl_layer_norm(**c, eps=EPS, stats=stats)
    got = rtl.rtl_layer_norm_backward(c["X"], stats, dY, **{k: v for k, v in c.items() if k not in ("X", "shift")})
    names = ("X", "weight", "bias", "scale", "shift")

    def value(d, s):
        moved = {n: B.f64(c[n]) + s * h * d[n] for n in names}
        y = A.norm_forward(moved["X"], moved["weight"], moved["bias"], moved["scale"], moved["shift"], A.norm_rows(M, g), E32)[0]
        return (y * B.f64(dY)).sum()

    rng = np.random.default_rng(1)
    for n in names:
        d = {k: rng.standard_normal(tuple(c[k].shape)) * (k == n) for k in names}
        # five-point difference: the error is of order h^4
        slope = (8 * (value(d, 1) - value(d, -1)) - (value(d, 2) - value(d, -2))) / (12 * h)
        want = (B.f64(got[names.index(n)]) * d[n]).sum()
        scale = np.abs(B.f64(got[names.index(n)]) * d[n]).sum()
        assert abs(slope - want) <= 1e-4 * scale, (n, slope, want)


def test_captured_and_replayed():
    M, D = 300, 520
    c, g, G = case(1, M, D, BF, "even")
    dY, stats = A.rnd(2, M, D, std=0.1), torch.empty(M, 2, device="cuda")
    args = {k: v for k, v in c.items() if k not in ("X", "shift")}

    def step():
        Y = rtl.rtl_layer_norm(**c, stats=stats)
        return (Y, *rtl.rtl_layer_norm_backward(c["X"], stats, dY, **args))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        c["X"].copy_(A.rnd(50 + k, M, D))
        dY.copy_(A.rnd(60 + k, M, D, std=0.1))
        c["groups"].copy_(torch.tensor([0, 10 * k, 100 + 50 * k, M], dtype=torch.int32))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_on_another_stream():
    """A call on a stream that is not the current one, allocations and all."""
    M, D = 2000, 2560
    c, g, G = case(1, M, D, BF, "even")
    want = rtl.rtl_layer_norm(**c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rtl.rtl_layer_norm(**c, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
