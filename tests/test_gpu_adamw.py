"""GPU tests of the AdamW step: bit for bit the fp32 operations that define it, with states in 32 and in 8
bits, over lists of every size, and near its definition in 64 bits."""
import numpy as np
import pytest
import torch

import _adapt as A
from _block import f64

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HOW = dict(lr=3e-4, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def host(t):
    return t.detach().cpu().float().numpy()


class Tensors:
    def __init__(self, sizes, p_dt, g_dt, eight, seed=1, zero=False):
        rng = np.random.default_rng(seed)
        self.eight, self.bf16 = eight, p_dt == BF
        self.p = [rng.standard_normal(n).astype(np.float32) * np.float32(0.02) for n in sizes]
        size = [np.exp(2 * rng.standard_normal(n)).astype(np.float32) * np.float32(1e-3) for n in sizes]
        self.g = [(s * rng.standard_normal(s.size)).astype(np.float32) for s in size]
        self.m = [(0 if zero else 1) * (s * rng.standard_normal(s.size)).astype(np.float32) for s in size]
        u = [(0 if zero else 1) * s for s in size]
        cuda = lambda ts, dt=F32: [torch.from_numpy(t).to(dt).cuda() for t in ts]  # noqa: E731
        self.dev = dict(params=cuda(self.p, p_dt), grads=cuda(self.g, g_dt))
        self.g = [host(t) for t in self.dev["grads"]]
        if self.bf16:
            self.dev["masters"] = cuda(self.p)
        if eight:
            mc, vc = [A.encode(t, False) for t in self.m], [A.encode(t, True) for t in u]
            self.m, self.v = [c for c, _ in mc], [c for c, _ in vc]
            self.scales = [(a[1], b[1]) for a, b in zip(mc, vc)]
            self.dev.update(m=cuda(self.m, E4), v=cuda(self.v, E4), m_scales=cuda([s for s, _ in self.scales]),
                            v_scales=cuda([s for _, s in self.scales]))
        else:
            self.v = [t * t for t in u]
            self.dev.update(m=cuda(self.m), v=cuda(self.v))

    def step(self, step, clip=None, how=HOW):
        """The definition, on the host's copies."""
        for i in range(len(self.p)):
            got = A.adamw(self.p[i], self.g[i], self.m[i], self.v[i], step, how["lr"], how["beta1"], how["beta2"], how["eps"],
                          how["weight_decay"], clip, self.scales[i] if self.eight else None)
            if self.eight:
                self.p[i], (self.m[i], ms), (self.v[i], vs) = got
                self.scales[i] = ms, vs
            else:
                self.p[i], self.m[i], self.v[i] = got

    def check(self):
        d = self.dev
        for i, p in enumerate(self.p):
            kinds = dict(m=self.m[i], v=self.v[i])
            if self.eight:
                kinds.update(m_scales=self.scales[i][0], v_scales=self.scales[i][1])
            kinds["masters" if self.bf16 else "params"] = p
            for name, want in kinds.items():
                got = host(d[name][i])
                bad = np.nonzero(got != want)[0]
                assert bad.size == 0, f"{name}[{i}] differs at {bad[:4]} of {want.size}: {got[bad[:4]]} {want[bad[:4]]}"
            if self.bf16:
                assert torch.equal(d["params"][i], d["masters"][i].to(BF))


ALL = [(p, g, e) for p in (F32, BF) for g in (F32, BF) for e in (False, True)]
LABEL = ["-".join(("bf16" if p == BF else "f32", "bf16" if g == BF else "f32", "8" if e else "32")) for p, g, e in ALL]
# ends inside pieces of four, blocks of 256, workgroups of 4096; an empty tensor among them
SIZES = (1, 2, 3, 5, 255, 256, 257, 0, 700, 4095, 4096, 4097, 20001)


@pytest.mark.parametrize("p,g,eight", ALL, ids=LABEL)
@pytest.mark.parametrize("clip", (None, 0.37))
def test_steps(p, g, eight, clip):
    t = Tensors(SIZES, p, g, eight)
    at = None if clip is None else torch.tensor([clip], device="cuda")
    tensors = rtl.rtl_adamw_tensors(**t.dev)
    for step in (1, 2, 3, 1000):
        rtl.rtl_adamw(tensors, step=step, grad_scale=at, **HOW)
        t.step(step, clip)
        t.check()


@pytest.mark.parametrize("p,g,eight", ALL, ids=LABEL)
def test_from_the_start(p, g, eight):
    """States of zeros, and a tensor whose gradients are zeros: its parameters only decay."""
    t = Tensors((300, 1000), p, g, eight, zero=True)
    t.dev["grads"][1].zero_()
    t.g[1][:] = 0
    for step in (1, 2):
        rtl.rtl_adamw(rtl.rtl_adamw_tensors(**t.dev), step=step, **HOW)
        t.step(step)
        t.check()


def test_more_tensors_than_a_launch_takes():
    for count in (56, 57, 130):
        t = Tensors([1 + 37 * i % 5000 for i in range(count)], BF, BF, True, seed=count)
        rtl.rtl_adamw(rtl.rtl_adamw_tensors(**t.dev), step=7, **HOW)
        t.step(7)
        t.check()


@pytest.mark.parametrize("eight", (False, True))
def test_blocks_of_zeros_and_of_wide_range(eight):
    """Blocks whose values span more than the codes do: small roots keep the least code."""
    t = Tensors((1024,), F32, F32, eight)
    t.g[0][:256] = 0
    t.g[0][256:512] = np.geomspace(1e-12, 1e3, 256).astype(np.float32)
    t.g[0][512:768] = np.float32(1e-25)  # squares of zero
    t.g[0][768:] = np.float32(1e18)
    t.dev["grads"][0].copy_(torch.from_numpy(t.g[0]))
    tensors = rtl.rtl_adamw_tensors(**t.dev)
    for step in (1, 2, 3):
        rtl.rtl_adamw(tensors, step=step, **HOW)
        t.step(step)
        t.check()
    assert np.isfinite(t.p[0]).all()


@pytest.mark.parametrize("eight", (False, True))
def test_numbers_on_the_device(eight):
    """Step, learning rate and factor as tensors, captured once and replayed while they change."""
    t = Tensors((1000, 70), BF, BF, eight)
    step, lr, clip = torch.tensor([5], device="cuda"), torch.tensor([1e-3], device="cuda"), torch.tensor([0.5], device="cuda")
    tensors = rtl.rtl_adamw_tensors(**t.dev)
    how = {k: v for k, v in HOW.items() if k != "lr"}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rtl.rtl_adamw(tensors, step=step, lr=lr, grad_scale=clip, **how)
    t.check()  # recording runs nothing
    for k in range(4):
        lr.fill_(1e-3 / (k + 1))
        clip.fill_(0.5 + k)
        graph.replay()
        torch.cuda.synchronize()
        t.step(5 + k, 0.5 + k, dict(HOW, lr=float(np.float32(1e-3 / (k + 1)))))
        t.check()
        step.add_(1)


def test_against_the_definition_in_64_bits():
    t = Tensors((50000,), F32, F32, False, seed=3)
    p, g, m, v = (x[0].astype(np.float64) for x in (t.p, t.g, t.m, t.v))
    b1, b2 = HOW["beta1"], HOW["beta2"]
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    ahead = (m1 / (1 - b1 ** 9)) / (np.sqrt(v1 / (1 - b2 ** 9)) + HOW["eps"])
    want = p - HOW["lr"] * (ahead + HOW["weight_decay"] * p)
    rtl.rtl_adamw(rtl.rtl_adamw_tensors(**t.dev), step=9, **HOW)
    u = 2.0 ** -24
    # m: the difference, its product and the sum round once each, the factor once; v: the same of two terms
    size_m, size_v = np.abs(m) + 2 * np.abs(g), b2 * v + (1 - b2) * g * g
    assert (np.abs(f64(t.dev["m"][0]) - m1) <= 4 * u * size_m).all()
    assert (np.abs(f64(t.dev["v"][0]) - v1) <= 5 * u * size_v).all()
    # the step's quotient: m's error, half of v's, the two factors, sum and quotient; then lr, decay and p
    off = (4 * u * size_m / (1 - b1 ** 9)) / (np.sqrt(v1 / (1 - b2 ** 9)) + HOW["eps"]) + 9 * u * np.abs(ahead)
    assert (np.abs(f64(t.dev["params"][0]) - want) <= HOW["lr"] * (off + 4 * u * (np.abs(ahead) + np.abs(p))) + u * np.abs(want)).all()


def test_nothing_else_changes():
    """Views of one buffer for each kind: the gaps between them stay."""
    sizes = (300, 256, 1)
    room = [512, 256, 256]
    bufs = {n: torch.full((1024,), 7.0, device="cuda") for n in ("params", "grads", "m", "v")}
    starts = np.r_[0, np.cumsum(room)[:-1]]
    views = {n: [b[s:s + k] for s, k in zip(starts, sizes)] for n, b in bufs.items()}
    before = {n: b.clone() for n, b in bufs.items()}
    rtl.rtl_adamw(rtl.rtl_adamw_tensors(**views), step=1, **HOW)
    inside = torch.zeros(1024, dtype=torch.bool, device="cuda")
    for s, k in zip(starts, sizes):
        inside[s:s + k] = True
    for n, b in bufs.items():
        assert torch.equal(b[~inside], before[n][~inside])
        # gradients equal to m leave it as it is
        assert (n in ("grads", "m")) == torch.equal(b[inside], before[n][inside])


def test_autograd_sees_the_change():
    """A parameter that a backward pass still needs: autograd refuses it after the step."""
    p = torch.ones(8, device="cuda", requires_grad=True)
    y = (p * p).sum()
    t = [torch.zeros(8, device="cuda") for _ in range(3)]
    rtl.rtl_adamw(rtl.rtl_adamw_tensors([p], [t[0]], [t[1]], [t[2]]), step=1, lr=0.1)
    with pytest.raises(RuntimeError):
        y.backward()


def test_gradient_factor_is_a_tensor_on_the_gpu():
    t = Tensors((300,), F32, F32, False)
    tensors = rtl.rtl_adamw_tensors(**t.dev)
    for bad in (0.5, torch.tensor([0.5]), torch.tensor([0.5], device="cuda", dtype=torch.float64), torch.ones(2, device="cuda")):
        with pytest.raises(ValueError):
            rtl.rtl_adamw(tensors, step=1, grad_scale=bad, **HOW)
    t.check()  # as they were
