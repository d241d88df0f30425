"""The operators of a transformer block together, as the layer policy's objects call them: the
sparse QKV projection, head norms and rotary positions in place, attention (plain torch), the
dense output projection, the gated block with its sparse down projection.  Each stage is held
against its definition in 64 bits on the stage's own input, and the whole block, captured in a
graph and replayed on new tokens, against its eager run."""
import numpy as np
import pytest
import torch

import _block as B
import oracle
from _gpu import check_y, f64, to_host

pytestmark = pytest.mark.gpu

rtl = pytest.importorskip("activation_sparse_gemm_amd")
from activation_sparse_gemm_amd import policy  # noqa: E402

BF = torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rnd(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def tokens(seed, M, K):
    """A few percent of the channels large, as in the layer's own tests."""
    g = torch.Generator().manual_seed(seed)
    big = torch.rand(M, K, generator=g) < 0.08
    return (torch.randn(M, K, generator=g) * torch.where(big, 3.0, 0.1)).to(BF).cuda()


class Block:
    def __init__(self, K=256, heads=6, kv_heads=2, D=64, H=384, R=32):
        n = (heads + 2 * kv_heads) * D
        lin = lambda s, N, k: policy.Linear(rnd(s, N, k, std=k ** -0.5), rnd(s + 1, N, R, std=0.02), rnd(s + 2, R, k, std=0.02))
        self.heads, self.kv, self.D = heads, kv_heads, D
        self.inp = policy.AttentionInput(lin(1, n, K), heads, kv_heads, 1 + rnd(4, D, std=0.2), 1 + rnd(5, D, std=0.2),
                                         axis_dims=(16, 24, 24))
        self.out = policy.Linear(rnd(6, K, heads * D, std=(heads * D) ** -0.5), sparse=False)
        self.mlp = policy.GatedMLP(rnd(7, H, K, std=K ** -0.5), rnd(8, H, K, std=K ** -0.5), lin(9, K, H))

    def attention(self, q, k, v):
        q, k, v = (t.float().transpose(0, 1) for t in (q, k, v))
        k, v = (t.repeat_interleave(self.heads // self.kv, dim=0) for t in (k, v))
        p = torch.softmax((q @ k.transpose(1, 2).contiguous()) * self.D ** -0.5, dim=-1)
        return (p @ v).transpose(0, 1).reshape(q.shape[1], -1).to(BF)

    def __call__(self, X, pos, stages=None):
        q, k, v = self.inp(X, pos)
        a = self.attention(q, k, v)
        h = X + self.out(a)
        y = h + self.mlp(h)
        if stages is not None:
            stages.update(q=q, k=k, v=v, a=a, h=h, mlp=self.mlp(h))
        return y


def positions(M):
    i = torch.arange(M)
    return torch.stack([i // 60, i // 10 % 6, i % 10], dim=1).float().cuda()


@pytest.mark.parametrize("M", (1, 130, 301))
def test_stages(M):
    blk, X, pos = Block(), tokens(100 + M, M, 256), positions(M)
    s = {}
    blk(X, pos, s)
    # the projection as the norms found it, then the norms and the rotation of what it holds
    lin = blk.inp.qkv
    raw = rtl.rtl_linear_fused(X, lin.W, lin.LA, lin.LB).view(M, -1, 64)
    want, _ = oracle.linear(to_host(X), to_host(lin.W), to_host(lin.LA), to_host(lin.LB))
    check_y(f64(to_host(raw.reshape(M, -1)), "bf16"), want, "bf16", "qkv")
    phi = B.angles(B.f64(pos), (16, 24, 24), 10000.0)
    B.check(s["q"], *B.qk_forward(B.f64(raw[:, :6]), B.f64(blk.inp.q_weight), phi, 0, 1e-6), BF, "q")
    B.check(s["k"], *B.qk_forward(B.f64(raw[:, 6:8]), B.f64(blk.inp.k_weight), phi, 0, 1e-6), BF, "k")
    assert torch.equal(s["v"], raw[:, 8:])
    # the gated block into the sparse down projection
    gated = rtl.rtl_glu_fused(s["h"], blk.mlp.Wg, blk.mlp.Wu)
    y, _, _, by, _, _ = B.glu_forward(B.f64(s["h"]), B.f64(blk.mlp.Wg), B.f64(blk.mlp.Wu), 0)
    B.check(gated, y, by, BF, "gated")
    d = blk.mlp.down
    want, _ = oracle.linear(to_host(gated), to_host(d.W), to_host(d.LA), to_host(d.LB))
    check_y(f64(to_host(s["mlp"]), "bf16"), want, "bf16", "down")


def test_block_captured_and_replayed():
    M = 200
    blk, X, pos = Block(), tokens(1, M, 256), positions(M)
    blk(X, pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = blk(X, pos)
    for k in range(4):
        X.copy_(tokens(50 + k, M, 256))
        pos.add_(1)
        want = blk(X, pos)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want)


def test_training_step_of_the_new_operators():
    """Forward and backward chained by hand: rotation and norms, then the gated block fed with
    the queries; the gradients of tokens and norm weights against the definition's."""
    M, heads, D, H = 90, 4, 64, 200
    dims = (16, 24, 24)
    Q, w, pos = rnd(1, M, heads, D), 1 + rnd(2, D, std=0.2), positions(M)
    Wg, Wu, dY = rnd(3, H, heads * D, std=1 / 16), rnd(4, H, heads * D, std=1 / 16), rnd(5, M, H, std=0.1)
    q, _ = rtl.rtl_qk_norm_rope(Q, None, w, None, pos, dims)
    G, U = torch.empty(M, H, dtype=BF, device="cuda"), torch.empty(M, H, dtype=BF, device="cuda")
    rtl.rtl_glu_fused(q.view(M, -1), Wg, Wu, G=G, U=U)
    dq, dWg, dWu = rtl.rtl_glu_backward(q.view(M, -1), Wg, Wu, G, U, dY)
    dQ, _, dw, _ = rtl.rtl_qk_norm_rope_backward(Q, None, w, None, pos, dims, dq.view(M, heads, D), None)
    (rq, rg, ru), (bq, bg, bu) = B.glu_backward(*map(B.f64, (q.view(M, -1), Wg, Wu, G, U, dY)), 0)
    B.check(dq, rq, bq, BF, "dq")
    B.check(dWg, rg, bg, BF, "dWg")
    B.check(dWu, ru, bu, BF, "dWu")
    phi = B.angles(B.f64(pos), dims, 10000.0)
    rx, rw, bx, bw = B.qk_backward(B.f64(Q), B.f64(w), phi, 0, 1e-6, B.f64(dq.view(M, heads, D)))
    B.check(dQ, rx, bx, BF, "dQ")
    B.check(dw, rw, bw, torch.float32, "dw")


def test_calls_while_another_gpu_is_current(monkeypatch):
    """Each call makes its tensors' GPU the current one first (here the current device's number and
    the context that changes it stand in for a second GPU)."""
    M, H, D, K, N = 5, 3, 64, 128, 40
    q, k, g = rnd(1, M, H, D), rnd(2, M, H, D), rnd(3, M, H, D)
    w, pos = rnd(4, D), torch.rand(M, 1, device="cuda")
    x, wg, wu, dy = rnd(5, M, K), rnd(6, N, K), rnd(7, N, K), rnd(8, M, N)

    def calls():
        return (rtl.rtl_rope_axes(q, pos, (D,)), *rtl.rtl_qk_norm_rope(q, k, w, w, pos, (D,)),
                *rtl.rtl_qk_norm_rope_backward(q, k, w, w, pos, (D,), g, g), rtl.rtl_glu_fused(x, wg, wu),
                *rtl.rtl_glu_backward(x, wg, wu, dy, dy, dy))

    want, here, entered = calls(), q.get_device(), []
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
    assert entered == [here] * 5
    assert all(torch.equal(a, b) for a, b in zip(got, want))
