"""Refusals of the rotary, head-norm and gated-block entry points: each bad call returns its
status and message, launches nothing and leaves the outputs alone (CPU only: the "device"
pointers are host buffers that no call reads)."""
import ctypes

import numpy as np
import pytest
import torch

rtl = pytest.importorskip("activation_sparse_gemm_amd")
CODE = {v: k for k, v in rtl.STATUS.items()}


class Buffers:
    def __init__(self):
        self.all = []

    def __call__(self, nbytes):
        a = np.full(nbytes + 64, 0xAB, np.uint8)
        self.all.append(a)
        return ctypes.c_void_p(a.ctypes.data + (-a.ctypes.data) % 16)

    def untouched(self):
        return all((a == 0xAB).all() for a in self.all)


def label(v):
    """A case's name, the same in every process: what the call is given instead, or its status."""
    return v if isinstance(v, str) else ",".join(f"{k}={'other' if callable(x) else str(x)[:16] if not hasattr(x, '_length_') else list(x)}"
                                                 for k, x in v.items())


def at(p, nbytes):
    return ctypes.c_void_p(p.value + nbytes)


def refused(status, want, bufs, over):
    assert status == CODE[want], (over, rtl.STATUS.get(status), rtl.lib.rtl_last_error())
    assert rtl.lib.rtl_last_error().decode() != "" and bufs.untouched(), over


def dims(*d):
    return (ctypes.c_int32 * max(len(d), 1))(*d)


def rope(**over):
    b = Buffers()
    a = dict(dt=rtl.RTL_BF16, M=4, H=3, D=64, x=b(4 * 3 * 64 * 4), xs=(192, 64), pos=b(4 * 4 * 4), n=2, dims=dims(32, 32),
             theta=1e4, pairs=0, inverse=0, y=b(4 * 3 * 64 * 4), ys=(192, 64))
    if callable(over.get("y")):
        over["y"] = over["y"](a)
    a.update(over)
    st = rtl.lib.rtl_rope_axes(a["dt"], a["M"], a["H"], a["D"], a["x"], *a["xs"], a["pos"], a["n"], a["dims"], a["theta"],
                               a["pairs"], a["inverse"], a["y"], *a["ys"], None)
    return st, b


ROPE = [
    (dict(dt=5), "RTL_ERR_UNSUPPORTED"), (dict(M=0), "RTL_ERR_SHAPE"), (dict(H=0), "RTL_ERR_SHAPE"),
    (dict(D=0), "RTL_ERR_SHAPE"), (dict(M=-3), "RTL_ERR_SHAPE"), (dict(D=60), "RTL_ERR_UNSUPPORTED"),
    (dict(D=264), "RTL_ERR_UNSUPPORTED"), (dict(M=2 ** 31), "RTL_ERR_SHAPE"), (dict(M=2 ** 16, H=2 ** 15), "RTL_ERR_SHAPE"),
    (dict(M=2 ** 62, H=2 ** 62), "RTL_ERR_SHAPE"), (dict(n=0), "RTL_ERR_UNSUPPORTED"), (dict(n=5), "RTL_ERR_UNSUPPORTED"),
    (dict(n=-1), "RTL_ERR_UNSUPPORTED"), (dict(pairs=2), "RTL_ERR_UNSUPPORTED"), (dict(pairs=-1), "RTL_ERR_UNSUPPORTED"),
    (dict(dims=dims(31, 33)), "RTL_ERR_SHAPE"), (dict(dims=dims(0, 32)), "RTL_ERR_SHAPE"),
    (dict(dims=dims(-8, 40)), "RTL_ERR_SHAPE"), (dict(dims=dims(40, 32)), "RTL_ERR_SHAPE"),
    (dict(dims=dims(2, 4)), "RTL_ERR_UNSUPPORTED"), (dict(theta=0.0), "RTL_ERR_ARG"), (dict(theta=-1.0), "RTL_ERR_ARG"),
    (dict(theta=float("nan")), "RTL_ERR_ARG"), (dict(theta=float("inf")), "RTL_ERR_ARG"),
    (dict(inverse=2), "RTL_ERR_ARG"), (dict(pos=None), "RTL_ERR_NULL"), (dict(dims=None), "RTL_ERR_NULL"),
    (dict(x=None), "RTL_ERR_NULL"), (dict(y=None), "RTL_ERR_NULL"), (dict(xs=(-192, 64)), "RTL_ERR_SHAPE"),
    (dict(xs=(192, 2 ** 62)), "RTL_ERR_SHAPE"), (dict(xs=(193, 64)), "RTL_ERR_ALIGN"), (dict(ys=(192, 68)), "RTL_ERR_ALIGN"),
    (dict(y=lambda a: at(a["y"], 8)), "RTL_ERR_ALIGN"), (dict(y=lambda a: at(a["x"], 16)), "RTL_ERR_ARG"),
    (dict(y=lambda a: a["x"], ys=(256, 64)), "RTL_ERR_ARG"), (dict(y=lambda a: a["pos"]), "RTL_ERR_ARG"),
    (dict(ys=(0, 64)), "RTL_ERR_ARG"), (dict(ys=(192, 0)), "RTL_ERR_ARG"), (dict(ys=(128, 64)), "RTL_ERR_ARG"),
    (dict(ys=(192, 32)), "RTL_ERR_ARG"),
]


@pytest.mark.parametrize("over,want", ROPE, ids=label)
def test_rope_refusals(over, want):
    st, b = rope(**over)
    refused(st, want, b, over)


def qk(back=False, **over):
    b = Buffers()
    size = 4 * 8 * 64 * 2
    a = dict(dt=rtl.RTL_BF16, M=4, Hq=3, Hk=2, D=64, Q=b(size), K=b(size), qw=b(256), kw=b(256), eps=1e-6, pos=b(64), n=2,
             dims=dims(32, 32), theta=1e4, pairs=0, Qo=b(size), Ko=b(size), dQ=b(size), dK=b(size), dqw=b(256), dkw=b(256),
             ws=b(rtl.rtl_qk_norm_rope_backward_workspace_bytes(64)),
             wsb=rtl.rtl_qk_norm_rope_backward_workspace_bytes(64), q=(192, 64), k=(128, 64))
    for name, v in over.items():
        a[name] = v(a) if callable(v) else v
    head = [a["dt"], a["M"], a["Hq"], a["Hk"], a["D"], a["Q"], *a["q"], a["K"], *a["k"], a["qw"], a["kw"], a["eps"],
            a["pos"], a["n"], a["dims"], a["theta"], a["pairs"], a["Qo"], 192, 64, a["Ko"], 128, 64]
    if not back:
        return rtl.lib.rtl_qk_norm_rope(*head, None), b
    return rtl.lib.rtl_qk_norm_rope_backward(*head, a["dQ"], 192, 64, a["dK"], 128, 64, a["dqw"], a["dkw"], a["ws"],
                                             a["wsb"], None), b


QK = [
    (dict(dt=2), "RTL_ERR_UNSUPPORTED"), (dict(Hq=0), "RTL_ERR_SHAPE"), (dict(Hk=-1), "RTL_ERR_SHAPE"),
    (dict(eps=0.0), "RTL_ERR_ARG"), (dict(eps=float("nan")), "RTL_ERR_ARG"), (dict(eps=2.0), "RTL_ERR_ARG"),
    (dict(n=5), "RTL_ERR_UNSUPPORTED"), (dict(Q=None), "RTL_ERR_NULL"), (dict(K=None), "RTL_ERR_NULL"),
    (dict(Qo=None), "RTL_ERR_NULL"), (dict(Ko=None), "RTL_ERR_NULL"), (dict(pos=None), "RTL_ERR_NULL"),
    (dict(qw=lambda a: at(a["qw"], 2)), "RTL_ERR_ALIGN"), (dict(k=(132, 64)), "RTL_ERR_ALIGN"),
]
QK_FORWARD = [
    (dict(Qo=lambda a: a["K"]), "RTL_ERR_ARG"), (dict(Ko=lambda a: a["Q"]), "RTL_ERR_ARG"),
    (dict(Ko=lambda a: a["Qo"]), "RTL_ERR_ARG"), (dict(Qo=lambda a: a["qw"]), "RTL_ERR_ARG"),
    (dict(Qo=lambda a: at(a["Q"], 128)), "RTL_ERR_ARG"),
]
QK_BACKWARD = [
    (dict(dQ=None), "RTL_ERR_NULL"), (dict(dK=None), "RTL_ERR_NULL"), (dict(dQ=lambda a: a["K"]), "RTL_ERR_ARG"),
    (dict(dQ=lambda a: a["Ko"]), "RTL_ERR_ARG"), (dict(dK=lambda a: a["dQ"]), "RTL_ERR_ARG"),
    (dict(dqw=lambda a: a["dkw"]), "RTL_ERR_ARG"), (dict(dqw=lambda a: a["Q"]), "RTL_ERR_ARG"),
    (dict(dkw=lambda a: a["dK"]), "RTL_ERR_ARG"), (dict(ws=lambda a: a["Qo"]), "RTL_ERR_ARG"),
    (dict(ws=lambda a: at(a["ws"], 8)), "RTL_ERR_ALIGN"), (dict(ws=None), "RTL_ERR_WORKSPACE"),
    (dict(wsb=16), "RTL_ERR_WORKSPACE"),
]


@pytest.mark.parametrize("over,want", QK + QK_FORWARD, ids=label)
def test_qk_refusals(over, want):
    st, b = qk(**over)
    refused(st, want, b, over)


@pytest.mark.parametrize("over,want", QK + QK_BACKWARD, ids=label)
def test_qk_backward_refusals(over, want):
    st, b = qk(back=True, **over)
    refused(st, want, b, over)


def glu(**over):
    b = Buffers()
    M, K, H = 3, 64, 40
    x, w, y = 2 * M * K, 2 * H * K, 2 * M * H
    a = dict(act=0, dt=rtl.RTL_BF16, M=M, K=K, H=H, X=b(x), Wg=b(w), Wu=b(w), Y=b(y), G=b(y), U=b(y))
    for name, v in over.items():
        a[name] = v(a) if callable(v) else v
    return rtl.lib.rtl_glu_fused(*[a[n] for n in ("act", "dt", "M", "K", "H", "X", "Wg", "Wu", "Y", "G", "U")], None), b


def glu_back(**over):
    b = Buffers()
    M, K, H = 3, 64, 40
    x, w, y = 2 * M * K, 2 * H * K, 2 * M * H
    need = rtl.rtl_glu_backward_workspace_bytes(M, K, H)
    a = dict(act=0, dt=rtl.RTL_BF16, M=M, K=K, H=H, X=b(x), Wg=b(w), Wu=b(w), G=b(y), U=b(y), dY=b(y), dX=b(x), dWg=b(w),
             dWu=b(w), ws=b(need), wsb=need)
    for name, v in over.items():
        a[name] = v(a) if callable(v) else v
    return rtl.lib.rtl_glu_backward(*[a[n] for n in ("act", "dt", "M", "K", "H", "X", "Wg", "Wu", "G", "U", "dY", "dX", "dWg",
                                                     "dWu", "ws", "wsb")], None), b


GLU = [
    (dict(act=2), "RTL_ERR_UNSUPPORTED"), (dict(act=-1), "RTL_ERR_UNSUPPORTED"), (dict(dt=rtl.RTL_F32), "RTL_ERR_UNSUPPORTED"),
    (dict(dt=9), "RTL_ERR_UNSUPPORTED"), (dict(M=0), "RTL_ERR_SHAPE"), (dict(K=0), "RTL_ERR_SHAPE"), (dict(H=-1), "RTL_ERR_SHAPE"),
    (dict(K=96), "RTL_ERR_UNSUPPORTED"), (dict(K=2 ** 22), "RTL_ERR_SHAPE"), (dict(M=2 ** 31), "RTL_ERR_SHAPE"),
    (dict(M=2 ** 62), "RTL_ERR_SHAPE"), (dict(M=2 ** 30, H=2 ** 30), "RTL_ERR_SHAPE"), (dict(X=None), "RTL_ERR_NULL"),
    (dict(Wg=None), "RTL_ERR_NULL"), (dict(M=1, H=2 ** 28 - 15), "RTL_ERR_SHAPE"), (dict(M=2 ** 20, H=2 ** 17), "RTL_ERR_SHAPE"), (dict(M=2 ** 31 - 1, H=129), "RTL_ERR_SHAPE"),
    (dict(X=lambda a: at(a["X"], 2)), "RTL_ERR_ALIGN"),
    (dict(U=lambda a: at(a["U"], 4)), "RTL_ERR_ALIGN"),
]


@pytest.mark.parametrize("over,want", GLU + [
    (dict(Y=None), "RTL_ERR_NULL"), (dict(Y=lambda a: a["X"]), "RTL_ERR_ARG"), (dict(G=lambda a: a["Wu"]), "RTL_ERR_ARG"),
    (dict(U=lambda a: a["Y"]), "RTL_ERR_ARG"), (dict(G=lambda a: a["U"]), "RTL_ERR_ARG"),
], ids=label)
def test_glu_refusals(over, want):
    st, b = glu(**over)
    refused(st, want, b, over)


@pytest.mark.parametrize("over,want", GLU + [
    (dict(dX=None, dWg=None, dWu=None), "RTL_ERR_NULL"), (dict(dWg=None), "RTL_ERR_NULL"), (dict(dY=None), "RTL_ERR_NULL"),
    (dict(U=None), "RTL_ERR_NULL"), (dict(dX=lambda a: a["X"]), "RTL_ERR_ARG"), (dict(dWu=lambda a: a["dWg"]), "RTL_ERR_ARG"),
    (dict(dX=lambda a: a["dY"]), "RTL_ERR_ARG"), (dict(ws=lambda a: a["G"]), "RTL_ERR_ARG"),
    (dict(ws=lambda a: at(a["ws"], 8)), "RTL_ERR_ALIGN"), (dict(ws=None), "RTL_ERR_WORKSPACE"),
    (dict(wsb=64), "RTL_ERR_WORKSPACE"), (dict(H=2 ** 21), "RTL_ERR_SHAPE"), (dict(M=2 ** 22), "RTL_ERR_SHAPE"),
    (dict(M=2 ** 20, H=2 ** 15), "RTL_ERR_SHAPE"),
], ids=label)
def test_glu_backward_refusals(over, want):
    st, b = glu_back(**over)
    refused(st, want, b, over)


def test_python_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        rtl.rtl_rope_axes(x, torch.zeros(2, 1), (64,))
    with pytest.raises(ValueError):
        rtl.rtl_glu_fused(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16),
                          torch.zeros(8, 64, dtype=torch.bfloat16))
    assert rtl.rtl_qk_norm_rope_backward_workspace_bytes(0) == 0
    assert rtl.rtl_glu_backward_workspace_bytes(0, 64, 64) == 0
    for M, K, H in ((2 ** 22, 64, 64), (64, 64, 2 ** 21), (64, 2 ** 22, 64), (2 ** 20, 64, 2 ** 15), (2 ** 62, 64, 2 ** 62)):
        assert rtl.rtl_glu_backward_workspace_bytes(M, K, H) == 0
    # more output tiles than 32 bits hold of parts: no part of a tile, P alone
    assert rtl.rtl_glu_backward_workspace_bytes(2 ** 22 - 64, 2 ** 22 - 64, 64) == (2 ** 22 - 64) * 2 * 64 * 2


def test_policy_objects_check_their_weights():
    from activation_sparse_gemm_amd import policy

    W = torch.zeros(8 * 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        policy.AttentionInput(policy.Linear(W, sparse=False), heads=3, kv_heads=1)
    with pytest.raises(ValueError):
        policy.AttentionInput(policy.Linear(W, sparse=False), heads=0, kv_heads=4)
    with pytest.raises(ValueError):
        policy.GatedMLP(W, W, policy.Linear(W, sparse=False))
    with pytest.raises(ValueError):
        policy.GatedMLP(W, W[:64], policy.Linear(torch.zeros(64, 8 * 64, dtype=torch.bfloat16), sparse=False))
