"""Refusals of the layer norm's, the adapters' and the AdamW step's entry points: each bad call returns its
status and message, launches nothing and leaves the outputs alone (CPU only: the "device" pointers
are host buffers that no call reads)."""
import ctypes

import pytest
import torch

from test_block_abi import Buffers, at, label, refused

rtl = pytest.importorskip("activation_sparse_gemm_amd")


def filled(a, over):
    for name, v in over.items():
        a[name] = v(a) if callable(v) else v
    return a


def norm(back=False, **over):
    b = Buffers()
    M, D, G = 6, 64, 2
    row, flat = 2 * M * D, 2 * D
    a = filled(dict(dt=rtl.RTL_BF16, M=M, D=D, X=b(row), xr=D, w=b(flat), b=b(flat), G=G, groups=b(16), sc=b(2 * G * D), scr=D,
                    sh=b(2 * G * D), shr=D, eps=1e-6, Y=b(row), yr=D, st=b(8 * M), dY=b(row), dyr=D, dw=b(4 * D), db=b(4 * D),
                    ds=b(4 * G * D), dh=b(4 * G * D), ws=b(rtl.rtl_layer_norm_backward_workspace_bytes(M, D, G)),
                    wsb=rtl.rtl_layer_norm_backward_workspace_bytes(M, D, G)), over)
    pick = lambda names: [a[n] for n in names.split()]  # noqa: E731
    if back:
        return rtl.lib.rtl_layer_norm_backward(*pick("dt M D X xr st dY dyr w b G groups sc scr Y yr dw db ds dh ws wsb"), None), b
    return rtl.lib.rtl_layer_norm(*pick("dt M D X xr w b G groups sc scr sh shr eps Y yr st"), None), b


NORM = [
    (dict(dt=7), "RTL_ERR_UNSUPPORTED"), (dict(M=0), "RTL_ERR_SHAPE"), (dict(D=0), "RTL_ERR_SHAPE"), (dict(G=-1), "RTL_ERR_SHAPE"),
    (dict(M=2 ** 31), "RTL_ERR_SHAPE"), (dict(M=2 ** 62), "RTL_ERR_SHAPE"), (dict(D=32769), "RTL_ERR_UNSUPPORTED"),
    (dict(D=2 ** 62), "RTL_ERR_UNSUPPORTED"), (dict(G=2 ** 31), "RTL_ERR_SHAPE"),
    (dict(dt=rtl.RTL_F32, D=16388), "RTL_ERR_UNSUPPORTED"), (dict(X=None), "RTL_ERR_NULL"), (dict(Y=None), "RTL_ERR_NULL"),
    (dict(groups=None), "RTL_ERR_NULL"), (dict(G=0), "RTL_ERR_SHAPE"), (dict(xr=-64), "RTL_ERR_SHAPE"),
    (dict(xr=2 ** 60), "RTL_ERR_SHAPE"), (dict(yr=63), "RTL_ERR_ARG"), (dict(yr=0), "RTL_ERR_ARG"),
    (dict(X=lambda a: at(a["X"], 1)), "RTL_ERR_ALIGN"), (dict(w=lambda a: at(a["w"], 1)), "RTL_ERR_ALIGN"),
    (dict(groups=lambda a: at(a["groups"], 2)), "RTL_ERR_ALIGN"), (dict(st=lambda a: at(a["st"], 4)), "RTL_ERR_ALIGN"),
    (dict(Y=lambda a: at(a["X"], 16)), "RTL_ERR_ARG"), (dict(Y=lambda a: a["w"]), "RTL_ERR_ARG"), (dict(Y=lambda a: a["sc"]), "RTL_ERR_ARG"),
    (dict(Y=lambda a: a["groups"]), "RTL_ERR_ARG"), (dict(scr=-1), "RTL_ERR_SHAPE"),
    # 8192 wide at the most where pieces of 16 bytes do not fit
    (dict(M=1, D=8200, G=0, groups=None, sc=None, sh=None, ds=None, dh=None, X=lambda a: at(a["X"], 2)), "RTL_ERR_UNSUPPORTED"),
]


@pytest.mark.parametrize("over,want", NORM + [
    (dict(eps=0.0), "RTL_ERR_ARG"), (dict(eps=float("nan")), "RTL_ERR_ARG"), (dict(eps=1.5), "RTL_ERR_ARG"),
    (dict(sh=None), "RTL_ERR_NULL"), (dict(sc=None), "RTL_ERR_NULL"), (dict(shr=-1), "RTL_ERR_SHAPE"),
    (dict(Y=lambda a: a["st"]), "RTL_ERR_ARG"), (dict(st=lambda a: a["X"]), "RTL_ERR_ARG"), (dict(st=lambda a: a["sh"]), "RTL_ERR_ARG"),
], ids=label)
def test_norm_refusals(over, want):
    st, b = norm(**over)
    refused(st, want, b, over)


@pytest.mark.parametrize("over,want", [c for c in NORM if "st" not in c[0]] + [
    (dict(st=None), "RTL_ERR_NULL"), (dict(st=lambda a: at(a["st"], 4)), "RTL_ERR_ALIGN"), (dict(dY=None), "RTL_ERR_NULL"),
    (dict(dyr=-1), "RTL_ERR_SHAPE"), (dict(sc=None), "RTL_ERR_ARG"), (dict(dw=lambda a: at(a["dw"], 4)), "RTL_ERR_ALIGN"),
    (dict(dw=lambda a: a["db"]), "RTL_ERR_ARG"), (dict(ds=lambda a: a["dh"]), "RTL_ERR_ARG"), (dict(dh=lambda a: a["Y"]), "RTL_ERR_ARG"),
    (dict(db=lambda a: a["st"]), "RTL_ERR_ARG"), (dict(ws=lambda a: a["X"]), "RTL_ERR_ARG"), (dict(ws=lambda a: a["Y"]), "RTL_ERR_ARG"),
    (dict(Y=lambda a: at(a["dY"], 16)), "RTL_ERR_ARG"), (dict(Y=lambda a: a["st"]), "RTL_ERR_ARG"),
    (dict(ws=lambda a: at(a["ws"], 8)), "RTL_ERR_ALIGN"), (dict(ws=None), "RTL_ERR_WORKSPACE"), (dict(wsb=64), "RTL_ERR_WORKSPACE"),
    (dict(G=2 ** 24), "RTL_ERR_SHAPE"),
], ids=label)
def test_norm_backward_refusals(over, want):
    st, b = norm(back=True, **over)
    refused(st, want, b, over)


def adapters(back=False, **over):
    b = Buffers()
    M, N, K, R, A = 5, 40, 64, 16, 3
    need, back_need = rtl.rtl_adapters_workspace_bytes(M, N, K, R, A), rtl.rtl_adapters_backward_workspace_bytes(M, N, K, R, A)
    a = filled(dict(dt=rtl.RTL_BF16, M=M, N=N, K=K, R=R, A=A, X=b(2 * M * K), xr=K, LA=b(2 * A * N * R), LB=b(2 * A * K * R),
                    al=b(4 * A), plan=b(rtl.rtl_adapters_plan_bytes(M, A)), pb=rtl.rtl_adapters_plan_bytes(M, A), Y0=b(2 * M * N),
                    y0r=N, Y=b(2 * M * N), yr=N, T=b(4 * M * R), ws=b(max(need, back_need)), wsb=max(need, back_need),
                    dY=b(2 * M * N), dyr=N, dX0=b(2 * M * K), dx0r=K, dX=b(2 * M * K), dxr=K, dLA=b(4 * A * N * R), dLB=b(4 * A * K * R)),
               over)
    pick = lambda names: [a[n] for n in names.split()]  # noqa: E731
    head = pick("dt M N K R A X xr LA LB al plan pb")
    if back:
        return rtl.lib.rtl_adapters_backward(*head, *pick("T dY dyr dX0 dx0r dX dxr dLA dLB ws wsb"), None), b
    return rtl.lib.rtl_adapters(*head, *pick("Y0 y0r Y yr T ws wsb"), None), b


ADAPTERS = [
    (dict(dt=rtl.RTL_F32), "RTL_ERR_UNSUPPORTED"), (dict(dt=3), "RTL_ERR_UNSUPPORTED"), (dict(M=0), "RTL_ERR_SHAPE"),
    (dict(N=0), "RTL_ERR_SHAPE"), (dict(K=-8), "RTL_ERR_SHAPE"), (dict(R=0), "RTL_ERR_SHAPE"), (dict(A=0), "RTL_ERR_SHAPE"),
    (dict(M=2 ** 24 + 1), "RTL_ERR_SHAPE"), (dict(A=4097), "RTL_ERR_SHAPE"), (dict(K=2 ** 22 + 8), "RTL_ERR_SHAPE"),
    (dict(N=2 ** 62), "RTL_ERR_SHAPE"), (dict(N=44), "RTL_ERR_UNSUPPORTED"), (dict(K=60), "RTL_ERR_UNSUPPORTED"),
    (dict(R=12), "RTL_ERR_UNSUPPORTED"), (dict(R=136), "RTL_ERR_UNSUPPORTED"), (dict(A=64, K=2 ** 22), "RTL_ERR_SHAPE"),
    (dict(X=None), "RTL_ERR_NULL"), (dict(LA=None), "RTL_ERR_NULL"), (dict(LB=None), "RTL_ERR_NULL"), (dict(plan=None), "RTL_ERR_NULL"),
    (dict(pb=16), "RTL_ERR_ARG"), (dict(pb=lambda a: a["pb"] + 4), "RTL_ERR_ARG"), (dict(xr=68), "RTL_ERR_ALIGN"),
    (dict(xr=-64), "RTL_ERR_SHAPE"), (dict(LB=lambda a: at(a["LB"], 8)), "RTL_ERR_ALIGN"), (dict(al=lambda a: at(a["al"], 2)), "RTL_ERR_ALIGN"),
    (dict(T=lambda a: at(a["T"], 4)), "RTL_ERR_ALIGN"), (dict(ws=lambda a: at(a["ws"], 8)), "RTL_ERR_ALIGN"),
    (dict(ws=lambda a: a["X"]), "RTL_ERR_ARG"), (dict(ws=lambda a: a["plan"]), "RTL_ERR_ARG"), (dict(ws=None), "RTL_ERR_WORKSPACE"),
    (dict(wsb=0), "RTL_ERR_WORKSPACE"),
]


@pytest.mark.parametrize("over,want", ADAPTERS + [
    (dict(Y=None), "RTL_ERR_NULL"), (dict(yr=32), "RTL_ERR_ARG"), (dict(yr=44), "RTL_ERR_ALIGN"), (dict(y0r=41), "RTL_ERR_ALIGN"),
    (dict(Y=lambda a: a["X"]), "RTL_ERR_ARG"), (dict(Y=lambda a: at(a["Y0"], 16)), "RTL_ERR_ARG"), (dict(Y=lambda a: a["LA"]), "RTL_ERR_ARG"),
    (dict(Y=lambda a: a["plan"]), "RTL_ERR_ARG"), (dict(T=lambda a: a["Y"]), "RTL_ERR_ARG"), (dict(T=lambda a: a["Y0"]), "RTL_ERR_ARG"),
    (dict(Y=lambda a: a["ws"]), "RTL_ERR_ARG"),
], ids=label)
def test_adapters_refusals(over, want):
    st, b = adapters(**over)
    refused(st, want, b, over)


@pytest.mark.parametrize("over,want", ADAPTERS + [
    (dict(dX=None, dLA=None, dLB=None), "RTL_ERR_NULL"), (dict(dY=None), "RTL_ERR_NULL"), (dict(T=None), "RTL_ERR_NULL"),
    (dict(dyr=44), "RTL_ERR_ALIGN"), (dict(dxr=60), "RTL_ERR_ARG"), (dict(dX=lambda a: a["dY"]), "RTL_ERR_ARG"),
    (dict(dX=lambda a: a["X"]), "RTL_ERR_ARG"), (dict(dX=lambda a: at(a["dX0"], 16)), "RTL_ERR_ARG"),
    (dict(dLA=lambda a: a["dLB"]), "RTL_ERR_ARG"), (dict(dLB=lambda a: a["LB"]), "RTL_ERR_ARG"), (dict(dLA=lambda a: a["T"]), "RTL_ERR_ARG"),
    (dict(dX=lambda a: a["dLA"]), "RTL_ERR_ARG"), (dict(dLA=lambda a: a["ws"]), "RTL_ERR_ARG"),
], ids=label)
def test_adapters_backward_refusals(over, want):
    st, b = adapters(back=True, **over)
    refused(st, want, b, over)


@pytest.mark.parametrize("over,want", [
    (dict(M=0), "RTL_ERR_SHAPE"), (dict(A=0), "RTL_ERR_SHAPE"), (dict(A=5000), "RTL_ERR_SHAPE"), (dict(M=2 ** 31), "RTL_ERR_SHAPE"),
    (dict(ids=None), "RTL_ERR_NULL"), (dict(plan=None), "RTL_ERR_NULL"), (dict(ids=lambda a: at(a["ids"], 1)), "RTL_ERR_ALIGN"),
    (dict(plan=lambda a: at(a["plan"], 4)), "RTL_ERR_ALIGN"), (dict(pb=8), "RTL_ERR_ARG"), (dict(plan=lambda a: a["ids"]), "RTL_ERR_ARG"),
], ids=label)
def test_plan_refusals(over, want):
    b = Buffers()
    a = filled(dict(M=9, A=2, ids=b(512), plan=b(512), pb=rtl.rtl_adapters_plan_bytes(9, 2)), over)
    refused(rtl.lib.rtl_adapters_plan(a["M"], a["A"], a["ids"], a["plan"], a["pb"], None), want, b, over)


def adamw(bf16=False, eight=False, tensor=None, **over):
    b = Buffers()
    n = 600
    entry = dict(p=b(4 * n), g=b(4 * n), master=b(4 * n) if bf16 else None, m=b(4 * n), v=b(4 * n), m_scale=b(16) if eight else None,
                 v_scale=b(16) if eight else None, n=n)
    entries = [entry, dict(entry, **{k: None if entry[k] is None else b(4 * n) for k in entry if k != "n"})]
    filled(entries[1], {k: (lambda a, f=f: f(entries[0])) if callable(f) else f for k, f in (tensor or {}).items()})
    array = (rtl._AdamWTensor * 2)()
    for to, e in zip(array, entries):
        for k, v in e.items():
            setattr(to, k, v.value if isinstance(v, ctypes.c_void_p) else v)
    a = filled(dict(p_dt=rtl.RTL_BF16 if bf16 else rtl.RTL_F32, g_dt=rtl.RTL_F32, states=8 if eight else 32, count=2, tensors=array,
                    step=1, step_at=None, lr=1e-3, lr_at=None, b1=0.9, b2=0.999, eps=1e-8, wd=0.01, gs=None), over)
    return rtl.lib.rtl_adamw(*a.values(), None), b


@pytest.mark.parametrize("over,want", [
    (dict(p_dt=4), "RTL_ERR_UNSUPPORTED"), (dict(g_dt=-1), "RTL_ERR_UNSUPPORTED"), (dict(states=16), "RTL_ERR_UNSUPPORTED"),
    (dict(count=0), "RTL_ERR_SHAPE"), (dict(count=2 ** 40), "RTL_ERR_SHAPE"), (dict(tensors=None), "RTL_ERR_NULL"),
    (dict(step=0), "RTL_ERR_ARG"), (dict(step=-5), "RTL_ERR_ARG"), (dict(lr=float("nan")), "RTL_ERR_ARG"),
    (dict(lr=1e39), "RTL_ERR_ARG"), (dict(b1=1.0), "RTL_ERR_ARG"), (dict(b1=-0.1), "RTL_ERR_ARG"), (dict(b2=0.99999999999), "RTL_ERR_ARG"),
    (dict(eps=-1.0), "RTL_ERR_ARG"), (dict(wd=float("inf")), "RTL_ERR_ARG"), (dict(step_at=ctypes.c_void_p(4)), "RTL_ERR_ALIGN"),
    (dict(gs=ctypes.c_void_p(2)), "RTL_ERR_ALIGN"), (dict(tensor=dict(n=-1)), "RTL_ERR_SHAPE"), (dict(tensor=dict(n=2 ** 35 + 1)), "RTL_ERR_SHAPE"),
    (dict(tensor=dict(p=None)), "RTL_ERR_NULL"), (dict(tensor=dict(g=None)), "RTL_ERR_NULL"), (dict(tensor=dict(v=None)), "RTL_ERR_NULL"),
    (dict(bf16=True, tensor=dict(master=None)), "RTL_ERR_NULL"), (dict(eight=True, tensor=dict(m_scale=None)), "RTL_ERR_NULL"),
    (dict(p_dt=rtl.RTL_BF16), "RTL_ERR_NULL"), (dict(states=8), "RTL_ERR_NULL"),
    (dict(tensor=dict(p=lambda e: e["p"])), "RTL_ERR_ARG"), (dict(tensor=dict(m=lambda e: e["g"])), "RTL_ERR_ARG"),
    (dict(tensor=dict(v=lambda e: at(e["m"], 2384))), "RTL_ERR_ARG"), (dict(tensor=dict(p=lambda e: at(e["p"], 4))), "RTL_ERR_ALIGN"),
    (dict(eight=True, tensor=dict(v_scale=lambda e: at(e["v_scale"], 8))), "RTL_ERR_ARG"),
    (dict(eight=True, tensor=dict(v_scale=lambda e: at(e["v_scale"], 2))), "RTL_ERR_ALIGN"),
    (dict(bf16=True, tensor=dict(master=lambda e: e["master"])), "RTL_ERR_ARG"),
], ids=lambda v: v if isinstance(v, str) else ",".join(f"{k}={sorted(x)[0] if isinstance(x, dict) else str(x)[:12]}" for k, x in v.items()))
def test_adamw_refusals(over, want):
    st, b = adamw(**over)
    refused(st, want, b, over)


def test_sizes_of_plans_and_workspaces():
    assert rtl.rtl_adapters_plan_bytes(0, 1) == rtl.rtl_adapters_plan_bytes(1, 0) == rtl.rtl_adapters_plan_bytes(2 ** 24 + 1, 1) == 0
    assert rtl.rtl_adapters_plan_bytes(1, 4097) == 0
    # tables of two numbers an adapter, four words a tile, one a row
    assert rtl.rtl_adapters_plan_bytes(2 ** 24, 4096) == 4 * (8200 + 4 * (2 ** 18 + 4097) + 2 ** 24)
    for bad in ((0, 8, 8, 8, 1), (1, 4, 8, 8, 1), (1, 8, 12, 8, 1), (1, 8, 8, 136, 1), (1, 2 ** 22, 8, 128, 33)):
        assert rtl.rtl_adapters_workspace_bytes(*bad) == rtl.rtl_adapters_backward_workspace_bytes(*bad) == 0
    for M, K, N, R, A in ((1, 8, 8, 8, 1), (2 ** 24, 8, 8, 8, 4096), (70, 2 ** 22, 2 ** 22, 8, 2)):
        assert 0 < rtl.rtl_adapters_workspace_bytes(M, N, K, R, A)
        # the gradient's holds the turned factors and three operands besides
        assert rtl.rtl_adapters_backward_workspace_bytes(M, N, K, R, A) >= 2 * A * R * (K + N)
    for bad in ((0, 8, 1), (1, 0, 1), (1, 8, -1), (2 ** 31, 8, 1), (1, 32769, 1), (1, 1024, 2 ** 19)):
        assert rtl.rtl_layer_norm_backward_workspace_bytes(*bad) == 0
    assert rtl.rtl_layer_norm_backward_workspace_bytes(1, 8, 0) > 0


def test_python_refusals():
    x, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rtl.rtl_layer_norm(x)
    with pytest.raises(ValueError):
        rtl.rtl_adapters_plan(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        rtl.rtl_adapters(x, f, f.transpose(0, 1), x)
    t = [torch.zeros(300)]
    for bad in (dict(params=[]), dict(grads=t * 2), dict(masters=t), dict(m_scales=t), dict(m=[t[0].to(torch.float8_e4m3fn)])):
        with pytest.raises(ValueError):
            rtl.rtl_adamw_tensors(**{**dict(params=t, grads=t, m=t, v=t), **bad})
    with pytest.raises(TypeError):
        rtl.rtl_adamw_tensors([t[0].half()], t, t, t)
