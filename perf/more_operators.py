"""Layer norm with per-request modulation, low-rank adapters of many requests beside a shared
projection, their gradients, and the AdamW step over many tensors: the cases on which they are
timed and compared.

``run`` computes an operator in its plain form, elementary torch operations in 32 bits with
one rounding at the end, or, where ``own`` is set, calls the library.  ``exact`` is the
definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # The norm in front of a projection for one token, with its request's scale and shift.  The
        # smallest call: its latency counts.
        dict(name="norm_one_token", op="norm", dtype="bf16", M=1, D=5120, affine=False, G=1, ragged=False, stats=False),
        # The tokens of several videos in one batch, each with its own scale and shift: the largest call.
        dict(name="norm_video", op="norm", dtype="bf16", M=32760, D=5120, affine=False, G=4, ragged=True, stats=False),
        # Gradients in fp32 at an odd width, rows that no 16-byte access reaches whole.
        dict(name="norm_backward_odd", op="norm_backward", dtype="f32", M=333, D=1153, affine=True, G=0, ragged=False),
        # Gradients of the batch of videos: tokens, weights, and every request's scale and shift.
        dict(name="norm_backward_video", op="norm_backward", dtype="bf16", M=32760, D=5120, affine=True, G=4,
             ragged=True),
        # A few rows of as many requests (one conditioning token each) through a wide projection, most
        # with an adapter of their own: the factors are streamed once.
        dict(name="adapters_tokens", op="adapters", M=24, K=5120, N=13824, R=32, A=16, mix="rows", bare=0.1,
             packed=False, keep=False),
        # Images of eight requests in one batch, beside a projection that lies in a packed output.
        dict(name="adapters_images", op="adapters", M=4608, K=2560, N=7680, R=64, A=8, mix="runs", bare=0.1,
             packed=True, keep=False),
        # The tokens of a video batch: the largest product.
        dict(name="adapters_video", op="adapters", M=32760, K=5120, N=5120, R=64, A=4, mix="runs", bare=0.0,
             packed=False, keep=True),
        # Gradients for one image's tokens, three adapters of a low rank trained together.
        dict(name="adapters_backward_image", op="adapters_backward", M=4173, K=2560, N=6912, R=16, A=3, mix="runs",
             bare=0.1),
        # Gradients for half a video batch.
        dict(name="adapters_backward_video", op="adapters_backward", M=16380, K=5120, N=5120, R=64, A=2, mix="runs",
             bare=0.0),
        # The norm weights of one block, fp32: the smallest step.
        dict(name="adamw_norms", op="adamw", sizes="128,128,2560,2560", repeat=1, param="f32", grad="f32", bits=32,
             step=1, clip=False),
        # The low-rank factors of forty blocks' four projections in bf16 beside fp32 masters.
        dict(name="adamw_factors", op="adamw", sizes="983040,327680,327680,327680,884736,327680,327680,884736", repeat=40,
             param="bf16", grad="bf16", bits=32, step=100, clip=True),
        # The weights of a gated block, a few large tensors, states in 8 bits.
        dict(name="adamw_block_8bit", op="adamw", sizes="70778880,70778880,70778880", repeat=1, param="bf16",
             grad="bf16", bits=8, step=1000, clip=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "adapters", "adapters_backward", "adamw"])
    if op in ("norm", "norm_backward"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        D = _spread(rng, 64, 13824 if dtype == "bf16" else 8192)
        D = max(8, D - D % 8) if rng.random() < 0.8 else min(D, 4096)
        M = _spread(rng, 1, min(32760, 32760 * 5120 // D // (1 if dtype == "bf16" else 2)))
        G = rng.choice([0, 1, _spread(rng, 1, min(M, 64))])
        case = dict(op=op, dtype=dtype, M=M, D=D, affine=G == 0 or rng.random() < 0.4, G=G, ragged=rng.random() < 0.6)
        if op == "norm":
            case["stats"] = rng.random() < 0.4
        return case
    if op in ("adapters", "adapters_backward"):
        K, N = 8 * _spread(rng, 8, 1728), 8 * _spread(rng, 8, 1728)
        mix = rng.choice(["rows", "runs", "runs"])
        if mix == "rows":  # single rows of many requests
            M, A = _spread(rng, 1, 512), _spread(rng, 1, 64)
        else:
            M, A = min(_spread(rng, 16, 32760), 16380 * 10240 // (K + N)), _spread(rng, 1, 8)
        case = dict(op=op, M=M, K=K, N=N, R=8 * _spread(rng, 1, 16), A=A, mix=mix, bare=rng.choice([0.0, 0.1, 0.5]))
        if op == "adapters":
            case.update(packed=rng.random() < 0.4, keep=rng.random() < 0.4)
        return case
    count = _spread(rng, 1, 60)
    total = _spread(rng, 100, 150000000)
    sizes = [max(1, int(total / count * math.exp(rng.gauss(0, 0.7)) / 1.6)) for _ in range(count)]
    return dict(op=op, sizes=",".join(map(str, sizes)), repeat=1, param=rng.choice(["f32", "bf16"]),
                grad=rng.choice(["f32", "bf16"]), bits=rng.choice([8, 32]), step=rng.choice([1, 2, 10, 1000, 100000]),
                clip=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

EPS = 1e-6
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.01
BLOCK = 256  # elements that share a scale where states are held in 8 bits


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """Token activations, a few percent of whose channels are large."""
    large = torch.rand(M, K, generator=g, device="cuda") < 0.08
    return _normal(g, M, K) * torch.where(large, 3.0, 0.1)


def _cuts(g, M, G, ragged):
    """Ascending offsets [G + 1] of G groups over M rows; ragged ones may be empty."""
    if not ragged:
        return torch.arange(G + 1, device="cuda") * M // G
    inner = torch.randint(0, M + 1, (G - 1,), generator=g, device="cuda").sort().values
    return torch.cat([inner.new_zeros(1), inner, inner.new_full((1,), M)])


def _norm_inputs(case, g):
    dt, M, D, G = _DTYPES[case["dtype"]], case["M"], case["D"], case["G"]
    # a residual stream: channels of different size, some of them off centre
    gain, centre = torch.exp(0.5 * _normal(g, D)), 0.5 * _normal(g, D)
    s = dict(X=(_activations(g, M, D) * gain + centre).to(dt))
    if case["affine"]:
        s["weight"], s["bias"] = (1 + 0.2 * _normal(g, D)).to(dt), (0.1 * _normal(g, D)).to(dt)
    if G:
        # scale and shift are two of the six parts of the modulation's projection
        parts = (0.3 * _normal(g, G, 6 * D)).to(dt)
        s["shift"], s["scale"] = parts[:, :D], parts[:, D:2 * D]
        s["groups"] = _cuts(g, M, G, case["ragged"]).to(torch.int32)
    if case["op"] == "norm_backward":
        s["dY"] = (0.1 * _normal(g, M, D)).to(dt)
        x = s["X"].double()  # what the forward pass kept
        mean = x.mean(dim=1)
        s["stats"] = torch.stack([mean, torch.rsqrt(x.var(dim=1, unbiased=False) + EPS)], dim=1).float()
    return s


def _adapter_inputs(case, g):
    M, K, N, R, A = (case[n] for n in "MKNRA")
    bf16 = torch.bfloat16
    s = dict(X=_activations(g, M, K).to(bf16), LB=(_normal(g, A, R, K) * K ** -0.5).to(bf16),
             LA=(_normal(g, A, N, R) * R ** -0.5).to(bf16), alpha=0.5 + torch.rand(A, generator=g, device="cuda"))
    if case["mix"] == "rows":
        request = torch.arange(M, device="cuda")
    else:  # requests of different lengths, one after another
        cuts = _cuts(g, M, min(M, 2 * A), True)
        request = torch.searchsorted(cuts[1:], torch.arange(M, device="cuda"), right=True)
    adapter = torch.randint(0, A, (M,), generator=g, device="cuda")
    adapter[torch.rand(M, generator=g, device="cuda") < case["bare"]] = -1
    s["ids"] = adapter[request].to(torch.int32)
    if case["op"] == "adapters":
        wide = _normal(g, M, (2 if case["packed"] else 1) * N).to(bf16)
        s["Y0"] = wide[:, wide.shape[1] - N:]
    else:
        s["dY"], s["dX0"] = (0.1 * _normal(g, M, N)).to(bf16), (0.1 * _normal(g, M, K)).to(bf16)
        rows = _rows(s["ids"], A)
        T = _padded(s["X"].double(), rows) @ s["LB"].double().transpose(1, 2).contiguous()  # what the forward pass kept
        s["T"] = _spread_rows(T.float(), rows, M)
    return s


def _rows(ids, A):
    """Each adapter's rows [A, P], filled up with the number of rows."""
    M = ids.shape[0]
    order = torch.sort(torch.where(ids < 0, A, ids), stable=True).indices
    counts = torch.bincount(torch.where(ids < 0, A, ids), minlength=A + 1)[:A]
    starts = torch.cumsum(counts, 0) - counts
    place = torch.arange(max(1, int(counts.max())), device=ids.device)
    at = (starts[:, None] + place).clamp_(max=M - 1)
    return torch.where(place < counts[:, None], order[at], M)


def _padded(x, rows):
    """x's rows [M, C] as [A, P, C], zeros in the places that hold none."""
    return torch.cat([x, x.new_zeros(1, x.shape[1])])[rows]


def _spread_rows(x, rows, M):
    """[A, P, C] back to the rows they belong to; zeros for the others."""
    out = x.new_zeros(M + 1, x.shape[-1])
    out[rows.flatten()] = x.flatten(0, 1)
    return out[:M]


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")] * case["repeat"]


def _step_inputs(case, g):
    """The tensors are views of one buffer for each of their kinds, at whole blocks."""
    sizes, bits = _sizes(case), case["bits"]
    room = [-(-n // BLOCK) * BLOCK for n in sizes]
    inside = torch.repeat_interleave(torch.tensor(room, device="cuda"))
    starts = torch.cumsum(torch.tensor([0] + room[:-1], device="cuda"), 0)
    inside = torch.arange(sum(room), device="cuda") - starts[inside] < torch.tensor(sizes, device="cuda")[inside]
    master = 0.02 * _normal(g, sum(room)) * inside
    # gradients and states of the sizes that a run reaches: elements differ by orders of magnitude
    size = 1e-3 * torch.exp(_normal(g, sum(room))) * inside
    grad = (size * _normal(g, sum(room))).to(_DTYPES[case["grad"]])
    if case["step"] == 1:
        m, u = torch.zeros_like(size), torch.zeros_like(size)
    else:
        m, u = 0.2 * size * _normal(g, sum(room)), size * (0.7 + 0.6 * torch.rand(sum(room), generator=g, device="cuda"))
    whole = dict(grads=grad)
    if case["param"] == "bf16":
        whole["params"], whole["masters"] = master.to(torch.bfloat16), master
    else:
        whole["params"] = master
    if bits == 32:
        whole["m"], whole["v"] = m, u * u
    else:
        whole["m"], whole["m_scales"] = (t.flatten() for t in _code(m.view(-1, BLOCK), False))
        whole["v"], whole["v_scales"] = (t.flatten() for t in _code(u.view(-1, BLOCK), True))
    s = dict(whole=whole)
    if case["clip"]:
        s["clip"] = torch.rand(1, generator=g, device="cuda") + 0.25
    return s


def _tensors(case, whole):
    """Each kind's tensors, as views of its buffer."""
    sizes = _sizes(case)
    blocks = [-(-n // BLOCK) for n in sizes]
    return {name: list(t.split(blocks)) if name.endswith("scales") else
            [v[:n] for v, n in zip(t.split([b * BLOCK for b in blocks]), sizes)] for name, t in whole.items()}


def _code(b, root):
    """Blocks [n, BLOCK] in 32 bits to E4M3 values and scales [n, 1]; a root that is not 0 is not coded as 0."""
    most = b.abs().amax(dim=1, keepdim=True)
    inverse = torch.full_like(most, 448.0) / most
    scaled = b * torch.where(torch.isfinite(inverse), inverse, torch.zeros_like(inverse))
    if root:
        scaled = torch.where(b > 0, scaled.clamp(min=2.0 ** -9), scaled)
    return scaled.to(torch.float8_e4m3fn), most / torch.full_like(most, 448.0)


def _inputs(case, seed):
    g, op = _generator(seed), case["op"]
    if op in ("norm", "norm_backward"):
        return _norm_inputs(case, g)
    if op in ("adapters", "adapters_backward"):
        return _adapter_inputs(case, g)
    return _step_inputs(case, g)


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if "ids" in state:
        state["rows"] = _rows(state["ids"], case["A"])
    if own:
        import activation_sparse_gemm_amd as rtl

        # what a program keeps: the batch's plan, which all its layers share, and the optimizer's list
        if "ids" in state:
            state["plan"] = rtl.rtl_adapters_plan(state["ids"], case["A"])
        if case["op"] == "adamw":
            state["list"] = rtl.rtl_adamw_tensors(**_tensors(case, state["whole"]))
    return state


# ---------------------------------------------------------------- one pass


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "adapters": _plain_adapters,
            "adapters_backward": _plain_adapters_backward, "adamw": _plain_adamw}[state["case"]["op"]](state)


def _run_own(s):
    import activation_sparse_gemm_amd as rtl

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        stats = torch.empty((case["M"], 2), dtype=torch.float32, device="cuda") if case["stats"] else None
        Y = rtl.rtl_layer_norm(s["X"], s.get("weight"), s.get("bias"), s.get("scale"), s.get("shift"), s.get("groups"),
                               eps=EPS, stats=stats)
        return (Y, stats) if case["stats"] else Y
    if op == "norm_backward":
        got = rtl.rtl_layer_norm_backward(s["X"], s["stats"], s["dY"], s.get("weight"), s.get("bias"), s.get("scale"),
                                          s.get("groups"))
        return [t for t in got if t is not None]
    if op == "adapters":
        T = torch.empty((case["M"], case["R"]), dtype=torch.float32, device="cuda") if case["keep"] else None
        Y = rtl.rtl_adapters(s["X"], s["LA"], s["LB"], s["plan"], s["alpha"], Y0=s["Y0"], T=T)
        return (Y, T) if case["keep"] else Y
    if op == "adapters_backward":
        return rtl.rtl_adapters_backward(s["X"], s["LA"], s["LB"], s["plan"], s["T"], s["dY"], s["alpha"], dX0=s["dX0"])
    rtl.rtl_adamw(s["list"], step=case["step"], lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY,
                  grad_scale=s.get("clip"))
    return _changed(s)


def _changed(s):
    return {n: t for n, t in s["whole"].items() if n != "grads"}


def _of_rows(s):
    """Each row's group."""
    M = s["case"]["M"]
    return torch.searchsorted(s["groups"][1:].long(), torch.arange(M, device="cuda"), right=True)


def _plain_norm(s):
    x = s["X"].float()
    mean = x.mean(dim=1, keepdim=True)
    d = x - mean
    r = torch.rsqrt((d * d).mean(dim=1, keepdim=True) + EPS)
    y = d * r
    if "weight" in s:
        y = y * s["weight"].float() + s["bias"].float()
    if "scale" in s:
        row = _of_rows(s)
        y = y * (1 + s["scale"].float())[row] + s["shift"].float()[row]
    y = y.to(s["X"].dtype)
    return (y, torch.cat([mean, r], dim=1)) if s["case"]["stats"] else y


def _plain_norm_backward(s):
    x, dy, r = s["X"].float(), s["dY"].float(), s["stats"][:, 1:]
    n = (x - s["stats"][:, :1]) * r
    c, sums = dy, []
    if "scale" in s:
        row, D, G = _of_rows(s), s["case"]["D"], s["case"]["G"]
        y = n * s["weight"].float() + s["bias"].float() if "weight" in s else n
        zeros = torch.zeros(G, D, device="cuda")
        sums = [zeros.index_add(0, row, dy * y), zeros.index_add(0, row, dy)]
        c = dy * (1 + s["scale"].float())[row]
    g = c
    if "weight" in s:
        sums = [(c * n).sum(dim=0), c.sum(dim=0)] + sums
        g = c * s["weight"].float()
    dx = r * (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True))
    return [dx.to(s["X"].dtype)] + sums


def _plain_adapters(s):
    case, rows = s["case"], s["rows"]
    T = torch.bmm(_padded(s["X"].float(), rows), s["LB"].float().transpose(1, 2).contiguous())
    Y = torch.bmm(T * s["alpha"][:, None, None], s["LA"].float().transpose(1, 2).contiguous())
    Y = (s["Y0"].float() + _spread_rows(Y, rows, case["M"])).to(torch.bfloat16)
    return (Y, _spread_rows(T, rows, case["M"])) if case["keep"] else Y


def _plain_adapters_backward(s):
    rows, M = s["rows"], s["case"]["M"]
    scaled = _padded(s["dY"].float(), rows) * s["alpha"][:, None, None]
    dT = torch.bmm(scaled, s["LA"].float())
    dX = s["dX0"].float() + _spread_rows(torch.bmm(dT, s["LB"].float()), rows, M)
    dLB = torch.bmm(dT.transpose(1, 2).contiguous(), _padded(s["X"].float(), rows))
    dLA = torch.bmm(scaled.transpose(1, 2).contiguous(), _padded(s["T"], rows))
    return dX.to(torch.bfloat16), dLA, dLB


def _plain_adamw(s):
    case, whole = s["case"], s["whole"]
    g, p = whole["grads"].float(), whole.get("masters", whole["params"])
    m, v = whole["m"].float(), whole["v"].float()
    if "clip" in s:
        g = g * s["clip"]
    if case["bits"] == 8:
        m = (m.view(-1, BLOCK) * whole["m_scales"][:, None]).flatten()
        u = (v.view(-1, BLOCK) * whole["v_scales"][:, None]).flatten()
        v = u * u
    m = m + (g - m) * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    u = torch.sqrt(v)
    step = m * (1 / (1 - BETA1 ** case["step"])) / (u * (1 / math.sqrt(1 - BETA2 ** case["step"])) + ADAM_EPS)
    p.sub_((step + p * DECAY) * LR)
    if "masters" in whole:
        whole["params"].copy_(p)
    if case["bits"] == 8:
        for x, codes, root in ((m, "m", False), (u, "v", True)):
            code, scale = _code(x.view(-1, BLOCK), root)
            whole[codes].copy_(code.flatten())
            whole[codes + "_scales"].copy_(scale.flatten())
    else:
        whole["m"].copy_(m)
        whole["v"].copy_(v)
    return _changed(s)


# ---------------------------------------------------------------- work, and the exact outputs


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        size, n, D, G = 2 if case["dtype"] == "bf16" else 4, case["M"] * case["D"], case["D"], case["G"]
        small = ((2 if case["affine"] else 0) + 2 * G) * D
        if op == "norm":
            return {"bytes": 2 * n * size + small * size + (8 * case["M"] if case["stats"] else 0), "flops": 8 * n}
        return {"bytes": 3 * n * size + small * (size + 4) + 8 * case["M"], "flops": 16 * n}
    if op in ("adapters", "adapters_backward"):
        M, K, N, R = (case[n] for n in "MKNR")
        met = M * (1 - case["bare"])
        used = min(case["A"], max(1, math.ceil(met)))
        if op == "adapters":  # X, Y0 and Y; the factors of the adapters that are met
            return {"bytes": 2 * M * (K + 2 * N) + 2 * used * R * (K + N) + (4 * M * R if case["keep"] else 0),
                    "flops": 2 * met * R * (K + N)}
        # X, dX0, dX, dY, the factors, T; the factors' gradients in 32 bits
        return {"bytes": 2 * M * (3 * K + N) + 2 * used * R * (K + N) + 4 * M * R + 4 * case["A"] * R * (K + N),
                "flops": 4 * met * R * (K + N)}
    n, wide = sum(_sizes(case)), {"bf16": 2, "f32": 4}
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * ((8 if case["param"] == "f32" else 8 + 2) + wide[case["grad"]] + states), "flops": 15 * n}


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(case, s["whole"], float(s.get("clip", 1.0)))
    groups, ids = s.get("groups"), s.get("ids")
    s = {k: v.double() for k, v in s.items()}
    if op in ("norm", "norm_backward"):
        return _exact_norm(case, s, groups)
    return _exact_adapters(case, s, ids)


def _exact_norm(case, s, groups):
    M, D = case["M"], case["D"]
    w, b = s.get("weight", torch.ones(D, device="cuda", dtype=torch.float64)), s.get("bias", 0.0)
    if case["op"] == "norm":
        var, mean = torch.var_mean(s["X"], dim=1, correction=0)
        size = torch.sqrt(var + EPS)
        y = (s["X"] - mean[:, None]) / size[:, None] * w + b
        if groups is not None:
            for g, (lo, hi) in enumerate(zip(groups.tolist()[:-1], groups.tolist()[1:])):
                y[lo:hi] = y[lo:hi] * (1 + s["scale"][g]) + s["shift"][g]
        return (y, torch.stack([mean, 1 / size], dim=1)) if case["stats"] else y
    mean, r = s["stats"][:, 0], s["stats"][:, 1]
    unit = (s["X"] - mean[:, None]) * r[:, None]
    up, dscale, dshift = s["dY"].clone(), [], []
    if groups is not None:
        for g, (lo, hi) in enumerate(zip(groups.tolist()[:-1], groups.tolist()[1:])):
            dscale.append((s["dY"][lo:hi] * (unit[lo:hi] * w + b)).sum(dim=0))
            dshift.append(s["dY"][lo:hi].sum(dim=0))
            up[lo:hi] *= 1 + s["scale"][g]
    out = [(up * unit).sum(dim=0), up.sum(dim=0)] if "weight" in s else []
    out += [torch.stack(dscale), torch.stack(dshift)] if groups is not None else []
    up *= w
    along = (up * unit).sum(dim=1, keepdim=True) / D
    return [(up - up.sum(dim=1, keepdim=True) / D - unit * along) * r[:, None]] + out


def _exact_adapters(case, s, ids):
    back = case["op"] == "adapters_backward"
    first = s["dX0"].clone() if back else s["Y0"].clone()
    T = torch.zeros(case["M"], case["R"], device="cuda", dtype=torch.float64)
    dLA, dLB = torch.zeros_like(s["LA"]), torch.zeros_like(s["LB"])
    for a in range(case["A"]):
        rows = torch.nonzero(ids == a).flatten()
        if back:
            dy = s["dY"][rows] * s["alpha"][a]
            dt = dy @ s["LA"][a]
            first[rows] += dt @ s["LB"][a]
            dLA[a], dLB[a] = dy.t() @ s["T"][rows], dt.t() @ s["X"][rows]
        else:
            T[rows] = s["X"][rows] @ s["LB"][a].t()
            first[rows] += s["alpha"][a] * (T[rows] @ s["LA"][a].t())
    if back:
        return first, dLA, dLB
    return (first, T) if case["keep"] else first


def _round_e4m3(x):
    """The nearest E4M3 value, ties to the even one."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(max=8)
    step = torch.exp2(exponent - 3)
    return torch.round(x / step) * step


def _exact_adamw(case, s, rate):
    t, n = case["step"], s["grads"].numel()
    p, g, m, v = s.get("masters", s["params"]).double(), s["grads"].double() * rate, s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m = m * s["m_scales"].double().repeat_interleave(BLOCK)
        v = (v * s["v_scales"].double().repeat_interleave(BLOCK)) ** 2
    m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    ahead = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
    p = p - LR * DECAY * p - LR * ahead
    out = dict(params=p)
    if "masters" in s:
        out["masters"] = p
    if case["bits"] == 32:
        return dict(out, m=m, v=v)
    for x, codes in ((m, "m"), (v.sqrt(), "v")):
        most = x.abs().view(-1, BLOCK).amax(dim=1)
        scaled = x * (448 / most).repeat_interleave(BLOCK)
        rounded = _round_e4m3(torch.where(torch.isfinite(scaled), scaled, 0.0))
        if codes == "v":
            rounded = torch.where((x > 0) & (rounded == 0), 2.0 ** -9, rounded)
        out[codes], out[codes + "_scales"] = rounded, most / 448
    return out
