"""Rotary positions over several axes, per-head norms of queries and keys with the rotation,
and the gated feed-forward block: the cases on which they are timed and compared.

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
        # The rotation alone, taken back (the gradient of a rotation): a caption's tokens, in the
        # layout that pairs channel i with i + 36, in fp32.  A small call: its latency counts.
        dict(name="rope_caption", op="rope", dtype="f32", M=77, H=6, D=80, dims="8,32,32", pairs="halves",
             inverse=True, packed=False, text=0, wide=9, high=9, scale=1.0, far=0, theta=10000.0),
        # The rotation of the queries of a video block (21 x 30 x 52 latent tokens, 40 heads), a
        # strided view of the packed qkv projection.
        dict(name="rope_video", op="rope", dtype="bf16", M=32760, H=40, D=128, dims="44,42,42", pairs="adjacent",
             inverse=False, packed=True, text=0, wide=52, high=30, scale=1.0, far=0, theta=10000.0),
        # Norm and rotation of one token's queries and keys: the smallest call.
        dict(name="qk_one_token", op="qk", dtype="bf16", M=1, Hq=24, Hk=24, D=128, dims="16,56,56",
             pairs="adjacent", packed=True, text=0, wide=64, high=64, scale=1.0, far=0, theta=10000.0),
        # A text-to-image block: 512 text tokens and 64 x 64 image tokens, 24 heads.
        dict(name="qk_image", op="qk", dtype="bf16", M=4608, Hq=24, Hk=24, D=128, dims="16,56,56",
             pairs="adjacent", packed=True, text=512, wide=64, high=64, scale=1.0, far=0, theta=10000.0),
        # The video block's queries and keys: the largest call.
        dict(name="qk_video", op="qk", dtype="bf16", M=32760, Hq=40, Hk=40, D=128, dims="44,42,42",
             pairs="adjacent", packed=True, text=0, wide=52, high=30, scale=1.0, far=0, theta=10000.0),
        # Gradients at the text-to-image block, keys shared by three queries each.
        dict(name="qk_backward_image", op="qk_backward", dtype="bf16", M=4608, Hq=24, Hk=8, D=128, dims="16,56,56",
             pairs="adjacent", packed=True, text=512, wide=64, high=64, scale=1.0, far=0, theta=10000.0),
        # Gradients in fp32 at odd sizes, positions far out and between the grid's points, some
        # channels left unrotated.
        dict(name="qk_backward_odd", op="qk_backward", dtype="f32", M=777, Hq=6, Hk=2, D=96, dims="16,24,24",
             pairs="halves", packed=False, text=7, wide=31, high=17, scale=0.75, far=100000, theta=256.0),
        # The gated block for one token: both weights are streamed once.
        dict(name="glu_one_token", op="glu", dtype="bf16", M=1, K=5120, H=13824, act="silu", save=False),
        # A training pass over one image's tokens, pre-activations kept for the backward pass;
        # ragged token count and width.
        dict(name="glu_image_train", op="glu", dtype="bf16", M=4173, K=2560, H=6916, act="gelu", save=True),
        # The video block's tokens: the largest product.
        dict(name="glu_video", op="glu", dtype="bf16", M=32760, K=5120, H=13824, act="silu", save=False),
        # Gradients for a few text tokens, where few rows meet whole weights.
        dict(name="glu_backward_text", op="glu_backward", dtype="bf16", M=333, K=2560, H=6912, act="silu"),
        # Gradients for a quarter of the video block's tokens.
        dict(name="glu_backward_video", op="glu_backward", dtype="bf16", M=8190, K=5120, H=13824, act="gelu"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "qk", "qk_backward", "glu", "glu_backward"])
    if op in ("glu", "glu_backward"):
        K = 64 * _spread(rng, 1, 80)
        H = _spread(rng, 32, 13824)
        if rng.random() < 0.5:
            H = max(8, H - H % 8)
        M = min(_spread(rng, 1, 32760), 32760 * 5120 * 13824 // (K * H))
        case = dict(op=op, dtype="bf16", M=M, K=K, H=H, act=rng.choice(["silu", "gelu"]))
        if op == "glu":
            case["save"] = rng.random() < 0.5
        else:
            case["M"] = min(M, 8190)
        return case
    D = rng.choice([32, 64, 72, 80, 96, 128, 128, 160, 256])
    pairs = rng.choice(["adjacent", "halves"])
    rotated = 8 * rng.randint(max(1, D // 16), D // 8)
    axes = rng.randint(1, 4)
    cuts = sorted(rng.sample(range(1, rotated // 2), axes - 1)) if rotated // 2 > axes else []
    ends = [0] + cuts + [rotated // 2]
    dims = ",".join(str(2 * (b - a)) for a, b in zip(ends, ends[1:]))
    heads = _spread(rng, 1, 40)
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), M=0, D=D, dims=dims, pairs=pairs,
                packed=rng.random() < 0.7, wide=rng.randint(1, 64), high=rng.randint(1, 64),
                scale=rng.choice([1.0, 1.0, 0.75]), far=rng.choice([0, 0, 1000, 100000]),
                theta=rng.choice([256.0, 10000.0, 1000000.0]))
    if op == "rope":
        case.update(H=heads, inverse=rng.random() < 0.5)
        channels = heads * D
    else:
        case.update(Hq=heads, Hk=rng.choice([h for h in range(1, heads + 1) if heads % h == 0]))
        channels = (case["Hq"] + case["Hk"]) * D
    most = 32760 * 40 * 128 // channels if case["dtype"] == "bf16" else 32760 * 20 * 128 // channels
    case["M"] = _spread(rng, 1, min(32760, max(1, most)))
    case["text"] = rng.randint(0, case["M"] // 4)
    return case


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """Token activations, a few percent of whose channels are large."""
    large = torch.rand(M, K, generator=g, device="cuda") < 0.08
    return (_normal(g, M, K) * torch.where(large, 3.0, 0.1)).to(torch.bfloat16)


def _positions(case, seed):
    """Text tokens at the origin, then a grid in row-major order of (time, height, width),
    moved by the seed; the width is the last axis."""
    axes = len(case["dims"].split(","))
    i = torch.arange(case["M"], device="cuda") - case["text"]
    w, h, t = i % case["wide"], i // case["wide"] % case["high"], i // (case["wide"] * case["high"])
    grid = torch.stack([torch.zeros_like(t), t, h, w][-axes:] if axes > 1 else [i], dim=1).to(torch.float64)
    start = torch.tensor([case["far"]] + [0] * (axes - 1), device="cuda", dtype=torch.float64) + seed % 5
    pos = grid * case["scale"] + start
    pos[i < 0] = 0
    return pos.to(torch.float32).contiguous()


def _heads(case, g, counts):
    """[M, heads, D] tensors side by side: views of one packed projection, or each its own."""
    dt, M, D = _DTYPES[case["dtype"]], case["M"], case["D"]
    gain = torch.exp(0.5 * _normal(g, D))  # channels of a head differ in size
    parts = [(_normal(g, M, n, D) * gain).to(dt) for n in counts]
    if not case["packed"]:
        return parts
    parts.append(torch.zeros(M, counts[-1], D, device="cuda", dtype=dt))  # the values, beside them
    whole = torch.cat(parts, dim=1)
    out, at = [], 0
    for n in counts:
        out.append(whole[:, at:at + n])
        at += n
    return out


def _inputs(case, seed):
    g, op = _generator(seed), case["op"]
    if op in ("glu", "glu_backward"):
        M, K, H = case["M"], case["K"], case["H"]
        s = dict(X=_activations(g, M, K), Wg=(_normal(g, H, K) * K ** -0.5).to(torch.bfloat16),
                 Wu=(_normal(g, H, K) * K ** -0.5).to(torch.bfloat16))
        if op == "glu_backward":
            # the pre-activations that the forward pass left, and the gradient from above
            s["G"], s["U"] = torch.mm(s["X"], s["Wg"].t()), torch.mm(s["X"], s["Wu"].t())
            s["dY"] = (_normal(g, M, H) * 0.01).to(torch.bfloat16)
        return s
    s = dict(pos=_positions(case, seed))
    if op == "rope":
        s["X"], = _heads(case, g, [case["H"]])
        return s
    dt, D = _DTYPES[case["dtype"]], case["D"]
    s["Q"], s["K"] = _heads(case, g, [case["Hq"], case["Hk"]])
    s["qw"], s["kw"] = (1 + 0.2 * _normal(g, D)).to(dt), (1 + 0.2 * _normal(g, D)).to(dt)
    if op == "qk_backward":
        s["dQ"] = (0.1 * _normal(g, case["M"], case["Hq"], D)).to(dt)
        s["dK"] = (0.1 * _normal(g, case["M"], case["Hk"], D)).to(dt)
    return s


EPS = 1e-6


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if "dims" in case:
        state["dims"] = [int(d) for d in case["dims"].split(",")]
    return state


# ---------------------------------------------------------------- one pass


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "qk": _plain_qk, "qk_backward": _plain_qk_backward, "glu": _plain_glu,
            "glu_backward": _plain_glu_backward}[state["case"]["op"]](state)


def _run_own(s):
    import activation_sparse_gemm_amd as rtl

    case, op = s["case"], s["case"]["op"]
    if op in ("glu", "glu_backward"):
        act = {"silu": rtl.RTL_ACT_SILU, "gelu": rtl.RTL_ACT_GELU}[case["act"]]
        if op == "glu_backward":
            return rtl.rtl_glu_backward(s["X"], s["Wg"], s["Wu"], s["G"], s["U"], s["dY"], act=act)
        if not case["save"]:
            return rtl.rtl_glu_fused(s["X"], s["Wg"], s["Wu"], act=act)
        G = torch.empty((case["M"], case["H"]), dtype=torch.bfloat16, device="cuda")
        U = torch.empty_like(G)
        return rtl.rtl_glu_fused(s["X"], s["Wg"], s["Wu"], act=act, G=G, U=U), G, U
    pairs = {"adjacent": rtl.RTL_ROPE_ADJACENT, "halves": rtl.RTL_ROPE_HALVES}[case["pairs"]]
    how = dict(theta=case["theta"], pairs=pairs)
    if op == "rope":
        return rtl.rtl_rope_axes(s["X"], s["pos"], s["dims"], inverse=case["inverse"], **how)
    if op == "qk":
        return rtl.rtl_qk_norm_rope(s["Q"], s["K"], s["qw"], s["kw"], s["pos"], s["dims"], eps=EPS, **how)
    return rtl.rtl_qk_norm_rope_backward(s["Q"], s["K"], s["qw"], s["kw"], s["pos"], s["dims"], s["dQ"], s["dK"],
                                         eps=EPS, **how)


def _cos_sin(s):
    """cos and sin of every pair's angle [M, 1, pairs], the angles in 64 bits."""
    parts = []
    for a, d in enumerate(s["dims"]):
        freq = s["case"]["theta"] ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
        parts.append(s["pos"][:, a:a + 1].double() * freq)
    angle = torch.cat(parts, dim=1)[:, None, :]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(x, cos, sin, pairs):
    """x [M, heads, D] in 32 bits; the first 2 * pairs channels are rotated."""
    n = 2 * cos.shape[-1]
    turned, rest = x[..., :n], x[..., n:]
    if pairs == "adjacent":
        x0, x1 = turned[..., 0::2], turned[..., 1::2]
        out = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], dim=-1).flatten(-2)
    else:
        x0, x1 = turned[..., :n // 2], turned[..., n // 2:]
        out = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], dim=-1)
    return torch.cat([out, rest], dim=-1)


def _plain_rope(s):
    cos, sin = _cos_sin(s)
    if s["case"]["inverse"]:
        sin = -sin
    return _rotate(s["X"].float(), cos, sin, s["case"]["pairs"]).to(s["X"].dtype)


def _plain_qk(s):
    cos, sin = _cos_sin(s)
    out = []
    for x, w in ((s["Q"], s["qw"]), (s["K"], s["kw"])):
        x = x.float()
        n = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w.float()
        out.append(_rotate(n, cos, sin, s["case"]["pairs"]).to(s["Q"].dtype))
    return tuple(out)


def _plain_qk_backward(s):
    cos, sin = _cos_sin(s)
    dx, dw = [], []
    for x, w, dy in ((s["Q"], s["qw"], s["dQ"]), (s["K"], s["kw"], s["dK"])):
        x, w = x.float(), w.float()
        r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
        dn = _rotate(dy.float(), cos, -sin, s["case"]["pairs"])
        dw.append((dn * x * r).sum(dim=(0, 1)))
        t = dn * w
        dx.append((r * t - x * r ** 3 * (t * x).mean(dim=-1, keepdim=True)).to(s["Q"].dtype))
    return tuple(dx + dw)


def _activation(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return g * 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))


def _activation_slope(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return p * (1 + g * (1 - p))
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _plain_glu(s):
    x = s["X"].float()
    g, u = x @ s["Wg"].float().t(), x @ s["Wu"].float().t()
    y = (_activation(g, s["case"]["act"]) * u).to(torch.bfloat16)
    return (y, g.to(torch.bfloat16), u.to(torch.bfloat16)) if s["case"]["save"] else y


def _plain_glu_backward(s):
    act = s["case"]["act"]
    g, u, dy, x = s["G"].float(), s["U"].float(), s["dY"].float(), s["X"].float()
    dg, du = dy * u * _activation_slope(g, act), dy * _activation(g, act)
    dx = dg @ s["Wg"].float() + du @ s["Wu"].float()
    return tuple(t.to(torch.bfloat16) for t in (dx, dg.t() @ x, du.t() @ x))


# ---------------------------------------------------------------- work, and the exact outputs


def work(case):
    op, M = case["op"], case["M"]
    if op in ("glu", "glu_backward"):
        K, H = case["K"], case["H"]
        if op == "glu":  # X, both weights, Y (G and U where they are kept)
            return {"bytes": 2 * (M * K + 2 * H * K + (3 if case["save"] else 1) * M * H), "flops": 4 * M * K * H}
        # X, both weights, G, U and dY; the gradients of X and of both weights
        return {"bytes": 2 * (2 * M * K + 4 * H * K + 3 * M * H), "flops": 8 * M * K * H}
    size = 2 if case["dtype"] == "bf16" else 4
    dims = [int(d) for d in case["dims"].split(",")]
    heads = case["H"] if op == "rope" else case["Hq"] + case["Hk"]
    n = M * heads * case["D"]
    turn = 3 * M * heads * sum(dims)
    positions = 4 * M * len(dims)
    if op == "rope":
        return {"bytes": 2 * n * size + positions, "flops": turn}
    if op == "qk":
        return {"bytes": 2 * n * size + positions + 2 * case["D"] * size, "flops": turn + 4 * n}
    return {"bytes": 3 * n * size + positions + 2 * case["D"] * (size + 4), "flops": turn + 11 * n}


def exact(case, seed):
    s = _inputs(case, seed)
    s = {k: v.double() for k, v in s.items()}
    op = case["op"]
    if op == "glu":
        g, u = torch.mm(s["X"], s["Wg"].t()), torch.mm(s["X"], s["Wu"].t())
        y = _value_and_slope64(g, case["act"])[0] * u
        return (y, g, u) if case["save"] else y
    if op == "glu_backward":
        value, slope = _value_and_slope64(s["G"], case["act"])
        dg, du = slope.mul_(s["U"]).mul_(s["dY"]), value.mul_(s["dY"])
        return (torch.mm(dg, s["Wg"]).addmm_(du, s["Wu"]), torch.mm(s["X"].t(), dg).t(),
                torch.mm(s["X"].t(), du).t())
    if op == "rope":
        return _turn64(case, s["pos"], s["X"], -1.0 if case["inverse"] else 1.0)
    first, second = [], []
    for x, w, dy in ((s["Q"], s["qw"], s.get("dQ")), (s["K"], s["kw"], s.get("dK"))):
        size = torch.sqrt(torch.square(x).sum(dim=2, keepdim=True) / case["D"] + EPS)
        if op == "qk":
            first.append(_turn64(case, s["pos"], x / size * w, 1.0))
            continue
        back = _turn64(case, s["pos"], dy, -1.0)
        unit = x / size
        second.append((back * unit).sum(dim=(0, 1)))
        scaled = back * w
        first.append((scaled - unit * (scaled * unit).sum(dim=2, keepdim=True) / case["D"]) / size)
    return tuple(first + second)


def _value_and_slope64(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p + g * p * (1 - p)
    p = torch.special.ndtr(g)
    return g * p, p + g * torch.exp(-g * g / 2) / (2 * math.pi) ** 0.5


def _turn64(case, pos, x, sign):
    """The rotation as a product of complex numbers."""
    angles = []
    for axis, width in enumerate(int(d) for d in case["dims"].split(",")):
        for i in range(width // 2):
            angles.append(pos[:, axis] * case["theta"] ** (-2 * i / width))
    phase = sign * torch.stack(angles, dim=1)[:, None, :]
    factor = torch.complex(torch.cos(phase), torch.sin(phase))
    n = 2 * len(angles)
    out = x.clone()
    first = (slice(0, n, 2), slice(1, n, 2)) if case["pairs"] == "adjacent" else (slice(0, n // 2), slice(n // 2, n))
    z = torch.complex(x[..., first[0]], x[..., first[1]]) * factor
    out[..., first[0]], out[..., first[1]] = z.real, z.imag
    return out
