"""Per-layer choice between the sparse layer and the dense one, and a layer object that
dispatches to the library's entry points.

"RT-Lynx: Putting the GEMM Sparsity In a Right Way for Diffusion Models", summary page,
method step 3 (selective layer skipping): in the double-stream Qwen-Image the QKV, MLP-up
and MLP-down projections are sparsified; in the single-stream models the residual of some
layers is too large for the rank-64 branch, so FLUX keeps the attention output projection
and MLP-down of its single-stream blocks dense and Z-Image keeps the attention output
projection and MLP-up dense; every other layer uses the sparse layer.

Beside the projections, what such a block runs around them: the layer norm in front, with each request's scale
and shift (AdaptiveNorm), the low-rank adapters of a batch's requests beside a projection (AdaptedLinear), the queries'
and keys' head norms and rotary positions (AttentionInput) and the gated feed-forward block (GatedMLP).

Reading taken where the page is silent: Qwen-Image's attention output projection, which the
page does not list, stays dense; FLUX's double-stream blocks sparsify all four projections.
"""
from __future__ import annotations

import torch

from . import (EPS, RTL_ACT_SILU, RTL_ROPE_ADJACENT, rtl_adapters, rtl_adapters_backward, rtl_adapters_plan,
               rtl_glu_fused, rtl_layer_norm, rtl_layer_norm_backward, rtl_linear_dense_ref, rtl_linear_fused, rtl_linear_fused_workspace_bytes, rtl_qk_norm_rope, _dt, _elsewhere, _empty, _stream)

__all__ = ["LAYER_KINDS", "MODELS", "dense_layers", "is_sparse", "Linear", "build_block", "AdaptiveNorm", "AdaptedLinear",
           "AttentionInput", "GatedMLP"]

LAYER_KINDS = ("attn.qkv", "attn.o_proj", "mlp.up", "mlp.down")

# (model, block stream) -> projections kept dense.
_DENSE = {
    ("qwen-image", "double"): frozenset({"attn.o_proj"}),
    ("flux", "double"): frozenset(),
    ("flux", "single"): frozenset({"attn.o_proj", "mlp.down"}),
    ("z-image", "single"): frozenset({"attn.o_proj", "mlp.up"}),
}
MODELS = tuple(sorted({m for m, _ in _DENSE}))


def dense_layers(model: str, stream: str) -> frozenset:
    """Projections of a (model, block stream) that keep the dense layer."""
    key = (model.lower(), stream.lower())
    if key not in _DENSE:
        raise KeyError(f"no layer policy for model {model!r} with {stream!r}-stream blocks; "
                       f"known: {sorted(_DENSE)}")
    return _DENSE[key]


def is_sparse(model: str, stream: str, layer: str) -> bool:
    """True when `layer` (one of LAYER_KINDS) of a `stream`-stream block of `model` uses the
    2:4 + low-rank layer."""
    if layer not in LAYER_KINDS:
        raise KeyError(f"unknown projection {layer!r}; known: {LAYER_KINDS}")
    return layer not in dense_layers(model, stream)


class Linear:
    """One projection Y = layer(X) with weights W [N,K] (and L_A [N,R], L_B [R,K] when sparse).

    Sparse: rtl_linear_fused (norm-compensated 2:4 + rank-R branch).  Dense:
    rtl_linear_dense_ref.  The workspace of the sparse layer is allocated on the first
    call with a given number of rows on a stream, for that stream, and reused after that, so
    later calls allocate nothing but Y (and not even Y when it is passed)."""

    def __init__(self, W: torch.Tensor, LA=None, LB=None, sparse: bool = True, eps: float = EPS):
        if sparse and (LA is None) != (LB is None):
            raise ValueError("L_A and L_B go together")
        self.W, self.LA, self.LB, self.sparse, self.eps = W, LA, LB, sparse, eps
        self._ws = {}

    @property
    def R(self) -> int:
        return 0 if self.LB is None else self.LB.shape[0]

    def workspace(self, M: int, stream=None):
        """What calls of M rows on `stream` (None: the current one) use: memory of that stream, so that neither other work
        that torch gave it to nor another stream's calls meet there."""
        key = M, _stream(stream).value if self.W.is_cuda else None
        if key not in self._ws:
            need = rtl_linear_fused_workspace_bytes(_dt(self.W), M, self.W.shape[0], self.W.shape[1], self.R)
            self._ws[key] = _empty((max(need, 1),), torch.uint8, self.W.device, stream)
        return self._ws[key]

    def __call__(self, X: torch.Tensor, Y=None, stream=None) -> torch.Tensor:
        there = _elsewhere(X, self.W, Y)
        if there is not None:
            with there:
                return self(X, Y, stream)
        if not self.sparse:
            return rtl_linear_dense_ref(X, self.W, Y=Y, stream=stream)
        return rtl_linear_fused(X, self.W, self.LA, self.LB, eps=self.eps, Y=Y,
                                workspace=self.workspace(X.shape[0], stream), stream=stream)


def build_block(model: str, stream: str, weights: dict) -> dict:
    """Linear objects for one transformer block.  `weights` maps each projection kind to
    (W, L_A, L_B); the low-rank factors of a projection that the policy keeps dense are
    not used."""
    out = {}
    for kind, (W, LA, LB) in weights.items():
        sp = is_sparse(model, stream, kind)
        out[kind] = Linear(W, LA if sp else None, LB if sp else None, sparse=sp)
    return out


class AdaptiveNorm:
    """The layer norm in front of a block's projections, with weights [D] (None: ones, zeros) and, a
    call, each request's scale and shift."""

    def __init__(self, weight=None, bias=None, eps: float = 1e-6):
        if weight is not None and bias is not None and weight.shape != bias.shape:
            raise ValueError("the weight and the bias have one length")
        self.weight, self.bias, self.eps = weight, bias, eps

    def __call__(self, X: torch.Tensor, scale=None, shift=None, groups=None, stats=None, Y=None, stream=None) -> torch.Tensor:
        """Rows groups[g] .. groups[g + 1] - 1 of X [M,D] are request g's (rtl_layer_norm); `stats` [M,2] float32
        receives what `backward` needs."""
        return rtl_layer_norm(X, self.weight, self.bias, scale, shift, groups, self.eps, Y=Y, stats=stats, stream=stream)

    def backward(self, X: torch.Tensor, stats: torch.Tensor, dY: torch.Tensor, scale=None, groups=None, stream=None, dX=None,
                 dweight=None, dbias=None, dscale=None, dshift=None):
        """(dX, dweight, dbias, dscale, dshift) of rtl_layer_norm_backward, in the tensors that are given: an
        optimizer's list (rtl_adamw_tensors) holds dweight and dbias from step to step."""
        return rtl_layer_norm_backward(X, stats, dY, self.weight, self.bias, scale, groups, dX, dweight, dbias, dscale, dshift,
                                       stream=stream)


class AdaptedLinear:
    """A projection that a batch's requests share, and beside it the low-rank adapters that they bring: Y = linear(X)
    + alpha_a (X LB_a^T) LA_a^T, a row's adapter a of LA [A,N,R] and LB [A,R,K] (bf16) as its batch's plan says.  The
    adapters add to the projection's output in place: rows without one are the projection's own, to the bit.  The
    adapters' workspace is the caller's, or allocated by each call on its stream."""

    def __init__(self, linear: Linear, LA: torch.Tensor, LB: torch.Tensor, alpha=None):
        N, K = linear.W.shape
        if LA.dim() != 3 or LB.dim() != 3 or tuple(LA.shape) != (LB.shape[0], N, LB.shape[1]) or LB.shape[2] != K:
            raise ValueError(f"LA and LB are [A,{N},R] and [A,R,{K}], got {tuple(LA.shape)} and {tuple(LB.shape)}")
        if alpha is not None and tuple(alpha.shape) != (LA.shape[0],):
            raise ValueError(f"alpha is [{LA.shape[0]}], got {tuple(alpha.shape)}")
        self.linear, self.LA, self.LB, self.alpha = linear, LA, LB, alpha

    def plan(self, ids: torch.Tensor, plan=None, stream=None) -> torch.Tensor:
        """The plan of a batch whose row m has adapter ids[m] (int32; outside 0..A-1: none)."""
        return rtl_adapters_plan(ids, self.LA.shape[0], plan, stream=stream)

    def __call__(self, X: torch.Tensor, plan: torch.Tensor, T=None, Y=None, stream=None, workspace=None) -> torch.Tensor:
        """`T` [M,R] float32 receives what `backward` needs; `workspace`: rtl_adapters_workspace_bytes bytes."""
        Y = self.linear(X, Y=Y, stream=stream)
        return rtl_adapters(X, self.LA, self.LB, plan, self.alpha, Y0=Y, Y=Y, T=T, workspace=workspace, stream=stream)

    def backward(self, X: torch.Tensor, plan: torch.Tensor, T: torch.Tensor, dY: torch.Tensor, dX0=None, need_dx: bool = True,
                 stream=None, workspace=None, dX=None, dLA=None, dLB=None):
        """(dX, dLA, dLB) of rtl_adapters_backward, in the tensors that are given: an optimizer's list
        (rtl_adamw_tensors) holds dLA and dLB from step to step.  `dX0`: what came through the projection."""
        return rtl_adapters_backward(X, self.LA, self.LB, plan, T, dY, self.alpha, dX0=dX0, dX=dX, dLA=dLA, dLB=dLB,
                                     workspace=workspace, need_dx=need_dx, stream=stream)


class AttentionInput:
    """Queries, keys and values of an attention layer from its tokens: the `qkv` projection (a
    Linear with (heads + 2 kv_heads) * D outputs: queries, then keys, then values), then the RMS
    norm of every query and key head (weights [D], None: ones) and the rotation by each token's
    positions (rtl_rope_axes; no `axis_dims`: none), in one pass over the projection's output,
    in place."""

    def __init__(self, qkv: Linear, heads: int, kv_heads: int, q_weight=None, k_weight=None, axis_dims=(),
                 theta: float = 10000.0, eps: float = 1e-6, pairs: int = RTL_ROPE_ADJACENT):
        outputs = qkv.W.shape[0]
        if heads < 1 or kv_heads < 1 or outputs % (heads + 2 * kv_heads) != 0:
            raise ValueError(f"{outputs} outputs are not {heads} query heads and twice {kv_heads} key heads")
        self.qkv, self.heads, self.kv_heads = qkv, heads, kv_heads
        self.q_weight, self.k_weight = q_weight, k_weight
        self.axis_dims, self.theta, self.eps, self.pairs = tuple(axis_dims), theta, eps, pairs

    def __call__(self, X: torch.Tensor, pos=None, stream=None):
        """(q [M, heads, D], k and v [M, kv_heads, D]), views of one buffer; `pos` [M, axes] float32."""
        n = self.heads + 2 * self.kv_heads
        rows = self.qkv(X, stream=stream).view(X.shape[0], n, -1)
        q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        rtl_qk_norm_rope(q, k, self.q_weight, self.k_weight, pos, self.axis_dims, theta=self.theta, eps=self.eps,
                         pairs=self.pairs, Qo=q, Ko=k, stream=stream)
        return q, k, v


class GatedMLP:
    """A gated feed-forward block whose up projections are dense (Z-Image's policy for mlp.up):
    rtl_glu_fused with weights Wg and Wu [H,K], then `down`, a Linear, sparse or dense."""

    def __init__(self, Wg: torch.Tensor, Wu: torch.Tensor, down: Linear, act: int = RTL_ACT_SILU):
        if Wg.shape != Wu.shape or down.W.shape[1] != Wg.shape[0]:
            raise ValueError("Wg and Wu are [H,K] and the down projection's weights [N,H]")
        self.Wg, self.Wu, self.down, self.act = Wg, Wu, down, act

    def __call__(self, X: torch.Tensor, Y=None, stream=None) -> torch.Tensor:
        return self.down(rtl_glu_fused(X, self.Wg, self.Wu, act=self.act, stream=stream), Y=Y, stream=stream)
