"""Per-layer choice between the sparse layer and the dense one, and a layer object that
dispatches to the library's entry points.

"RT-Lynx: Putting the GEMM Sparsity In a Right Way for Diffusion Models", summary page,
method step 3 (selective layer skipping): in the double-stream Qwen-Image the QKV, MLP-up
and MLP-down projections are sparsified; in the single-stream models the residual of some
layers is too large for the rank-64 branch, so FLUX keeps the attention output projection
and MLP-down of its single-stream blocks dense and Z-Image keeps the attention output
projection and MLP-up dense; every other layer uses the sparse layer.

Beside the projections, what such a block runs on their outputs: the queries' and keys' head norms
and rotary positions (AttentionInput) and the gated feed-forward block (GatedMLP).

Reading taken where the page is silent: Qwen-Image's attention output projection, which the
page does not list, stays dense; FLUX's double-stream blocks sparsify all four projections.
"""
from __future__ import annotations

import torch

from . import (EPS, RTL_ACT_SILU, RTL_ROPE_ADJACENT, rtl_glu_fused, rtl_linear_dense_ref, rtl_linear_fused,
               rtl_linear_fused_workspace_bytes, rtl_qk_norm_rope, _dt)

__all__ = ["LAYER_KINDS", "MODELS", "dense_layers", "is_sparse", "Linear", "build_block", "AttentionInput", "GatedMLP"]

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
    call with a given number of rows and reused after that, so later calls allocate
    nothing but Y (and not even Y when it is passed)."""

    def __init__(self, W: torch.Tensor, LA=None, LB=None, sparse: bool = True, eps: float = EPS):
        if sparse and (LA is None) != (LB is None):
            raise ValueError("L_A and L_B go together")
        self.W, self.LA, self.LB, self.sparse, self.eps = W, LA, LB, sparse, eps
        self._ws = {}

    @property
    def R(self) -> int:
        return 0 if self.LB is None else self.LB.shape[0]

    def workspace(self, M: int):
        if M not in self._ws:
            need = rtl_linear_fused_workspace_bytes(_dt(self.W), M, self.W.shape[0], self.W.shape[1], self.R)
            self._ws[M] = torch.empty((max(need, 1),), dtype=torch.uint8, device=self.W.device)
        return self._ws[M]

    def __call__(self, X: torch.Tensor, Y=None, stream=None) -> torch.Tensor:
        if not self.sparse:
            return rtl_linear_dense_ref(X, self.W, Y=Y, stream=stream)
        return rtl_linear_fused(X, self.W, self.LA, self.LB, eps=self.eps, Y=Y,
                                workspace=self.workspace(X.shape[0]), stream=stream)


def build_block(model: str, stream: str, weights: dict) -> dict:
    """Linear objects for one transformer block.  `weights` maps each projection kind to
    (W, L_A, L_B); the low-rank factors of a projection that the policy keeps dense are
    not used."""
    out = {}
    for kind, (W, LA, LB) in weights.items():
        sp = is_sparse(model, stream, kind)
        out[kind] = Linear(W, LA if sp else None, LB if sp else None, sparse=sp)
    return out


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
