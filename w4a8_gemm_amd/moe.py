"""The expert half of a decoder layer: Python interface of libw4a8's norms around a
block, its choice of each token's experts, and the experts' products on MXFP4 weights
(C ABI in include/w4a8.h, where each call's arithmetic is stated).

As in attention.py, nothing is computed here: the compiled module _moe
(csrc/moe_bind.cpp) turns tensors into pointers, the current torch stream into the
HIP stream and status codes into exceptions.  Ids live on the GPU and are bounded there.
Inference only, as the library: results carry no gradient, whatever the inputs require.
"""
from __future__ import annotations

import importlib
import os

import torch

from . import binding

__all__ = ["ExpertsMXFP4", "MoEWorkspace", "residual_norm", "moe_route", "moe_mxfp4", "moe_workspace_bytes"]

MODULE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_moe.so")

_module = None


def _native():
    """The compiled module, loaded on the first call (after libw4a8.so, which it calls)."""
    global _module
    if _module is None:
        binding.lib()
        if not os.path.exists(MODULE_PATH):
            raise RuntimeError(f"_moe.so is not built ({MODULE_PATH}); run "
                               "`python -m w4a8_gemm_amd.build` (there is no fallback path)")
        _module = importlib.import_module("._moe", __package__)
        _module.set_error(binding.W4A8Error)
    return _module


def residual_norm(y: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                  post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
                  eps: float = 1e-6, values: bool = True, fp8: bool = False, residual_out: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, x_fp8: torch.Tensor | None = None,
                  x_scale: torch.Tensor | None = None):
    """The norms around a block, in one pass over its output y [tokens, hidden] (bf16 or
    fp16, rows may be strided): y normed where a fp32 post_weight [hidden] is given, times
    gate ([tokens or 1, hidden or 1] of y's type), times scale, plus the residual (y's type
    or float32) gives the new residual; its norm times the fp32 weight [hidden] (None: ones)
    leaves as values of y's type (values=True) and as per-token e4m3 codes with their
    scales (fp8=True), the linears' and moe_mxfp4's activations.

    Returns (residual_out, out, x_fp8, x_scale), None for what was not asked for; without a
    residual the sum is stored only where residual_out is given.  residual_out may be
    residual itself, and out y.  An output given for what is not asked for is refused."""
    return _native().residual_norm(y, residual, weight, post_weight, gate, scale, eps, values, fp8, residual_out, out, x_fp8,
                                   x_scale)


_SCORES = {"softmax": 0, "sigmoid": 1}
_ACTS = {"silu": 0, "gelu_tanh": 1}


def _one_of(names, value, what):
    try:
        return names[value]
    except (KeyError, TypeError):
        raise ValueError(f"{what} must be one of {', '.join(map(repr, names))}, got {value!r}") from None


def moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
              groups_kept: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
              weights: torch.Tensor | None = None, ids: torch.Tensor | None = None):
    """The top_k experts of each token from the router's logits [tokens, experts] (float32,
    bf16 or fp16) -> (weights float32 [tokens, top_k], ids int32 [tokens, top_k]), in
    descending order, ties to the lower id.  score: "softmax" or "sigmoid" of the logits
    gives the weights, over their sum with renormalize, times scale.  A fp32 bias [experts]
    is added to the scores for the choice alone; of `groups` equal runs of experts the
    groups_kept with the largest sums of their group_top (1 or 2) best take part.  Experts of
    a logit of -inf are off; a row with too few left ends in ids of -1 and weights of 0."""
    return _native().route(logits, top_k, _one_of(_SCORES, score, "score"), bias, groups, groups_kept, group_top, renormalize,
                           scale, weights, ids)


class ExpertsMXFP4:
    """The experts' prepared MXFP4 weights: up, one PreparedMXFP4 of [experts * 2 inter, hidden]
    (of each expert the gate's rows, then the up rows), and down, one of
    [experts * hidden, inter].  hidden and inter are multiples of 128."""

    def __init__(self, up: binding.PreparedMXFP4, down: binding.PreparedMXFP4, experts: int):
        for name, w in (("up", up), ("down", down)):
            if not isinstance(w, binding.PreparedMXFP4):
                raise TypeError(f"{name} must be a PreparedMXFP4")
        experts = int(experts)
        hidden, inter = up.K, down.K
        if experts < 1 or up.N != 2 * experts * inter or down.N != experts * hidden:
            raise ValueError(f"{experts} experts of {hidden} and {inter} need up weights of [{2 * experts * inter}, {hidden}] and "
                             f"down weights of [{experts * hidden}, {inter}], got [{up.N}, {up.K}] and [{down.N}, {down.K}]")
        self._c = _native().experts(up.w, up.s, down.w, down.s, experts, hidden, inter)
        self.up, self.down = up, down
        self.experts, self.hidden, self.inter, self.device = experts, hidden, inter, up.w.device

    @classmethod
    def prepare(cls, up_packed: torch.Tensor, up_e8m0: torch.Tensor, down_packed: torch.Tensor, down_e8m0: torch.Tensor,
                experts: int) -> "ExpertsMXFP4":
        """From row-major codes and exponents: up [experts * 2 inter, hidden / 2] and
        [.., hidden / 32], down [experts * hidden, inter / 2] and [.., inter / 32]."""
        return cls(binding.mxfp4_prepare(up_packed, up_e8m0), binding.mxfp4_prepare(down_packed, down_e8m0), experts)


def moe_workspace_bytes(tokens: int, top_k: int, hidden: int, inter: int) -> int:
    return int(binding.lib().w4a8_moe_workspace_bytes(int(tokens), int(top_k), int(hidden), int(inter)))


class MoEWorkspace:
    """Caller-owned workspace of moe_mxfp4: what the first product hands to the second.  It
    serves every call of at most these tokens with this top_k, hidden and inter.  Its contents
    mean nothing between calls; calls that share one must not overlap in time."""

    def __init__(self, tokens: int, top_k: int, experts: int, hidden: int, inter: int, device="cuda"):
        if min(tokens, top_k, experts, hidden, inter) < 1 or top_k > experts or hidden % 128 or inter % 128:
            raise ValueError("sizes must be positive, top_k at most experts, hidden and inter multiples of 128")
        self.nbytes = moe_workspace_bytes(tokens, top_k, hidden, inter)
        if not self.nbytes:
            raise ValueError("sizes beyond what moe_mxfp4 serves")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)


def moe_mxfp4(x_fp8: torch.Tensor, x_scale: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, experts: ExpertsMXFP4,
              act: str = "silu", workspace: MoEWorkspace | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = sum over j of weights[t, j] * down_e(act(gate_e(x[t])) * up_e(x[t])), e = ids[t, j],
    as bf16 [tokens, hidden], for the fp8 activations of quant_act_fp8_per_token or residual_norm
    (codes uint8 [tokens, hidden], scales [tokens]) and moe_route's ids and weights
    [tokens, top_k].  An id outside the experts, as -1 for padding or for an expert of another
    GPU, is left out.  act: "silu" or "gelu_tanh".  Made for up to some hundreds of tokens per expert: an
    expert's weights are read once for every 16 to 64 of its slots, anew for each 2048 / top_k
    tokens.  Without a workspace one is allocated for the call."""
    if not isinstance(experts, ExpertsMXFP4):
        raise TypeError("experts must be an ExpertsMXFP4")
    if workspace is not None and not isinstance(workspace, MoEWorkspace):
        raise TypeError("workspace must be a MoEWorkspace")
    return _native().moe(x_fp8, x_scale, ids, weights, experts._c, _one_of(_ACTS, act, "act"),
                         None if workspace is None else workspace.buf, out)
