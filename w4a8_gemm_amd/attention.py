"""Attention block on a 4-bit cache: Python interface of libw4a8's head norms with the
position rotation, the paged MXFP4 key/value cache and the attention over it
(C ABI in include/w4a8.h, where each call's arithmetic is stated).

As in binding.py, nothing is computed here: tensors become pointers, the current
torch stream becomes the HIP stream, and status codes become exceptions, in the
compiled module _attention (csrc/attention_bind.cpp).  Its checks are those that a
pointer cannot carry (types, devices, shapes, strides); lengths, slots, positions and
block tables live on the GPU and are bounded there.
"""
from __future__ import annotations

import importlib
import os

import torch

from . import binding

__all__ = ["KVCacheMXFP4", "AttentionWorkspace", "qk_norm_rope", "kv_append_mxfp4", "kv_read_mxfp4",
           "attention_mxfp4", "attention_workspace_bytes"]

HEAD_DIMS = (64, 128, 256)
MODULE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_attention.so")

_module = None


def _native():
    """The compiled module, loaded on the first call (after libw4a8.so, which it calls)."""
    global _module
    if _module is None:
        binding.lib()
        if not os.path.exists(MODULE_PATH):
            raise RuntimeError(f"_attention.so is not built ({MODULE_PATH}); run "
                               "`python -m w4a8_gemm_amd.build` (there is no fallback path)")
        _module = importlib.import_module("._attention", __package__)
        _module.set_error(binding.W4A8Error)
    return _module


class KVCacheMXFP4:
    """A paged MXFP4 cache of keys and values, over four uint8 tensors that the caller
    owns: codes [pages, kv_heads, page, head_dim / 2] and exponent bytes
    [pages, kv_heads, head_dim / 32, page], for keys and for values.  page is a power of
    two from 16 to 1024, head_dim 64, 128 or 256.  Token i of a sequence lies in row
    i % page of page block_table[i // page]; its slot is that page times `page` plus
    the row."""

    def __init__(self, k_codes: torch.Tensor, k_e8m0: torch.Tensor, v_codes: torch.Tensor, v_e8m0: torch.Tensor):
        self._c = _native().cache(k_codes, k_e8m0, v_codes, v_e8m0)
        self._tensors = (k_codes, k_e8m0, v_codes, v_e8m0)
        self.pages, self.kv_heads, self.page, half = k_codes.shape
        self.head_dim, self.device = 2 * half, k_codes.device

    k_codes = property(lambda self: self._tensors[0])
    k_e8m0 = property(lambda self: self._tensors[1])
    v_codes = property(lambda self: self._tensors[2])
    v_e8m0 = property(lambda self: self._tensors[3])

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda") -> "KVCacheMXFP4":
        """A cache of zeros."""
        if head_dim not in HEAD_DIMS:
            raise ValueError(f"head_dim must be one of {HEAD_DIMS}, got {head_dim}")
        z = [torch.zeros(s, dtype=torch.uint8, device=device)
             for s in ((pages, kv_heads, page, head_dim // 2), (pages, kv_heads, head_dim // 32, page)) * 2]
        return cls(*z)


def _cache(c):
    if not isinstance(c, KVCacheMXFP4):
        raise TypeError("cache must be a KVCacheMXFP4")
    return c._c


_MODES = {m: binding.EXP_MODES[m] for m in ("ocp", "noclip")}


def _mode(mode):
    try:
        return _MODES[mode]
    except (KeyError, TypeError):
        raise ValueError(f"mode must be 'ocp' or 'noclip', got {mode!r}") from None


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, cos_sin: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None):
    """Norms of queries [tokens, q_heads, head_dim] and keys [tokens, k_heads, head_dim] for
    each head (where a fp32 weight [head_dim] is given) and the rotation of their first rot
    values by the fp32 table cos_sin [rows, rot] (rot/2 cosines, then rot/2 sines) at
    positions int64 [tokens], in one pass.  bf16 or fp16; q and k may be views of a fused
    projection's rows; either may be None.  Returns (q_out, k_out), contiguous."""
    return _native().norm_rope(q, k, cos_sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out)


def kv_append_mxfp4(cache: KVCacheMXFP4, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, mode: str = "ocp",
                    cos_sin: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                    k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                    q: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                    q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Keys (normed and turned on the way, as qk_norm_rope does) and values
    [tokens, kv_heads, head_dim] into the cache rows slots (int64 [tokens]; a slot outside the
    cache, as -1 for padding, is skipped).  With q also norms and turns the tokens' queries
    in the same launch and returns them."""
    return _native().append(_cache(cache), k, v, slots, _mode(mode), cos_sin, positions, k_weight, eps, interleaved, q,
                            q_weight, q_out)


def kv_read_mxfp4(cache: KVCacheMXFP4, slots: torch.Tensor):
    """The cache rows slots (int64 [n]) as bf16 keys and values [n, kv_heads, head_dim], exact;
    zeros for a slot outside the cache."""
    return _native().read(_cache(cache), slots)


def attention_workspace_bytes(seqs: int, max_q: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(binding.lib().w4a8_attention_workspace_bytes(int(seqs), int(max_q), int(q_heads), int(kv_heads),
                                                            int(head_dim)))


class AttentionWorkspace:
    """Caller-owned workspace of attention_mxfp4: partial results of sequences whose keys
    are shared by several workgroups, and the counters of their joins.  It serves every call
    of at most these sequences and query tokens with these heads.  Allocated by torch and its
    counters zeroed once; every call leaves them at zero.  Calls that share one must not
    overlap in time."""

    def __init__(self, seqs: int, max_q: int, q_heads: int, kv_heads: int, head_dim: int, device="cuda"):
        if min(seqs, max_q, q_heads, kv_heads) < 1 or q_heads % kv_heads or head_dim not in HEAD_DIMS:
            raise ValueError("sizes must be positive, q_heads a multiple of kv_heads and head_dim one of "
                             f"{HEAD_DIMS}")
        self.nbytes = attention_workspace_bytes(seqs, max_q, q_heads, kv_heads, head_dim)
        if not self.nbytes:
            raise ValueError("sizes beyond what the attention serves")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.buf[:binding.lib().w4a8_attention_counter_bytes()].zero_()


def _buf(workspace):
    if workspace is None:
        return None
    # the linears' Workspace keeps partial results where the joins' counters must be zero
    if not isinstance(workspace, AttentionWorkspace):
        raise TypeError("workspace must be an AttentionWorkspace")
    return workspace.buf


def attention_mxfp4(q: torch.Tensor, cache: KVCacheMXFP4, block_table: torch.Tensor, context_lens: torch.Tensor,
                    cu_q: torch.Tensor | None = None, max_q: int = 1, scale: float | None = None, causal: bool = True,
                    window: int = 0, workspace: AttentionWorkspace | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Softmax attention of the queries [tokens, q_heads, head_dim] (bf16 or fp16) over the cached keys and
    values of their sequences.  block_table int32 [seqs, width] (rows may be strided); context_lens
    int32 [seqs], the new tokens among them; cu_q int32 [seqs + 1] with at most max_q query
    tokens per sequence, or None for one each.  scale: head_dim ** -0.5 by default.  window > 0: each
    query sees the last `window` keys up to its own.  Output rows of no sequence, and those past
    max_q, are not written.  Without a workspace one is
    allocated for the call."""
    return _native().attention(q, _cache(cache), block_table, context_lens, cu_q, max_q, scale, causal, window,
                               _buf(workspace), out)
