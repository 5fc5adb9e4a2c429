"""Attention block on a 4-bit cache: binding of libw4a8's head norms with the
position rotation, the paged MXFP4 key/value cache and the attention over it
(C ABI in include/w4a8.h, where each call's arithmetic is stated).

As in binding.py, nothing is computed here: tensors become pointers, the current
torch stream becomes the HIP stream, and status codes become exceptions.  The
checks are those that a pointer cannot carry (types, devices, shapes, strides);
lengths, slots, positions and block tables live on the GPU and are bounded there.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import EXP_MODES, _check, lib

__all__ = ["KVCacheMXFP4", "AttentionWorkspace", "qk_norm_rope", "kv_append_mxfp4", "kv_read_mxfp4",
           "attention_mxfp4", "attention_workspace_bytes"]

_TYPES = {torch.bfloat16: 0, torch.float16: 1}
HEAD_DIMS = (64, 128, 256)
PAGES = tuple(1 << s for s in range(4, 11))

_vp, _i64, _int, _size, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_e8m0", _vp), ("v_codes", _vp), ("v_e8m0", _vp), ("pages", _i64),
                ("kv_heads", _int), ("page", _int), ("head_dim", _int)]


_ready = None


def _lib():
    """The library with this module's signatures set."""
    global _ready
    if _ready is None:
        L = lib()
        cache = ctypes.POINTER(_Cache)
        heads = [_vp, _i64, _i64]
        turn = [_vp, _i64, _vp, _int, _int]
        L.w4a8_qk_norm_rope.argtypes = [_int, *heads, _int, *heads, _int, _i64, _int, _vp, _vp, _f32, *turn, _vp, _vp,
                                        _vp]
        L.w4a8_kv_append_mxfp4.argtypes = [cache, _int, *heads, *heads, _i64, _vp, _int, _vp, _f32, *turn, *heads, _int,
                                           _vp, _vp, _vp]
        L.w4a8_kv_read_mxfp4.argtypes = [cache, _i64, _vp, _vp, _vp, _vp]
        L.w4a8_attention_workspace_bytes.argtypes = [_i64, _i64, _int, _int, _int]
        L.w4a8_attention_workspace_bytes.restype = _size
        L.w4a8_attention_mxfp4.argtypes = [cache, _int, *heads, _int, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _f32,
                                           _int, _int, _vp, _vp, _size, _vp]
        for f in ("w4a8_qk_norm_rope", "w4a8_kv_append_mxfp4", "w4a8_kv_read_mxfp4", "w4a8_attention_mxfp4"):
            getattr(L, f).restype = _int
        _ready = L
    return _ready


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _same(t, name, dtype, device):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _heads(t, name, dtype, device, head_dim, tokens=None, heads=None):
    """A [tokens, heads, head_dim] tensor with contiguous heads (any other strides)."""
    _same(t, name, dtype, device)
    if t.dim() != 3 or t.shape[2] != head_dim or (tokens is not None and t.shape[0] != tokens) or \
            (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [{'tokens' if tokens is None else tokens}, "
                         f"{'heads' if heads is None else heads}, {head_dim}], got {tuple(t.shape)}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must have contiguous heads (unit last stride)")


def _vector(t, name, dtype, device, n):
    _same(t, name, dtype, device)
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}")


def _output(t, name, like, shape):
    if t is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    _same(t, name, like.dtype, like.device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor")
    return t


def _turn(cos_sin, positions, device, tokens, head_dim):
    """(table, rows, positions, rot) of the rotation, zeros without one."""
    if cos_sin is None:
        return None, 0, None, 0
    _same(cos_sin, "cos_sin", torch.float32, device)
    if cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous [positions, rot] tensor")
    rows, rot = cos_sin.shape
    if rot == 0 or rot % 16 or rot > head_dim:
        raise ValueError(f"cos_sin: rot must be a multiple of 16 up to head_dim = {head_dim}, got {rot}")
    if positions is None:
        raise ValueError("a rotation needs positions")
    _vector(positions, "positions", torch.int64, device, tokens)
    return cos_sin.data_ptr(), rows, positions.data_ptr(), rot


def _weight(w, name, device, head_dim):
    if w is None:
        return None
    _vector(w, name, torch.float32, device, head_dim)
    return w.data_ptr()


class KVCacheMXFP4:
    """A paged MXFP4 cache of keys and values, over four uint8 tensors that the caller
    owns: codes [pages, kv_heads, page, head_dim / 2] and exponent bytes
    [pages, kv_heads, head_dim / 32, page], for keys and for values.  Token i of a
    sequence lies in row i % page of page block_table[i // page]; its slot is that
    page times `page` plus the row."""

    def __init__(self, k_codes: torch.Tensor, k_e8m0: torch.Tensor, v_codes: torch.Tensor, v_e8m0: torch.Tensor):
        dev = getattr(k_codes, "device", None)
        for t, n in ((k_codes, "k_codes"), (k_e8m0, "k_e8m0"), (v_codes, "v_codes"), (v_e8m0, "v_e8m0")):
            _same(t, n, torch.uint8, dev)
            if t.dim() != 4 or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous 4-D tensor")
        pages, heads, page, half = k_codes.shape
        d = 2 * half
        if d not in HEAD_DIMS:
            raise ValueError(f"head_dim must be one of {HEAD_DIMS}, got {d}")
        if page not in PAGES:
            raise ValueError(f"page must be a power of two from 16 to 1024, got {page}")
        if pages < 1 or heads < 1:
            raise ValueError("a cache needs at least one page and one head")
        if tuple(v_codes.shape) != (pages, heads, page, half) or tuple(k_e8m0.shape) != (pages, heads, d // 32, page) or \
                tuple(v_e8m0.shape) != (pages, heads, d // 32, page):
            raise ValueError("codes must be [pages, kv_heads, page, head_dim / 2], exponents "
                             "[pages, kv_heads, head_dim / 32, page], the same for keys and values")
        self.k_codes, self.k_e8m0, self.v_codes, self.v_e8m0 = k_codes, k_e8m0, v_codes, v_e8m0
        self.pages, self.kv_heads, self.page, self.head_dim, self.device = pages, heads, page, d, dev
        self._c = _Cache(k_codes.data_ptr(), k_e8m0.data_ptr(), v_codes.data_ptr(), v_e8m0.data_ptr(), pages, heads,
                         page, d)
        self._ref = ctypes.byref(self._c)

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
    if c.device.type != "cuda":
        raise ValueError("the cache must be on a GPU")
    return c


def _mode(mode):
    if mode not in ("ocp", "noclip"):
        raise ValueError(f"mode must be 'ocp' or 'noclip', got {mode!r}")
    return EXP_MODES[mode]


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in _TYPES:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, cos_sin: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None):
    """Norms of queries [tokens, q_heads, head_dim] and keys [tokens, k_heads, head_dim] for
    each head (where a fp32 weight [head_dim] is given) and the rotation of their first rot
    values by the fp32 table cos_sin [rows, rot] (rot/2 cosines, then rot/2 sines) at
    positions int64 [tokens], in one pass.  bf16 or fp16; q and k may be views of a fused
    projection's rows; either may be None.  Returns (q_out, k_out), contiguous."""
    x, n = (k, "k") if q is None else (q, "q")
    _gpu(x, n)
    if x.dim() != 3 or x.shape[2] not in HEAD_DIMS:
        raise ValueError(f"{n} must be [tokens, heads, head_dim] with head_dim one of {HEAD_DIMS}")
    dt, dev, tokens, d = x.dtype, x.device, x.shape[0], x.shape[2]
    cs, rows, pos, rot = _turn(cos_sin, positions, dev, tokens, d)
    qa = ka = (None, 0, 0, 0)
    if q is not None:
        _heads(q, "q", dt, dev, d, tokens)
        q_out = _output(q_out, "q_out", q, q.shape)
        qa = (q.data_ptr(), q.stride(0), q.stride(1), q.shape[1])
    if k is not None:
        _heads(k, "k", dt, dev, d, tokens)
        k_out = _output(k_out, "k_out", k, k.shape)
        ka = (k.data_ptr(), k.stride(0), k.stride(1), k.shape[1])
    qw, kw = _weight(q_weight, "q_weight", dev, d), _weight(k_weight, "k_weight", dev, d)
    if tokens and qa[3] + ka[3]:
        _check(_lib().w4a8_qk_norm_rope(_TYPES[dt], *qa, *ka, tokens, d, qw, kw, eps, cs, rows, pos, rot, interleaved,
                                        q_out.data_ptr() if q is not None else None,
                                        k_out.data_ptr() if k is not None else None, _stream(dev)), "w4a8_qk_norm_rope")
    return (q_out if q is not None else None), (k_out if k is not None else None)


def kv_append_mxfp4(cache: KVCacheMXFP4, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, mode: str = "ocp",
                    cos_sin: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                    k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                    q: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                    q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Keys (normed and turned on the way, as qk_norm_rope does) and values
    [tokens, kv_heads, head_dim] into the cache rows slots (int64 [tokens]; a slot outside the
    cache, as -1 for padding, is skipped).  With q also norms and turns the tokens' queries
    in the same launch and returns them."""
    c = _cache(cache)
    _gpu(k, "k")
    dt, dev, d = k.dtype, c.device, c.head_dim
    tokens = k.shape[0] if k.dim() else 0
    _heads(k, "k", dt, dev, d, tokens, c.kv_heads)
    _heads(v, "v", dt, dev, d, tokens, c.kv_heads)
    _vector(slots, "slots", torch.int64, dev, tokens)
    m = _mode(mode)
    cs, rows, pos, rot = _turn(cos_sin, positions, dev, tokens, d)
    qa, qo = (None, 0, 0, 0), None
    if q is not None:
        _heads(q, "q", dt, dev, d, tokens)
        q_out = _output(q_out, "q_out", q, q.shape)
        if q.shape[1]:
            qa, qo = (q.data_ptr(), q.stride(0), q.stride(1), q.shape[1]), q_out.data_ptr()
    qw, kw = _weight(q_weight, "q_weight", dev, d), _weight(k_weight, "k_weight", dev, d)
    if tokens:
        _check(_lib().w4a8_kv_append_mxfp4(c._ref, _TYPES[dt], k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                                           v.stride(0), v.stride(1), tokens, slots.data_ptr(), m, kw, eps, cs, rows, pos,
                                           rot, interleaved, *qa, qw, qo, _stream(dev)), "w4a8_kv_append_mxfp4")
    return q_out if q is not None else None


def kv_read_mxfp4(cache: KVCacheMXFP4, slots: torch.Tensor):
    """The cache rows slots (int64 [n]) as bf16 keys and values [n, kv_heads, head_dim], exact;
    zeros for a slot outside the cache."""
    c = _cache(cache)
    n = slots.shape[0] if isinstance(slots, torch.Tensor) and slots.dim() == 1 else -1
    _vector(slots, "slots", torch.int64, c.device, n)
    k, v = (torch.empty((n, c.kv_heads, c.head_dim), dtype=torch.bfloat16, device=c.device) for _ in range(2))
    if n:
        _check(_lib().w4a8_kv_read_mxfp4(c._ref, n, slots.data_ptr(), k.data_ptr(), v.data_ptr(), _stream(c.device)),
               "w4a8_kv_read_mxfp4")
    return k, v


def attention_workspace_bytes(seqs: int, max_q: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_lib().w4a8_attention_workspace_bytes(int(seqs), int(max_q), int(q_heads), int(kv_heads), int(head_dim)))


class AttentionWorkspace:
    """Caller-owned workspace of attention_mxfp4 for one batch shape: partial results of
    sequences whose keys are shared by several workgroups.  Calls that share one must
    not overlap in time."""

    def __init__(self, seqs: int, max_q: int, q_heads: int, kv_heads: int, head_dim: int, device="cuda"):
        if min(seqs, max_q, q_heads, kv_heads) < 1 or q_heads % kv_heads or head_dim not in HEAD_DIMS:
            raise ValueError("sizes must be positive, q_heads a multiple of kv_heads and head_dim one of "
                             f"{HEAD_DIMS}")
        self.nbytes = attention_workspace_bytes(seqs, max_q, q_heads, kv_heads, head_dim)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device) if self.nbytes else None

    def args(self):
        return (None, 0) if self.buf is None else (self.buf.data_ptr(), self.nbytes)


def attention_mxfp4(q: torch.Tensor, cache: KVCacheMXFP4, block_table: torch.Tensor, context_lens: torch.Tensor,
                    cu_q: torch.Tensor | None = None, max_q: int = 1, scale: float | None = None, causal: bool = True,
                    window: int = 0, workspace: AttentionWorkspace | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Softmax attention of the queries [tokens, q_heads, head_dim] (bf16 or fp16) over the cached keys and
    values of their sequences.  block_table int32 [seqs, width] (rows may be strided); context_lens
    int32 [seqs], the new tokens among them; cu_q int32 [seqs + 1] with at most max_q query
    tokens per sequence, or None for one each.  scale: head_dim ** -0.5 by default.  window > 0: each
    query sees the last `window` keys up to its own.  Without a workspace one is
    allocated for the call."""
    c = _cache(cache)
    _gpu(q, "q")
    dev, d = c.device, c.head_dim
    _heads(q, "q", q.dtype, dev, d)
    tokens, hq = q.shape[0], q.shape[1]
    if hq == 0 or hq % c.kv_heads:
        raise ValueError(f"q_heads = {hq} must be a multiple of kv_heads = {c.kv_heads}")
    _same(context_lens, "context_lens", torch.int32, dev)
    seqs = context_lens.shape[0] if context_lens.dim() == 1 else -1
    _vector(context_lens, "context_lens", torch.int32, dev, seqs)
    _same(block_table, "block_table", torch.int32, dev)
    if block_table.dim() != 2 or block_table.shape[0] != seqs or block_table.stride(1) != 1 or \
            (seqs > 1 and block_table.stride(0) < block_table.shape[1]):
        raise ValueError("block_table must be [seqs, width] with contiguous rows")
    if cu_q is None:
        if tokens != seqs or max_q != 1:
            raise ValueError(f"without cu_q every sequence has one query token: {tokens} tokens, {seqs} sequences, "
                             f"max_q = {max_q}")
        cu = None
    else:
        _vector(cu_q, "cu_q", torch.int32, dev, seqs + 1)
        cu = cu_q.data_ptr()
    max_q = int(max_q)
    if max_q < 1:
        raise ValueError("max_q must be at least 1")
    if window < 0 or (window and not causal):
        raise ValueError("window must be >= 0, and 0 without a causal mask")
    out = _output(out, "out", q, q.shape)
    if tokens == 0 or seqs == 0:
        return out
    width = block_table.shape[1]
    if width == 0:
        raise ValueError("block_table needs at least one column")
    if workspace is None:
        workspace = AttentionWorkspace(seqs, max_q, hq, c.kv_heads, d, dev)
    ws, n = workspace.args()
    _check(_lib().w4a8_attention_mxfp4(c._ref, _TYPES[q.dtype], q.data_ptr(), q.stride(0), q.stride(1), hq, tokens, seqs,
                                       cu, max_q, block_table.data_ptr(),
                                       block_table.stride(0) if seqs > 1 else width, width,
                                       context_lens.data_ptr(), d ** -0.5 if scale is None else scale, causal, window,
                                       out.data_ptr(), ws, n, _stream(dev)), "w4a8_attention_mxfp4")
    return out
