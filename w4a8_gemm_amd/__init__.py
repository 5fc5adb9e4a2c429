"""MXFP4 W4A8 linear layer for MI355X (gfx950), the attention block on a 4-bit cache that
stands between such layers, and the expert half of a decoder layer on the same weights:
Python binding of libw4a8.so.

The binding only marshals arguments (torch tensors -> device pointers, the
current HIP stream) and maps status codes to exceptions; every step of the
computation runs in the library's HIP kernels.  The library is loaded on the
first call and its absence is an error: there is no fallback path.
"""
from .attention import *  # noqa: F401,F403
from .attention import __all__ as _attention
from .binding import *  # noqa: F401,F403
from .binding import __all__ as _binding
from .moe import *  # noqa: F401,F403
from .moe import __all__ as _moe

__all__ = [*_binding, *_attention, *_moe]
