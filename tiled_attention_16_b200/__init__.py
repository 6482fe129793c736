"""Exact tiled (flash) attention for NVIDIA B200 (sm_100a).

The compute lives in ``libfa_sm100.so`` (C ABI declared in include/fa.h);
``attention`` is its thin Python binding, ``rope`` that of fa_rope.h (per-head
norm with rotation) and ``cache`` that of fa_cache.h (K/V cache, decoding over
it).  The shared library is loaded on
first use, so importing this package (for example for the seeded workloads
in ``workloads``) needs no GPU.
"""
from .attention import (  # noqa: F401
    FA_ERR_CUDA,
    FA_ERR_INVALID_ARG,
    FA_ERR_TIMEOUT,
    FA_ERR_UNSUPPORTED,
    FA_OK,
    FAError,
    bwd,
    device_status,
    fwd,
    workspace_bytes,
)
from .cache import cache_read, cache_write, decode_cache, make_cache  # noqa: F401
from .rope import qk_norm_rope, qk_norm_rope_bwd  # noqa: F401
