"""B200-native (sm_100a) fused scaled dot-product attention forward.

The compute path is hand-written CUDA kernels behind a C ABI
(``include/attn_fwd.h``, ``attn_bwd.h``, ``attn_cache.h``); :mod:`scaled_dot_product_10_b200.attn` is the thin
ctypes binding over it.  Importing this package does not load the CUDA
library; the first call does, and it fails loudly if the library is missing.
"""
from .attn import (  # noqa: F401
    ATTN_ERR_ALIGN, ATTN_ERR_CUDA, ATTN_ERR_INVALID, ATTN_ERR_TIMEOUT, ATTN_ERR_UNSUPPORTED,
    ATTN_OK, AttnError, KVCache, attn_cache_append, attn_fwd, attn_fwd_cache, attn_fwd_host,
    attn_status, attn_strerror, cache_workspace_bytes, host_workspace_bytes, library_path, load_library,
)
