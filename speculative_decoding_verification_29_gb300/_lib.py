"""ctypes declarations of libspecverify.so (the C ABI in include/specverify.h).

Loading fails loudly when the library has not been built: there is no
fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libspecverify.so")

SPEC_F32, SPEC_BF16, SPEC_F16 = 0, 1, 2
SPEC_OK, SPEC_ERR_ARG, SPEC_ERR_ALIGN, SPEC_ERR_CUDA, SPEC_ERR_TIMEOUT, SPEC_ERR_UNIMPLEMENTED = 0, -1, -2, -3, -4, -5
SPEC_ERR_WORKSPACE, SPEC_ERR_UNSUPPORTED = SPEC_ERR_ALIGN, SPEC_ERR_UNIMPLEMENTED  # older names of the same codes
SPEC_ROW_TOKEN, SPEC_ROW_TARGET, SPEC_ROW_DRAFT, SPEC_ROW_TREE, SPEC_ROW_MASK, SPEC_ROW_WARP = 1, 2, 4, 8, 16, 32
SPEC_ROW_CACHE, SPEC_ROW_TIMEOUT = 64, 128

P = ctypes.c_void_p
I = ctypes.c_int
F = ctypes.c_float
Z = ctypes.c_size_t
L = ctypes.c_int64


class Kv8Cache(ctypes.Structure):
    """spec_kv8_cache of include/specverify.h."""

    _fields_ = ([(n, P) for n in ("k", "v", "k_scale", "v_scale", "block_table", "cache_len")] +
                [(n, ctypes.c_int32) for n in ("B", "num_blocks", "max_blocks", "block", "kv_heads", "head_dim")] +
                [(n, L) for n in ("stride_block", "stride_head", "stride_slot")])

class LatentCache(ctypes.Structure):
    """spec_latent_cache of include/specverify.h."""

    _fields_ = ([(n, P) for n in ("data", "block_table", "cache_len")] +
                [(n, ctypes.c_int32) for n in ("B", "num_blocks", "max_blocks", "block", "latent_dim", "rot_dim", "dtype")] +
                [(n, L) for n in ("stride_block", "stride_slot")])


class PagesPool(ctypes.Structure):
    """spec_pages_pool of include/specverify.h."""

    _fields_ = [("data", P), ("n_planes", ctypes.c_int32)] + [(n, L) for n in ("stride_plane", "stride_block", "block_bytes")]


SIGNATURES = {
    "spec_workspace_bytes": (Z, [I, I, I, I]),
    "spec_warped_workspace_bytes": (Z, [I, I, I, I]),
    "spec_verify_chain": (I, [P, P, I, P, P, P, F, I, I, I, P, P, P, P, P, P, P, P, Z, P]),
    "spec_verify_chain_noalloc": (I, [P, P, I, P, P, P, F, I, I, I, P, P, P, P, P, P, P, P]),
    "spec_host_workspace_bytes": (Z, [I, I, I, I]),
    "spec_verify_chain_host": (I, [P, P, I, P, P, P, F, I, I, I, P, P, P, P, Z, P]),
    "spec_chain_scan": (I, [P, P, I, P, P, P, F, I, I, I, P, P, P, P, P, P, P, P, Z, P]),
    "spec_chain_sample": (I, [P, P, I, P, P, P, F, I, I, I, P, P, P, P, P, P, P, P, Z, P]),
    "spec_verify_chain_warped": (I, [P, P, I, P, P, P, F, I, F, I, I, I, P, P, P, P, P, P, Z, P]),
    "spec_verify_chain_greedy": (I, [P, I, P, I, I, I, P, P, P, P, P, Z, P]),
    "spec_verify_tree_greedy": (I, [P, I, P, P, P, I, I, I, I, I, I, P, P, P, P, P, P, P, Z, P]),
    "spec_tree_confidence": (I, [P, I, I, I, P, P, P]),
    "spec_merge_trees": (I, [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P, P, P]),
    "spec_tree_entropy": (I, [P, I, F, I, I, I, I, P, P, P, P, P, Z, P]),
    "spec_expand_workspace_bytes": (Z, [I, I, I, I, I]),
    "spec_tree_expand": (I, [P, I, F, P, I, I, I, I, P, P, P, P, P, Z, P]),
    "spec_kv_compact": (I, [P, I, I, I, I, I, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_longlong, P, P, I, P, P, P,
                            P]),
    "spec_kv8_append": (I, [P, P, L, L, P, L, L, I, I, P, P, P, I, I, P, L, L, P, L, L, I, P, P]),
    "spec_kv8_workspace_bytes": (Z, [P, I, I, I]),
    "spec_kv8_attention": (I, [P, P, L, L, I, I, I, P, I, P, F, P, L, L, P, P, Z, P]),
    "spec_kv8_compact": (I, [P, I, L, L, P, I, P, P, P, P]),
    "spec_latent_append": (I, [P, P, L, P, L, I, I, P, P, P, I, P, I, F, P, L, L, P, L, L, I, P, P]),
    "spec_latent_workspace_bytes": (Z, [P, I, I]),
    "spec_latent_attention": (I, [P, P, L, L, I, I, P, I, P, F, P, L, L, P, P, Z, P]),
    "spec_latent_compact": (I, [P, I, L, P, I, P, P, P, P]),
    "spec_pages_workspace_bytes": (Z, [I, I, I]),
    "spec_pages_update": (I, [P, P, P, P, P, P, P, I, I, I, I, P, I, P, P, P, Z, P]),
    "spec_status_string": (ctypes.c_char_p, [I]),
}

_lock = threading.Lock()
_lib = None


class LibraryMissing(ImportError):
    pass


def load(path: str = LIB_PATH):
    """Load the CUDA library once; raise LibraryMissing if it was not built."""
    global _lib
    if _lib is not None:  # loaded: no lock on the per-call path
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise LibraryMissing(
                    f"{path} not found: build it first (python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


class SpecError(RuntimeError):
    def __init__(self, fn: str, code: int):
        msg = load().spec_status_string(code).decode()
        super().__init__(f"{fn} returned {code}: {msg}")
        self.code = code


def check(fn: str, code: int) -> None:
    if code != SPEC_OK:
        raise SpecError(fn, code)
