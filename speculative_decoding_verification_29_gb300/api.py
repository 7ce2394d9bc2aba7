"""Torch-facing binding of the C ABI: argument marshalling only.

Each function takes torch tensors, allocates the outputs (and the
workspace) on the logits' device unless they are passed in, and calls the
C entry point of the same name on the current CUDA stream. Every step of
verification runs in the library's CUDA kernels. Host (CPU) inputs are
copied to ``device`` first; that is the end-to-end path a caller with host
buffers uses.
"""

from __future__ import annotations

import array
import ctypes
import functools
import inspect
import math
from typing import Dict, Optional

import torch

from . import _lib
from ._lib import SPEC_BF16, SPEC_F16, SPEC_F32, check


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, device, dtype=None) -> torch.Tensor:
    if t.is_cuda and (dtype is None or t.dtype == dtype) and t.is_contiguous():
        return t  # the common case, kept cheap: small batches are bound by this host path
    if not t.is_cuda:
        t = t.to(device, non_blocking=True)
    if dtype is not None and t.dtype != dtype:
        t = t.to(dtype)
    return t.contiguous()


def _here(dev: torch.device) -> torch.device:
    """A call's device. Kernels are launched on the current one, which cannot use another's pointers."""
    if dev.index is not None and dev.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {dev}, the current device is cuda:{torch.cuda.current_device()}: kernels are "
                         f"launched there (torch.cuda.device)")
    return dev


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:  # the current stream's handle without building a Stream object
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on_stream(fn):
    """`stream=` of a call that makes tensors of its own: they are made on that stream, where its kernels use them. From the
    current stream's memory they could be a block that work queued there still reads or writes. The outputs are the caller's
    on the current stream, so they are kept until that has passed the point at which they are dropped."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = kw.get("stream") if len(args) <= at else args[at]
        if stream is None:
            return fn(*args, **kw)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        current = torch.cuda.current_stream()
        if stream.cuda_stream == current.cuda_stream:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        for t in out.values():
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(current)
        return out

    return call


def workspace_bytes(B: int, K: int, V: int, dtype) -> int:
    code = dtype if isinstance(dtype, int) else (SPEC_BF16 if dtype == torch.bfloat16 else SPEC_F32)
    return int(_lib.load().spec_workspace_bytes(B, K, V, code))


def warped_workspace_bytes(B: int, K: int, V: int, dtype) -> int:
    """Workspace with room for the stats pass's lane records (half-lane
    maxima), which let spec_verify_chain_warped select top-k sets without a
    second pass over the rows (workspace_bytes suffices, but is slower)."""
    code = dtype if isinstance(dtype, int) else (SPEC_BF16 if dtype == torch.bfloat16 else SPEC_F32)
    return int(_lib.load().spec_warped_workspace_bytes(B, K, V, code))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """Device workspace with a 256-byte aligned start."""
    buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off: off + nbytes]


@_on_stream
def spec_verify_chain(target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature: float,
                      out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                      device="cuda", stream=None, stats: bool = True) -> Dict[str, torch.Tensor]:
    """Chain verification (sampling at T > 0, greedy at T == 0).

    target_logits [B, K+1, V], draft_logits [B, K, V] (bf16 or fp32),
    draft_tokens [B, K] int32, u_accept [B, K] fp32, u_resample [B] fp32.
    Returns accept_len, out_tokens, row_status and (with ``stats``)
    lse_target, lse_draft, p_at_x, q_at_x."""
    lib = _lib.load()
    dev = _here(target_logits.device if target_logits.is_cuda else torch.device(device))
    Lp = _dev(target_logits, dev)
    Lq = _dev(draft_logits, dev)
    x = _dev(draft_tokens, dev, torch.int32)
    ua = _dev(u_accept, dev, torch.float32)
    ur = _dev(u_resample, dev, torch.float32)
    B, K1, V = Lp.shape
    K = K1 - 1
    dt = _dtype_code(Lp)
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty(B, K + 1, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
        if stats:
            out.update(lse_target=torch.empty(B, K + 1, device=dev), lse_draft=torch.empty(B, K, device=dev),
                       p_at_x=torch.empty(B, K, device=dev), q_at_x=torch.empty(B, K, device=dev))
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(B, K, V, dt), dev)
    rc = lib.spec_verify_chain(
        Lp.data_ptr(), Lq.data_ptr(), dt, x.data_ptr(), ua.data_ptr(), ur.data_ptr(), float(temperature), B, K, V,
        out["accept_len"].data_ptr(), out["out_tokens"].data_ptr(), _ptr(out.get("lse_target")),
        _ptr(out.get("lse_draft")), _ptr(out.get("p_at_x")), _ptr(out.get("q_at_x")), out["row_status"].data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(stream))
    check("spec_verify_chain", rc)
    return out


def _prepared_inputs(target_logits, draft_logits, draft_tokens, u_accept, u_resample):
    """The prepared call's inputs exactly as the caller holds them: the
    pointers baked into the call must be the caller's own buffers, or later
    refills would go unseen. Nothing is converted or copied; anything else is
    refused."""
    named = (("target_logits", target_logits), ("draft_logits", draft_logits), ("draft_tokens", draft_tokens),
             ("u_accept", u_accept), ("u_resample", u_resample))
    for name, t in named:
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name}: a torch tensor is required")
    if target_logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"target_logits: bfloat16 or float32 required, got {target_logits.dtype}")
    want = dict(draft_logits=target_logits.dtype, draft_tokens=torch.int32, u_accept=torch.float32,
                u_resample=torch.float32)
    for name, t in named[1:]:
        if t.dtype != want[name]:
            raise ValueError(f"{name}: {want[name]} required, got {t.dtype} (it is not converted: the prepared "
                             f"call must read the caller's own buffer)")
    if target_logits.dim() != 3:
        raise ValueError(f"target_logits must be [B, K+1, V], got {tuple(target_logits.shape)}")
    B, K1, V = target_logits.shape
    K = K1 - 1
    shapes = dict(draft_logits=(B, K, V), draft_tokens=(B, K), u_accept=(B, K), u_resample=(B,))
    for name, t in named[1:]:
        if tuple(t.shape) != shapes[name]:
            raise ValueError(f"{name} must be {list(shapes[name])}, got {list(t.shape)}")
    for name, t in named:
        if not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous tensor is required (a strided view is not copied)")
    dev = target_logits.device
    for name, t in named:
        if t.device.type != "cuda" or t.device != dev:
            raise ValueError(f"{name}: a CUDA tensor on {dev} is required, got {t.device}")
    return B, K, V


def prepare_verify_chain(target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature: float,
                         out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                         stats: bool = False):
    """spec_verify_chain on fixed device buffers, for a serving loop that
    refills the same tensors every step: the checks and the argument
    marshalling happen once here, and the returned function enqueues one
    verification on the current stream (or on the stream it is given) and
    returns ``out``. The inputs must be contiguous CUDA tensors on one device
    with the call's dtypes (bf16 or fp32 logits of one dtype, int32 tokens,
    fp32 uniforms): the call keeps their addresses, so a tensor that would
    need a conversion is refused (ValueError) rather than silently replaced
    by a copy. The tensors must stay alive and keep their shapes; their
    contents may change between calls. Outputs and workspace are made here, on
    the current stream: a stream that the function is given later has to be
    ordered behind it."""
    B, K, V = _prepared_inputs(target_logits, draft_logits, draft_tokens, u_accept, u_resample)
    lib = _lib.load()
    dev = target_logits.device
    Lp = target_logits
    dt = _dtype_code(Lp)
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty(B, K + 1, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
        if stats:
            out.update(lse_target=torch.empty(B, K + 1, device=dev), lse_draft=torch.empty(B, K, device=dev),
                       p_at_x=torch.empty(B, K, device=dev), q_at_x=torch.empty(B, K, device=dev))
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(B, K, V, dt), dev)
    fn = lib.spec_verify_chain
    head = (Lp.data_ptr(), draft_logits.data_ptr(), dt, draft_tokens.data_ptr(), u_accept.data_ptr(),
            u_resample.data_ptr(), float(temperature), B, K, V, out["accept_len"].data_ptr(),
            out["out_tokens"].data_ptr(), _ptr(out.get("lse_target")), _ptr(out.get("lse_draft")),
            _ptr(out.get("p_at_x")), _ptr(out.get("q_at_x")), out["row_status"].data_ptr(), workspace.data_ptr(),
            workspace.numel())
    # the buffers the pointers refer to stay alive with the function
    keep = (target_logits, draft_logits, draft_tokens, u_accept, u_resample, workspace)
    index = dev.index if dev.index is not None else torch.cuda.current_device()

    def call(stream=None):
        rc = fn(*head, _raw_stream(index) if stream is None and _raw_stream is not None else _stream(stream))
        if rc:
            check("spec_verify_chain", rc)
        return out

    call.buffers = keep
    return call


def host_workspace_bytes(B: int, K: int, V: int, dtype) -> int:
    """Device workspace for spec_verify_chain_host (staged inputs and
    outputs plus the verification workspace)."""
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(_lib.load().spec_host_workspace_bytes(B, K, V, code))


def _host(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if t.device.type != "cpu" or not t.is_contiguous() or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name}: a contiguous CPU tensor{'' if dtype is None else f' of {dtype}'} is required")
    return t


@_on_stream
def spec_verify_chain_host(target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature: float,
                           out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                           device="cuda", stream=None, synchronize: bool = True) -> Dict[str, torch.Tensor]:
    """Chain verification from host (CPU) tensors through
    spec_verify_chain_host: the library copies the inputs to the device,
    verifies and copies accept_len, out_tokens and row_status back into host
    tensors (pinned, allocated unless ``out`` holds them). Inputs: contiguous
    CPU tensors as spec_verify_chain takes them (pinned memory makes the
    copies asynchronous). With ``synchronize`` the stream is synchronised
    before returning; otherwise the caller synchronises it before reading the
    outputs and keeps the inputs alive until then."""
    lib = _lib.load()
    dev = torch.device(device)
    Lp = _host(target_logits, "target_logits")
    dt = _dtype_code(Lp)
    B, K1, V = Lp.shape
    K = K1 - 1
    sampling = float(temperature) != 0.0
    Lq = _host(draft_logits, "draft_logits", Lp.dtype) if sampling else None
    x = _host(draft_tokens, "draft_tokens", torch.int32)
    ua = _host(u_accept, "u_accept", torch.float32) if sampling else None
    ur = _host(u_resample, "u_resample", torch.float32) if sampling else None
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, pin_memory=True),
                   out_tokens=torch.empty(B, K + 1, dtype=torch.int32, pin_memory=True),
                   row_status=torch.empty(B, dtype=torch.int32, pin_memory=True))
    if workspace is None:
        workspace = alloc_workspace(host_workspace_bytes(B, K, V, dt), dev)
    st = _stream(stream)
    rc = lib.spec_verify_chain_host(
        Lp.data_ptr(), _ptr(Lq), dt, x.data_ptr(), _ptr(ua), _ptr(ur), float(temperature), B, K, V,
        out["accept_len"].data_ptr(), out["out_tokens"].data_ptr(), out["row_status"].data_ptr(),
        workspace.data_ptr(), workspace.numel(), st)
    check("spec_verify_chain_host", rc)
    if synchronize:
        if stream is None:
            torch.cuda.current_stream(dev).synchronize()
        elif hasattr(stream, "synchronize"):
            stream.synchronize()
        else:
            torch.cuda.ExternalStream(st).synchronize()
    return out


def _stage(name, target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature: float,
           out: Dict[str, torch.Tensor], workspace: torch.Tensor, stream=None) -> None:
    B, K1, V = target_logits.shape
    fn = getattr(_lib.load(), name)
    rc = fn(target_logits.data_ptr(), draft_logits.data_ptr(), _dtype_code(target_logits), draft_tokens.data_ptr(),
            u_accept.data_ptr(), u_resample.data_ptr(), float(temperature), B, K1 - 1, V, out["accept_len"].data_ptr(),
            out["out_tokens"].data_ptr(), _ptr(out.get("lse_target")), _ptr(out.get("lse_draft")),
            _ptr(out.get("p_at_x")), _ptr(out.get("q_at_x")), out["row_status"].data_ptr(), workspace.data_ptr(),
            workspace.numel(), _stream(stream))
    check(name, rc)


def spec_chain_scan(target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature: float,
                    out: Dict[str, torch.Tensor], workspace: torch.Tensor, stream=None) -> None:
    """Stage A only: streaming pass, normalisers and the acceptance decision
    (device tensors, outputs preallocated as spec_verify_chain returns them)."""
    _stage("spec_chain_scan", target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature, out,
           workspace, stream)


def spec_chain_sample(target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature: float,
                      out: Dict[str, torch.Tensor], workspace: torch.Tensor, stream=None) -> None:
    """Stage B only: the residual / bonus draw (after spec_chain_scan)."""
    _stage("spec_chain_sample", target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature, out,
           workspace, stream)


@_on_stream
def spec_verify_chain_greedy(target_logits, draft_tokens, out: Optional[Dict[str, torch.Tensor]] = None,
                             workspace: Optional[torch.Tensor] = None, device="cuda",
                             stream=None) -> Dict[str, torch.Tensor]:
    """Greedy chain verification: accept_len, out_tokens, argmax_ids, row_status."""
    lib = _lib.load()
    dev = _here(target_logits.device if target_logits.is_cuda else torch.device(device))
    Lp = _dev(target_logits, dev)
    x = _dev(draft_tokens, dev, torch.int32)
    B, K1, V = Lp.shape
    K = K1 - 1
    dt = _dtype_code(Lp)
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty(B, K + 1, dtype=torch.int32, device=dev),
                   argmax_ids=torch.empty(B, K + 1, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(B, K, V, dt), dev)
    rc = lib.spec_verify_chain_greedy(Lp.data_ptr(), dt, x.data_ptr(), B, K, V, out["accept_len"].data_ptr(),
                                      out["out_tokens"].data_ptr(), _ptr(out.get("argmax_ids")),
                                      out["row_status"].data_ptr(), workspace.data_ptr(), workspace.numel(),
                                      _stream(stream))
    check("spec_verify_chain_greedy", rc)
    return out


@_on_stream
def spec_verify_tree_greedy(node_logits, node_tokens, retrieve_indices, n1: int, tree_mask=None,
                            out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                            device="cuda", stream=None) -> Dict[str, torch.Tensor]:
    """Merged-tree greedy verification: accept_len, best_row, path_nodes,
    out_tokens, subtree, row_status."""
    lib = _lib.load()
    dev = _here(node_logits.device if node_logits.device.type == "cuda" else torch.device(device))
    Lt = _dev(node_logits, dev)
    tok = _dev(node_tokens, dev, torch.int32)
    R = _dev(retrieve_indices, dev, torch.int32)
    mask = None if tree_mask is None else _dev(tree_mask, dev, torch.uint8)
    B, N, V = Lt.shape
    Rn, D = R.shape[1], R.shape[2]
    dt = _dtype_code(Lt)
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   best_row=torch.empty(B, dtype=torch.int32, device=dev),
                   path_nodes=torch.empty(B, D, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty(B, D, dtype=torch.int32, device=dev),
                   subtree=torch.empty(B, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(B, N - 1, V, dt), dev)
    rc = lib.spec_verify_tree_greedy(Lt.data_ptr(), dt, tok.data_ptr(), R.data_ptr(), _ptr(mask), B, N, Rn, D, V,
                                     int(n1), out["accept_len"].data_ptr(), out["best_row"].data_ptr(),
                                     out["path_nodes"].data_ptr(), out["out_tokens"].data_ptr(),
                                     out["subtree"].data_ptr(), out["row_status"].data_ptr(), workspace.data_ptr(),
                                     workspace.numel(), _stream(stream))
    check("spec_verify_tree_greedy", rc)
    return out


@_on_stream
def spec_tree_confidence(node_conf, n1: int, out: Optional[Dict[str, torch.Tensor]] = None, device="cuda",
                         stream=None) -> Dict[str, torch.Tensor]:
    """Confidence routing: scores [B, 2] and choice [B] (1 or 2)."""
    lib = _lib.load()
    dev = _here(node_conf.device if node_conf.device.type == "cuda" else torch.device(device))
    c = _dev(node_conf, dev, torch.float32)
    B, N = c.shape
    if out is None:
        out = dict(scores=torch.empty(B, 2, device=dev), choice=torch.empty(B, dtype=torch.int32, device=dev))
    rc = lib.spec_tree_confidence(c.data_ptr(), B, N, int(n1), out["scores"].data_ptr(), out["choice"].data_ptr(),
                                  _stream(stream))
    check("spec_tree_confidence", rc)
    return out


@_on_stream
def spec_kv_compact(kv: torch.Tensor, base_pos, accept_len, path=None, out: Optional[Dict[str, torch.Tensor]] = None,
                    stream=None) -> Dict[str, torch.Tensor]:
    """KV-cache compaction after verification, in place on ``kv``.

    kv: a CUDA tensor viewed as [planes, B, S, W] (any strides, last dimension
    contiguous), for example a [layers * 2, B, S, heads * head_dim] cache.
    base_pos [B] int32: position of node 0; accept_len [B] int32 and path
    [B, D] int32 (None for chain verification) as returned by the
    verification call. Returns new_len [B] and row_status [B]."""
    lib = _lib.load()
    if kv.device.type != "cuda":
        raise ValueError("kv must be a CUDA tensor (it is compacted in place)")
    if kv.dim() != 4 or kv.stride(3) != 1:
        raise ValueError("kv must be viewed as [planes, B, S, W] with a contiguous last dimension")
    P_, B, S, W = kv.shape
    sp, sb, ss, _ = kv.stride()
    dev = _here(kv.device)
    base = _dev(torch.as_tensor(base_pos), dev, torch.int32)
    acc = _dev(torch.as_tensor(accept_len), dev, torch.int32)
    pth = None if path is None else _dev(torch.as_tensor(path), dev, torch.int32)
    if out is None:
        out = dict(new_len=torch.empty(B, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
    D = 0 if pth is None else pth.shape[1]
    check("spec_kv_compact", lib.spec_kv_compact(kv.data_ptr(), kv.element_size(), P_, B, S, W, sp, sb, ss,
                                                 _ptr(base), _ptr(pth), D, _ptr(acc), _ptr(out["new_len"]),
                                                 _ptr(out["row_status"]), _stream(stream)))
    return out


# -------------------------------------------------- the 8-bit paged KV cache --

_KV8_DTYPES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}


def _kv8_cache(k_cache, v_cache, k_scale, v_scale, block_table, cache_len, planes: bool = False):
    """The C record of a cache and its tensors' device, checked; the tensors stay the caller's. With ``planes`` the
    codes and scales have a leading plane dimension."""
    dev = k_cache.device
    shape, stride = k_cache.shape, k_cache.stride()
    if dev.type != "cuda" or v_cache.device != dev:
        raise ValueError("k_cache and v_cache must be CUDA tensors of one device (the cache lives there)")
    _here(dev)
    if len(shape) != 4 + planes or v_cache.shape != shape or v_cache.stride() != stride:
        raise ValueError("k_cache and v_cache must both be [blocks, kv_heads, block, head_dim], with the same strides")
    if k_cache.element_size() != 1 or v_cache.element_size() != 1 or stride[-1] != 1:
        raise ValueError("k_cache and v_cache hold one byte per code (uint8 or float8_e4m3fn), head_dim contiguous")
    nb, H, bs, D = shape[-4:]
    for t in (k_scale, v_scale):
        if t.device != dev or t.element_size() != 1 or t.shape != shape[:-2] or t.stride()[-2:] != (H, 1):
            raise ValueError("k_scale and v_scale must be [blocks, kv_heads] tensors of bytes (uint8 or float8_e8m0fnu), "
                             "contiguous in each plane")
    _int32(block_table, "block_table", dev)
    _int32(cache_len, "cache_len", dev)
    B = cache_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B or cache_len.dim() != 1:
        raise ValueError("block_table must be [B, max_blocks] and cache_len [B]")
    return _lib.Kv8Cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                         block_table.data_ptr(), cache_len.data_ptr(), B, nb, block_table.shape[1], bs, H, D,
                         stride[-4], stride[-3], stride[-2]), dev


def _int32(t, name, dev, n=0):
    if t.dtype != torch.int32 or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on {dev}")
    if t.numel() < n:
        raise ValueError(f"{name} must have {n} entries, not {t.numel()}")


def _kv8_rows(t, name, D, dev, written=False):
    """The token and head strides of a packed [T, heads, head_dim] activation; one that is written has no rows that share
    memory."""
    stride = t.stride()
    if t.device != dev or len(stride) != 3 or t.shape[2] != D or stride[2] != 1:
        raise ValueError(f"{name} must be a [tokens, heads, {D}] tensor on {dev}, head_dim contiguous")
    if t.dtype not in _KV8_DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if written and (stride[0] < D and t.shape[0] > 1 or stride[1] < D and t.shape[1] > 1):
        raise ValueError(f"{name} is written: its rows must not overlap")
    return stride[0], stride[1]


def _rows_meet(x, y):
    """Whether rows of two [tokens, heads, D] activations of the same tokens and heads share memory."""
    T, H, D = x.shape
    if T == 0 or H == 0:
        return False
    size, (xt, xh, _), (yt, yh, _) = x.element_size(), x.stride(), y.stride()
    off, V = y.data_ptr() - x.data_ptr(), y.shape[2]
    if off >= ((T - 1) * xt + (H - 1) * xh + D) * size or -off >= ((T - 1) * yt + (H - 1) * yh + V) * size:
        return False  # the common case, kept cheap
    return _meet(T, H, off, xt * size, xh * size, D * size, yt * size, yh * size, V * size)


def _meets_itself(x, y):
    """Whether y, of x's shape, is written over other rows of x than its own."""
    same = x.data_ptr() == y.data_ptr() and all(n < 2 or a == b for n, a, b in zip(x.shape, x.stride(), y.stride()))
    return not same and _rows_meet(x, y)


@functools.lru_cache(maxsize=64)
def _meet(T: int, H: int, off: int, xt: int, xh: int, W: int, yt: int, yh: int, V: int) -> bool:
    """Whether rows of W bytes at t * xt + h * xh and of V bytes at off + t * yt + h * yh, t < T, h < H, share a byte."""
    xs, ys = (H - 1) * xh + W, (H - 1) * yh + V
    if xt == yt and max(xs, ys) <= xt and xs <= off % xt <= xt - ys:
        return False  # side by side in every token
    if (xt, xh) == (yt, yh) and xh > 0 and xt % xh == 0 and W <= off % xh <= xh - V:
        return False  # side by side in every head
    if T * H > 1 << 24:
        return True  # not looked at row by row
    t, h = torch.arange(T, device="cpu")[:, None], torch.arange(H, device="cpu")
    x, y = (t * xt + h * xh).flatten().sort().values, (off + t * yt + h * yh).flatten()
    before = torch.searchsorted(x, y + V) - 1  # the last row of x that begins before y's ends
    return bool(((before >= 0) & (x[before.clamp(min=0)] + W > y)).any())


def _kv8_workspace(t, dev):
    if t.device != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")


@_on_stream
def spec_kv8_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, cu_tokens, *, inv_freq=None,
                    interleaved: bool = False, positions=None, q=None, q_out=None,
                    out: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Append the step's keys and values to an 8-bit paged cache, keys rotated.

    k, v [T, kv_heads, head_dim] (fp32, bf16 or fp16; any token and head
    strides): the packed step tokens, sequence b's at cu_tokens[b] ..
    cu_tokens[b + 1] - 1 (cu_tokens [B + 1] int32), stored at positions
    cache_len[b] + i. Cache: k_cache, v_cache [blocks, kv_heads, block,
    head_dim] (uint8 or float8_e4m3fn codes; strides multiples of 16),
    k_scale, v_scale [blocks, kv_heads] (uint8 or float8_e8m0fnu), block_table
    [B, max_blocks] int32, cache_len [B] int32 (not changed by the call).
    inv_freq: the rotation's rot_dim / 2 angular frequencies (a sequence or a
    CPU float64 tensor; None: no rotation), pairs (i, i + rot_dim / 2) or, with
    ``interleaved``, (2 i, 2 i + 1); positions [T] int32 where a token is rotated
    by another position than it is stored at (tree nodes: cache_len + depth).
    q [T, q_heads, head_dim]: queries, rotated alike into q_out (allocated when
    None; may be q, must not overlap it otherwise). Returns row_status [B] and, with q, q_out."""
    lib = _lib.load()
    cache, dev = _kv8_cache(k_cache, v_cache, k_scale, v_scale, block_table, cache_len)
    D = cache.head_dim
    kst, ksh = _kv8_rows(k, "k", D, dev)
    vst, vsh = _kv8_rows(v, "v", D, dev)
    T, H, _ = k.shape
    if v.shape != k.shape or v.dtype != k.dtype or H != cache.kv_heads:
        raise ValueError("k and v must have the same type and shape [tokens, kv_heads, head_dim]")
    _int32(cu_tokens, "cu_tokens", dev)
    if cu_tokens.numel() != cache.B + 1:
        raise ValueError("cu_tokens must have B + 1 entries")
    if positions is not None:
        _int32(positions, "positions", dev)
        if positions.numel() != T:
            raise ValueError("positions must have one entry per token")
    qst = qsh = ost = osh = hq = 0
    if q is not None:
        qst, qsh = _kv8_rows(q, "q", D, dev)
        given = q_out is not None
        if not given:
            q_out = torch.empty_like(q)
        ost, osh = _kv8_rows(q_out, "q_out", D, dev, True)
        if q.dtype != k.dtype or q_out.dtype != q.dtype or q.shape[0] != T or q_out.shape != q.shape:
            raise ValueError("q and q_out must be [tokens, q_heads, head_dim] of the keys' type")
        if given and _meets_itself(q, q_out):
            raise ValueError("q_out must be q or not overlap it")
        hq = q.shape[1]
    rot, freq, held = 0, None, None
    if inv_freq is not None:
        if isinstance(inv_freq, torch.Tensor):
            held = inv_freq.detach().to("cpu", torch.float64).contiguous()
            rot, freq = 2 * held.numel(), held.data_ptr()
        else:
            held = array.array("d", inv_freq)
            rot, freq = 2 * len(held), held.buffer_info()[0]
    if out is None:
        out = dict(row_status=torch.empty(cache.B, dtype=torch.int32, device=dev))
    else:
        _int32(out["row_status"], "row_status", dev, cache.B)
    if q is not None:
        out["q_out"] = q_out
    check("spec_kv8_append", lib.spec_kv8_append(
        ctypes.byref(cache), k.data_ptr(), kst, ksh, v.data_ptr(), vst, vsh, _KV8_DTYPES[k.dtype], T, cu_tokens.data_ptr(),
        _ptr(positions), freq, rot, int(bool(interleaved)), _ptr(q), qst, qsh, None if q is None else q_out.data_ptr(), ost,
        osh, hq, out["row_status"].data_ptr(), _stream(stream)))
    return out


def kv8_workspace_bytes(k_cache, block_table, q_heads: int, max_tokens: int, dtype) -> int:
    """Workspace of spec_kv8_attention for a cache's sizes, the query heads and the longest step."""
    nb, H, bs, D = k_cache.shape
    sb, sh, ss, _ = k_cache.stride()
    cache = _lib.Kv8Cache(*[k_cache.data_ptr()] * 6, block_table.shape[0], nb, block_table.shape[1], bs, H, D, sb, sh, ss)
    code = dtype if isinstance(dtype, int) else _KV8_DTYPES[dtype]
    return int(_lib.load().spec_kv8_workspace_bytes(ctypes.byref(cache), q_heads, max_tokens, code))


@_on_stream
def spec_kv8_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, cu_tokens, *, max_tokens: int,
                       sm_scale: Optional[float] = None, tree_mask=None,
                       out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> Dict[str, torch.Tensor]:
    """Attention of the step's queries over an 8-bit paged cache that already
    holds the step's tokens (spec_kv8_append).

    q [T, q_heads, head_dim] (bf16 or fp16; any token and head strides), packed
    as the tokens of spec_kv8_append, whose cache arguments it shares; query
    head a reads KV head a // (q_heads // kv_heads). Token i of sequence b sees the
    cache_len[b] tokens of the context and the step's tokens j <= i, or with
    tree_mask [B, max_tokens, max_tokens] uint8 (as written by spec_merge_trees)
    those with tree_mask[b, i, j] != 0. max_tokens: no sequence has more step
    tokens. sm_scale: head_dim ** -0.5 when None. Returns out (like q) and
    row_status [B]; a caller's own out["out"] may have any token and head
    strides, but must not overlap q."""
    lib = _lib.load()
    cache, dev = _kv8_cache(k_cache, v_cache, k_scale, v_scale, block_table, cache_len)
    qst, qsh = _kv8_rows(q, "q", cache.head_dim, dev)
    if q.dtype == torch.float32:
        raise TypeError("q must be bfloat16 or float16")
    T, hq, _ = q.shape
    _int32(cu_tokens, "cu_tokens", dev)
    if cu_tokens.numel() != cache.B + 1:
        raise ValueError("cu_tokens must have B + 1 entries")
    if tree_mask is not None:
        if tree_mask.device != dev or tree_mask.element_size() != 1 or not tree_mask.is_contiguous() or \
                tree_mask.shape != (cache.B, max_tokens, max_tokens):
            raise ValueError("tree_mask must be a contiguous [B, max_tokens, max_tokens] tensor of bytes")
    code = _KV8_DTYPES[q.dtype]
    if out is None:
        out = dict(out=torch.empty_like(q), row_status=torch.empty(cache.B, dtype=torch.int32, device=dev))
    else:
        _int32(out["row_status"], "row_status", dev, cache.B)
    o = out["out"]
    ost, osh = _kv8_rows(o, "out", cache.head_dim, dev, True)
    if o.shape != q.shape or o.dtype != q.dtype:
        raise ValueError("out must have q's shape and type")
    if _rows_meet(q, o):
        raise ValueError("out must not overlap q: queries are read again after the first results were written")
    if workspace is None:
        nbytes = lib.spec_kv8_workspace_bytes(ctypes.byref(cache), hq, max_tokens, code)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if workspace.data_ptr() % 256:
            workspace = alloc_workspace(nbytes, dev)
    else:
        _kv8_workspace(workspace, dev)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(cache.head_dim)
    check("spec_kv8_attention", lib.spec_kv8_attention(
        ctypes.byref(cache), q.data_ptr(), qst, qsh, code, T, hq, cu_tokens.data_ptr(), max_tokens, _ptr(tree_mask),
        sm_scale, o.data_ptr(), ost, osh, out["row_status"].data_ptr(), workspace.data_ptr(), workspace.numel(),
        _stream(stream)))
    return out


@_on_stream
def spec_kv8_compact(k_cache, v_cache, k_scale, v_scale, block_table, cache_len, accept_len, path=None,
                     out: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Compaction of an 8-bit paged cache along the accepted path of a tree
    verification, in place.

    k_cache, v_cache [blocks, kv_heads, block, head_dim] with k_scale, v_scale
    [blocks, kv_heads], or, for layers that share the block table, [planes, ...] of
    each (any plane stride). cache_len [B]: position of node 0; accept_len [B] and
    path [B, D] (None for chain verification) as returned by the verification
    call. Returns new_len [B] and row_status [B]."""
    lib = _lib.load()
    planes, sp, ssp = 1, 0, 0
    cache, dev = _kv8_cache(k_cache, v_cache, k_scale, v_scale, block_table, cache_len, k_cache.dim() == 5)
    if k_cache.dim() == 5:
        planes, sp, ssp = k_cache.shape[0], k_cache.stride(0), k_scale.stride(0)
        if v_scale.stride(0) != ssp:
            raise ValueError("k_scale and v_scale must have the same plane stride")
    _int32(accept_len, "accept_len", dev)
    if accept_len.numel() != cache.B:
        raise ValueError("accept_len must have B entries")
    D = 0
    if path is not None:
        _int32(path, "path", dev)
        if path.dim() != 2 or path.shape[0] != cache.B:
            raise ValueError("path must be [B, D]")
        D = path.shape[1]
    if out is None:
        out = dict(new_len=torch.empty(cache.B, dtype=torch.int32, device=dev),
                   row_status=torch.empty(cache.B, dtype=torch.int32, device=dev))
    else:
        _int32(out["new_len"], "new_len", dev, cache.B)
        _int32(out["row_status"], "row_status", dev, cache.B)
    check("spec_kv8_compact", lib.spec_kv8_compact(ctypes.byref(cache), planes, sp, ssp, _ptr(path), D,
                                                   accept_len.data_ptr(), out["new_len"].data_ptr(),
                                                   out["row_status"].data_ptr(), _stream(stream)))
    return out


@_on_stream
def spec_tree_entropy(draft_logits, n1: int, temperature: float = 1.0, out: Optional[Dict[str, torch.Tensor]] = None,
                      workspace: Optional[torch.Tensor] = None, device="cuda", stream=None,
                      node_entropy: bool = True) -> Dict[str, torch.Tensor]:
    """Entropy routing over merged drafter trees: draft_logits [B, N, V]
    (bf16 or fp32). Returns scores [B, 2], choice [B], row_status [B] and
    (with ``node_entropy``) the per-node entropies [B, N]."""
    lib = _lib.load()
    dev = _here(draft_logits.device if draft_logits.device.type == "cuda" else torch.device(device))
    Ld = _dev(draft_logits, dev)
    B, N, V = Ld.shape
    code = _dtype_code(Ld)
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(B, N, V, code), dev)
    if out is None:
        out = dict(scores=torch.empty(B, 2, dtype=torch.float32, device=dev),
                   choice=torch.empty(B, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
        if node_entropy:
            out["node_entropy"] = torch.empty(B, N, dtype=torch.float32, device=dev)
    check("spec_tree_entropy", lib.spec_tree_entropy(Ld.data_ptr(), code, float(temperature), B, N, V, int(n1),
                                                     _ptr(out.get("node_entropy")), _ptr(out["scores"]),
                                                     _ptr(out["choice"]), _ptr(out["row_status"]),
                                                     workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out


@_on_stream
def spec_tree_expand(draft_logits, logc, M: int, temperature: float = 1.0,
                     out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                     device="cuda", stream=None) -> Dict[str, torch.Tensor]:
    """One drafter-tree expansion step by cumulative probability:
    draft_logits [B, F, V] (bf16 or fp32) at the F frontier nodes, logc [B, F]
    their paths' log cumulative probabilities. Returns the M best children
    as parent, token [B, M] int32, score [B, M] fp32 and row_status [B]."""
    lib = _lib.load()
    dev = _here(draft_logits.device if draft_logits.device.type == "cuda" else torch.device(device))
    Ld = _dev(draft_logits, dev)
    B, F, V = Ld.shape
    lc = _dev(logc, dev, torch.float32)
    if tuple(lc.shape) != (B, F):
        raise ValueError(f"logc must be [{B}, {F}], got {tuple(lc.shape)}")
    code = _dtype_code(Ld)
    if workspace is None:
        need = lib.spec_expand_workspace_bytes(B, F, V, int(M), code)
        if need == 0:
            check("spec_expand_workspace_bytes", _lib.SPEC_ERR_UNSUPPORTED)
        workspace = alloc_workspace(need, dev)
    if out is None:
        out = dict(parent=torch.empty(B, M, dtype=torch.int32, device=dev),
                   token=torch.empty(B, M, dtype=torch.int32, device=dev),
                   score=torch.empty(B, M, dtype=torch.float32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev))
    check("spec_tree_expand", lib.spec_tree_expand(Ld.data_ptr(), code, float(temperature), lc.data_ptr(), B, F, V,
                                                   int(M), out["parent"].data_ptr(), out["token"].data_ptr(),
                                                   out["score"].data_ptr(), out["row_status"].data_ptr(),
                                                   workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out


@_on_stream
def spec_merge_trees(tokens1, mask1, retrieve1, pos1, tokens2, mask2, retrieve2, pos2, device="cuda",
                     stream=None) -> Dict[str, torch.Tensor]:
    """Merge B pairs of drafter trees under one shared root on the device.

    tokens* [B, n+1] int32, mask* [B, n+1, n+1] uint8, retrieve* [B, R, D]
    int32, pos* [B, n+1] int32. Returns tokens [B, N], mask [B, N, N],
    retrieve [B, R1+R2, max(D1, D2)], pos [B, N] and n1."""
    lib = _lib.load()
    dev = _here(tokens1.device if tokens1.device.type == "cuda" else torch.device(device))
    t1, t2 = _dev(tokens1, dev, torch.int32), _dev(tokens2, dev, torch.int32)
    m1, m2 = _dev(mask1, dev, torch.uint8), _dev(mask2, dev, torch.uint8)
    r1, r2 = _dev(retrieve1, dev, torch.int32), _dev(retrieve2, dev, torch.int32)
    p1, p2 = _dev(pos1, dev, torch.int32), _dev(pos2, dev, torch.int32)
    B, n1, n2 = t1.shape[0], t1.shape[1] - 1, t2.shape[1] - 1
    N, (R1, D1), (R2, D2) = n1 + n2 + 1, r1.shape[1:], r2.shape[1:]
    D = max(D1, D2)
    out = dict(tokens=torch.empty(B, N, dtype=torch.int32, device=dev),
               mask=torch.empty(B, N, N, dtype=torch.uint8, device=dev),
               retrieve=torch.empty(B, R1 + R2, D, dtype=torch.int32, device=dev),
               pos=torch.empty(B, N, dtype=torch.int32, device=dev))
    check("spec_merge_trees", lib.spec_merge_trees(_ptr(t1), _ptr(m1), _ptr(r1) if R1 else None, _ptr(p1), _ptr(t2),
                                                   _ptr(m2), _ptr(r2) if R2 else None, _ptr(p2), B, n1, n2, R1, D1,
                                                   R2, D2, _ptr(out["tokens"]), _ptr(out["mask"]),
                                                   _ptr(out["retrieve"]), _ptr(out["pos"]), _stream(stream)))
    out["n1"] = n1
    return out


@_on_stream
def spec_verify_chain_warped(target_logits, draft_logits, draft_tokens, u_accept, u_resample, temperature: float,
                             top_k: int = 0, top_p: float = 1.0, out: Optional[Dict[str, torch.Tensor]] = None,
                             workspace: Optional[torch.Tensor] = None, device="cuda",
                             stream=None) -> Dict[str, torch.Tensor]:
    """Chain verification with top-k / top-p applied to p and q (0 and 1.0:
    off). Returns accept_len, out_tokens, row_status, p_at_x, q_at_x."""
    lib = _lib.load()
    dev = _here(target_logits.device if target_logits.is_cuda else torch.device(device))
    Lp, Lq = _dev(target_logits, dev), _dev(draft_logits, dev)
    B, K1, V = Lp.shape
    K = K1 - 1
    x = _dev(draft_tokens, dev, torch.int32)
    ua = _dev(u_accept, dev, torch.float32)
    ur = _dev(u_resample, dev, torch.float32)
    code = _dtype_code(Lp)
    if workspace is None:
        workspace = alloc_workspace(warped_workspace_bytes(B, K, V, code), dev)
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty(B, K + 1, dtype=torch.int32, device=dev),
                   row_status=torch.empty(B, dtype=torch.int32, device=dev),
                   p_at_x=torch.empty(B, K, dtype=torch.float32, device=dev),
                   q_at_x=torch.empty(B, K, dtype=torch.float32, device=dev))
    check("spec_verify_chain_warped",
          lib.spec_verify_chain_warped(Lp.data_ptr(), Lq.data_ptr(), code, _ptr(x), _ptr(ua), _ptr(ur),
                                       float(temperature), int(top_k), float(top_p), B, K, V,
                                       _ptr(out["accept_len"]), _ptr(out["out_tokens"]), _ptr(out.get("p_at_x")),
                                       _ptr(out.get("q_at_x")), _ptr(out["row_status"]), workspace.data_ptr(),
                                       workspace.numel(), _stream(stream)))
    return out
