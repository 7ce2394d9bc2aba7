"""Torch-facing binding of the paged latent cache and of the pages under a cache: argument marshalling only, in the manner
of ``api``."""

from __future__ import annotations

import array
import ctypes
import functools
from typing import Dict, Optional

import torch

from . import _lib
from ._lib import SPEC_BF16, SPEC_F16, SPEC_F32, check
from .api import _here, _int32, _kv8_rows, _kv8_workspace, _meets_itself, _on_stream, _ptr, _raw_stream, _rows_meet, _stream, alloc_workspace

_DTYPES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}


def _whole(t, name, dev, at, n=0):
    """_int32, kept cheap: small calls are bound by this host path. at: the device's index."""
    if t.dtype is not torch.int32 or t.get_device() != at or not t.is_contiguous() or n and t.numel() < n:
        _int32(t, name, dev, n)


def _queue(stream, at):
    return _raw_stream(at) if stream is None and _raw_stream is not None else _stream(stream)


def _cache(cache, block_table, cache_len, latent_dim: int, planes: bool = False):
    """The C record of a cache and its device, checked; the tensors stay the caller's."""
    dev, at = cache.device, cache.get_device()
    if at < 0:
        raise ValueError("cache must be a CUDA tensor (the cache lives there)")
    if at != torch.cuda.current_device():
        _here(dev)
    shape, stride = cache.shape, cache.stride()
    if len(shape) != 3 + planes or stride[-1] != 1:
        raise ValueError("cache must be [blocks, block, latent_dim + rot_dim], an entry contiguous")
    dtype = _DTYPES.get(cache.dtype, SPEC_F32)
    if dtype == SPEC_F32:
        raise TypeError(f"cache must be bfloat16 or float16, got {cache.dtype}")
    nb, bs, W = shape[-3:]
    if not 0 < latent_dim < W:
        raise ValueError(f"an entry of {W} elements cannot hold a latent vector of {latent_dim} and rotated dimensions")
    _whole(block_table, "block_table", dev, at)
    _whole(cache_len, "cache_len", dev, at)
    rows, lens = block_table.shape, cache_len.shape
    if len(rows) != 2 or len(lens) != 1 or rows[0] != lens[0]:
        raise ValueError("block_table must be [B, max_blocks] and cache_len [B]")
    return _lib.LatentCache(cache.data_ptr(), block_table.data_ptr(), cache_len.data_ptr(), rows[0], nb, rows[1], bs,
                            latent_dim, W - latent_dim, dtype, 2 * stride[-3], 2 * stride[-2]), dev, at


def _vectors(t, name, D, dev):
    """The token stride of a packed [T, D] activation."""
    if t.device != dev or t.dim() != 2 or t.shape[1] != D or t.stride(1) != 1:
        raise ValueError(f"{name} must be a [tokens, {D}] tensor on {dev}, a token contiguous")
    return t.stride(0)


def _cu(cu_tokens, B, dev, at):
    _whole(cu_tokens, "cu_tokens", dev, at)
    if cu_tokens.numel() != B + 1:
        raise ValueError("cu_tokens must have B + 1 entries")


@_on_stream
def spec_latent_append(latent, rope_key, cache, block_table, cache_len, cu_tokens, *, inv_freq, interleaved: bool = False,
                       positions=None, norm_weight=None, eps: float = 1e-6, q_rope=None, q_out=None,
                       out: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Append the step's latent vectors, normalised, and their shared key dimensions, rotated, to a paged latent cache.

    latent [T, latent_dim], rope_key [T, rot_dim] (the cache's type or fp32;
    any token stride): the packed step tokens, sequence b's at cu_tokens[b] ..
    cu_tokens[b + 1] - 1 (cu_tokens [B + 1] int32), stored at positions
    cache_len[b] + i. cache [blocks, block, latent_dim + rot_dim] (bf16 or fp16;
    block and slot strides multiples of 16 bytes), block_table [B, max_blocks]
    int32, cache_len [B] int32 (not changed by the call). norm_weight [latent_dim]
    (fp32 or latent's type): the vector is stored as x / sqrt(mean(x^2) + eps) *
    norm_weight; None: as it is. inv_freq, interleaved, positions: as in
    spec_kv8_append, over all rot_dim dimensions. q_rope [T, q_heads, rot_dim]
    of latent's type (any strides, for example the last dimensions of the
    attention's queries): rotated alike into q_out (allocated when None; may be
    q_rope, must not overlap it otherwise). Returns row_status [B] and, with q_rope, q_out."""
    lib = _lib.load()
    if latent.dim() != 2:
        raise ValueError("latent must be [tokens, latent_dim]")
    rec, dev, at = _cache(cache, block_table, cache_len, latent.shape[1])
    T, R = latent.shape[0], rec.rot_dim
    xst, rst = _vectors(latent, "latent", rec.latent_dim, dev), _vectors(rope_key, "rope_key", R, dev)
    if latent.dtype not in (cache.dtype, torch.float32) or rope_key.dtype != latent.dtype:
        raise TypeError("latent and rope_key must both be of the cache's type or float32")
    if rope_key.shape[0] != T:
        raise ValueError("latent and rope_key must have the same tokens")
    _cu(cu_tokens, rec.B, dev, at)
    if positions is not None:
        _whole(positions, "positions", dev, at)
        if positions.numel() != T:
            raise ValueError("positions must have one entry per token")
    wcode = 0
    if norm_weight is not None:
        if norm_weight.device != dev or norm_weight.shape != (rec.latent_dim,) or not norm_weight.is_contiguous():
            raise ValueError(f"norm_weight must be a contiguous [{rec.latent_dim}] tensor on {dev}")
        if norm_weight.dtype not in (latent.dtype, torch.float32):
            raise TypeError("norm_weight must be of latent's type or float32")
        wcode = _DTYPES[norm_weight.dtype]
    qst = qsh = ost = osh = hq = 0
    if q_rope is not None:
        qst, qsh = _kv8_rows(q_rope, "q_rope", R, dev)
        given = q_out is not None
        if not given:
            q_out = q_rope.new_empty(q_rope.shape)
        ost, osh = _kv8_rows(q_out, "q_out", R, dev, True)
        if q_rope.dtype != latent.dtype or q_out.dtype != q_rope.dtype or q_rope.shape[0] != T or q_out.shape != q_rope.shape:
            raise ValueError("q_rope and q_out must be [tokens, q_heads, rot_dim] of latent's type")
        if given and _meets_itself(q_rope, q_out):
            raise ValueError("q_out must be q_rope or not overlap it")
        hq = q_rope.shape[1]
    if isinstance(inv_freq, torch.Tensor):
        held = inv_freq.detach().to("cpu", torch.float64).contiguous()
        n, freq = held.numel(), held.data_ptr()
    else:
        held = array.array("d", inv_freq)
        n, freq = len(held), held.buffer_info()[0]
    if 2 * n != R:
        raise ValueError(f"inv_freq must have {R // 2} entries for {R} rotated dimensions, not {n}")
    if out is None:
        out = dict(row_status=cache_len.new_empty(rec.B))
    else:
        _whole(out["row_status"], "row_status", dev, at, rec.B)
    if q_rope is not None:
        out["q_out"] = q_out
    check("spec_latent_append", lib.spec_latent_append(
        ctypes.byref(rec), latent.data_ptr(), xst, rope_key.data_ptr(), rst, _DTYPES[latent.dtype], T, cu_tokens.data_ptr(),
        _ptr(positions), freq, int(bool(interleaved)), _ptr(norm_weight), wcode, eps, _ptr(q_rope), qst, qsh,
        None if q_rope is None else q_out.data_ptr(), ost, osh, hq, out["row_status"].data_ptr(), _queue(stream, at)))
    return out


def latent_workspace_bytes(cache, value_dim: int, q_heads: int, max_tokens: int) -> int:
    """Workspace of spec_latent_attention for a cache's sizes, the query heads and the longest step."""
    return _attention_bytes(cache.shape[1], value_dim, cache.shape[2] - value_dim, q_heads, max_tokens)


@functools.lru_cache(maxsize=256)
def _attention_bytes(block: int, value_dim: int, rot: int, q_heads: int, max_tokens: int) -> int:
    W = 2 * (value_dim + rot)
    rec = _lib.LatentCache(256, 256, 256, 1, 1, 1, block, value_dim, rot, SPEC_BF16, block * W, W)  # only sizes matter
    return int(_lib.load().spec_latent_workspace_bytes(ctypes.byref(rec), q_heads, max_tokens))


@_on_stream
def spec_latent_attention(q, cache, block_table, cache_len, cu_tokens, *, max_tokens: int, value_dim: int, sm_scale: float,
                          tree_mask=None, out: Optional[Dict[str, torch.Tensor]] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Attention of the step's queries over a paged latent cache that already holds the step's tokens
    (spec_latent_append); all heads read the same entries.

    q [T, q_heads, value_dim + rot_dim] (the cache's type; any token and head
    strides): the keys' up-projection absorbed into its first value_dim
    dimensions, the rest rotated. Token i of sequence b sees the cache_len[b]
    tokens of the context and the step's tokens j <= i, or with tree_mask [B,
    max_tokens, max_tokens] uint8 (as written by spec_merge_trees) those with
    tree_mask[b, i, j] != 0. max_tokens: no sequence has more step tokens.
    sm_scale: of the scores; the heads' own key dimension decides it, which the
    cache does not know. Returns out [T, q_heads, value_dim], to which the
    caller applies the values' up-projection, and row_status [B]; a caller's
    own out["out"] may have any token and head strides, but must not overlap q."""
    lib = _lib.load()
    rec, dev, at = _cache(cache, block_table, cache_len, value_dim)
    qst, qsh = _kv8_rows(q, "q", cache.shape[2], dev)
    if q.dtype != cache.dtype:
        raise TypeError("q must have the cache's type")
    T, hq, _ = q.shape
    _cu(cu_tokens, rec.B, dev, at)
    if tree_mask is not None:
        if tree_mask.device != dev or tree_mask.element_size() != 1 or not tree_mask.is_contiguous() or \
                tree_mask.shape != (rec.B, max_tokens, max_tokens):
            raise ValueError("tree_mask must be a contiguous [B, max_tokens, max_tokens] tensor of bytes")
    if out is None:
        out = dict(out=q.new_empty((T, hq, value_dim)),
                   row_status=cache_len.new_empty(rec.B))
    else:
        _whole(out["row_status"], "row_status", dev, at, rec.B)
    o = out["out"]
    ost, osh = _kv8_rows(o, "out", value_dim, dev, True)
    if o.shape != (T, hq, value_dim) or o.dtype != q.dtype:
        raise ValueError(f"out must be [{T}, {hq}, {value_dim}] of q's type")
    if _rows_meet(q, o):
        raise ValueError("out must not overlap q: queries are read again after the first results were written")
    if workspace is None:
        nbytes = _attention_bytes(rec.block, value_dim, rec.rot_dim, hq, max_tokens)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if workspace.data_ptr() % 256:
            workspace = alloc_workspace(nbytes, dev)
    else:
        _kv8_workspace(workspace, dev)
    check("spec_latent_attention", lib.spec_latent_attention(
        ctypes.byref(rec), q.data_ptr(), qst, qsh, T, hq, cu_tokens.data_ptr(), max_tokens, _ptr(tree_mask), sm_scale,
        o.data_ptr(), ost, osh, out["row_status"].data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _queue(stream, at)))
    return out


@_on_stream
def spec_latent_compact(cache, block_table, cache_len, accept_len, path=None,
                        out: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Compaction of a paged latent cache along the accepted path of a tree verification, in place.

    cache [blocks, block, entry], or, for layers that share the block table,
    [planes, ...] (any plane stride that is a multiple of 16 bytes). cache_len [B]:
    position of node 0; accept_len [B] and path [B, D] (None for chain
    verification) as returned by the verification call. Returns new_len [B]
    and row_status [B]; a caller's own out["new_len"] may be cache_len, which
    then is brought up to date in place."""
    lib = _lib.load()
    W = cache.shape[-1]
    C = (W - 1) // 128 * 128  # entries move whole: how they are divided does not matter here
    rec, dev, at = _cache(cache, block_table, cache_len, C, cache.dim() == 4)
    planes, sp = (cache.shape[0], 2 * cache.stride(0)) if cache.dim() == 4 else (1, 0)
    _whole(accept_len, "accept_len", dev, at)
    if accept_len.numel() != rec.B:
        raise ValueError("accept_len must have B entries")
    D = 0
    if path is not None:
        _whole(path, "path", dev, at)
        if path.dim() != 2 or path.shape[0] != rec.B:
            raise ValueError("path must be [B, D]")
        D = path.shape[1]
    if out is None:
        out = dict(new_len=cache_len.new_empty(rec.B),
                   row_status=cache_len.new_empty(rec.B))
    else:
        _whole(out["new_len"], "new_len", dev, at, rec.B)
        _whole(out["row_status"], "row_status", dev, at, rec.B)
    check("spec_latent_compact", lib.spec_latent_compact(ctypes.byref(rec), planes, sp, _ptr(path), D, accept_len.data_ptr(),
                                                         out["new_len"].data_ptr(), out["row_status"].data_ptr(),
                                                         _queue(stream, at)))
    return out


def _pages_pools(pools, num_blocks, dev, planes):
    """The C records of pools: [blocks, ...] or, with ``planes``, [planes, blocks, ...], a block contiguous."""
    recs = (_lib.PagesPool * max(1, len(pools)))()
    lead = int(planes)
    for rec, t in zip(recs, pools):
        if t.device != dev:
            raise ValueError(f"pools must be on {dev}")
        shape, stride, inner = t.shape, t.stride(), 1
        for i in range(len(shape) - 1, lead, -1):
            if shape[i] != 1 and stride[i] != inner:
                inner = 0
            inner *= shape[i]
        if len(shape) < lead + 2 or shape[lead] != num_blocks or inner == 0:
            raise ValueError(f"pools must be [{'planes, ' * lead}{num_blocks}, ...], the elements of a block contiguous; got "
                             f"{tuple(shape)} with strides {stride}")
        size = t.element_size()
        rec.data, rec.n_planes, rec.stride_plane = t.data_ptr(), shape[0] if lead else 1, stride[0] * size if lead else 0
        rec.stride_block, rec.block_bytes = stride[lead] * size, inner * size
    return recs


@_on_stream
def spec_pages_update(block_table, cache_len, refs, pools=(), *, planes: bool = False, block: Optional[int] = None, keep_len=None, source=None,
                      need=None, out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> Dict[str, torch.Tensor]:
    """The pages of a paged cache between two steps: cut sequences back, fork or end them, and take blocks for the next step.

    block_table [B, max_blocks] int32 (-1 behind a sequence's blocks), cache_len
    [B] int32, refs [num_blocks] int32: how many rows hold a block, 0 for a free
    one; brought up to date in place. Sequence b keeps the first keep_len[b]
    tokens (None: all) of sequence source[b] (None: its own; keep 0 ends it) as it
    was before the call, gives back what it no longer holds, and, where need[b] >
    0 (None: 0), takes free blocks until need[b] more tokens fit, lowest ids first.
    A partly filled block that b goes on writing while others hold it is replaced
    by a copy, in every one of ``pools``: tensors [num_blocks, ...] of a layer
    or, with ``planes``, [planes, num_blocks, ...] of layers that share the table
    (a latent cache; codes and scales of an 8-bit cache), the elements of a block
    contiguous. block: tokens of a block (None: the second last dimension of the
    first pool, as the latent cache and the codes of an 8-bit one have it; a pool of scales does not tell it). out: cache_len, row_status and, where the
    rows are to go elsewhere, block_table; it is not changed. Returns block_table (without one in out: the
    given one, or with source a new one), cache_len [B] (the tokens kept), row_status [B], and refs. A
    sequence with SPEC_ROW_CACHE in row_status must not be appended to. Where blocks do not suffice, that sequence and all later
    ones with need > 0 are marked so and take none; they keep their tokens, and a further call with need 0 for those that have
    to wait serves the others."""
    lib = _lib.load()
    dev, at = block_table.device, block_table.get_device()
    if at < 0:
        raise ValueError("block_table must be a CUDA tensor")
    if at != torch.cuda.current_device():
        _here(dev)
    _whole(block_table, "block_table", dev, at)
    _whole(cache_len, "cache_len", dev, at)
    _whole(refs, "refs", dev, at)
    if block_table.dim() != 2 or cache_len.dim() != 1 or refs.dim() != 1 or block_table.shape[0] != cache_len.numel():
        raise ValueError("block_table must be [B, max_blocks], cache_len [B] and refs [num_blocks]")
    B, M = block_table.shape
    for t, name in ((keep_len, "keep_len"), (source, "source"), (need, "need")):
        if t is not None:
            _whole(t, name, dev, at)
            if t.numel() != B:
                raise ValueError(f"{name} must have B entries")
    if block is None:
        if not len(pools) or pools[0].dim() < 3 + planes:
            raise ValueError("block is needed where the first pool does not tell it: [..., block, elements of a token]")
        block = pools[0].shape[-2]
    n = refs.numel()
    recs = _pages_pools(pools, n, dev, planes)
    if out is None:
        out = dict(cache_len=cache_len.new_empty(B), row_status=cache_len.new_empty(B))
    else:
        _whole(out["cache_len"], "out's cache_len", dev, at, B)
        _whole(out["row_status"], "row_status", dev, at, B)
    table = out.get("block_table")  # the caller's dict is left as it is: no call's rows become the next one's destination
    if table is None:
        table = block_table if source is None else torch.empty_like(block_table)
    _whole(table, "out's block_table", dev, at)
    if table.shape != block_table.shape:
        raise ValueError("out's block_table must have block_table's shape")
    if source is not None and table.data_ptr() == block_table.data_ptr():
        raise ValueError("with source, the new rows cannot be written over the old ones")
    if out["cache_len"].data_ptr() == cache_len.data_ptr():
        raise ValueError("out's cache_len must not be cache_len: it is read until the end of the call")
    if workspace is None:
        nbytes = lib.spec_pages_workspace_bytes(B, M, n)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if workspace.data_ptr() % 256:
            workspace = alloc_workspace(nbytes, dev)
    else:
        _kv8_workspace(workspace, dev)
    check("spec_pages_update", lib.spec_pages_update(
        block_table.data_ptr(), table.data_ptr(), cache_len.data_ptr(), _ptr(keep_len), _ptr(source), _ptr(need),
        refs.data_ptr(), B, M, n, block, recs, len(pools), out["cache_len"].data_ptr(), out["row_status"].data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _queue(stream, at)))
    return dict(out, block_table=table, refs=refs)
