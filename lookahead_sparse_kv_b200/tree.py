"""Draft-tree calls of liboasis.so: one speculative decode step over the sparse KV cache.

``tree_layout``    visibility words and positions of a tree's nodes (once a step)
``qk_norm_rope``   projection rows -> normed and rotated queries, draft keys and values (per layer)
``tree_attn``      attention of the nodes over the resident slots and the tree itself (per layer)
``verify_tree``    which drafted tokens stand, from given random numbers (once a step)
``commit_path``    the accepted rows into the cache of every layer (once a step)

Like the rest of the package this is argument marshalling only; the contract
of each call stands in ``include/oasis.h``.  The names are offered by the
package itself (``lookahead_sparse_kv_b200.tree_attn``).  The calls are made
many times a step on small batches, where the host's time counts, so the
checks here are kept to a few attribute reads a tensor; dims are checked by
the library.  Tensors must be on the current device.
"""

from __future__ import annotations

import ctypes

import torch

from . import EINVAL, Dims, Layer, OasisError, last_error, lib

__all__ = ["tree_layout", "qk_norm_rope", "tree_workspace_bytes", "tree_attn", "verify_tree", "make_cache_layers",
           "commit_path"]

_BF16, _F32, _I32, _I64, _U64 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint64
_byref = ctypes.byref
_dev = -2                                # -2: not asked yet whether there is a device, -1: there is none


def _device():
    """Index of the current device, None without one (no tensor passes then)."""
    global _dev
    if _dev == -2:
        _dev = 0 if torch.cuda.is_available() else -1
        if _dev == 0:
            torch.cuda.init()
    return torch._C._cuda_getDevice() if _dev == 0 else None


def _stream_of(stream, dev):
    if stream is None:
        return None if dev is None else torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _bad(what, msg):
    return OasisError(EINVAL, what, msg)


def _why(x, what, name, dtype, numel, dev):
    """The error of an argument that _arg turned down."""
    if x is None:
        return _bad(what, f"{name} is None")
    if not isinstance(x, torch.Tensor):
        return _bad(what, f"{name} must be a tensor, got {type(x).__name__}")
    if x.dtype is not dtype:
        return _bad(what, f"{name} must be {str(dtype)[6:]}, got {x.dtype}")
    if not x.is_contiguous():
        return _bad(what, f"{name} must be contiguous")
    if x.numel() < numel:
        return _bad(what, f"{name} holds {x.numel()} elements, the call needs {numel}")
    if not x.is_cuda:
        return _bad(what, f"{name} must be on a CUDA device, got {x.device}")
    return _bad(what, f"{name} is on {x.device}, the current device is cuda:{dev}")


def _arg(x, what, name, dtype, numel, dev):
    """Address of a contiguous tensor of `numel` elements on the current device (raw addresses pass unchecked)."""
    try:
        if x.dtype is dtype and x.get_device() == dev and x.is_contiguous() and x.numel() >= numel:
            return x.data_ptr()
    except AttributeError:
        if x.__class__ is int:
            return x
    raise _why(x, what, name, dtype, numel, dev)


def _rows(x, what, name, dtype, rows, width, dev):
    """Address and row stride (elements) of a tensor whose leading dims are `rows` evenly spaced rows of >= width."""
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype or x.get_device() != dev:
        raise _why(x, what, name, dtype, 0, dev)
    shape, stride = x.shape, x.stride()
    if len(shape) == 3:                          # the usual case: [B, T, W], or a slice of a wider one along W
        b, t, n = shape
        if t > 1 and n >= width and b * t == rows and stride[2] == 1 and stride[0] == t * stride[1]:
            return x.data_ptr(), stride[1]
    if len(shape) < 2 or shape[-1] < width or x.numel() != rows * shape[-1]:
        raise _bad(what, f"{name} must be {rows} rows of at least {width} elements, got {tuple(shape)}")
    if shape[-1] > 1 and stride[-1] != 1:
        raise _bad(what, f"{name}'s rows must be contiguous")
    step = None
    span = 1
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n > 1:
            if step is None:
                step = s
            elif s != span * step:
                raise _bad(what, f"{name}'s rows must be evenly spaced")
            span *= n
    return x.data_ptr(), shape[-1] if step is None else step


def _failed(rc, what):
    return OasisError(rc, what, last_error())


def _check_tree(n_tree, what):
    if not 1 <= n_tree <= 64:
        raise _bad(what, f"n_tree must be in [1, 64] (got {n_tree})")


def _word_type(mask):
    """int64 words or uint64 ones (anything else is held against int64)."""
    return _U64 if getattr(mask, "dtype", None) is _U64 else _I64


def tree_layout(d: Dims, n_tree, parent, n_nodes, ctx_len, mask, pos, stream=None):
    """Visibility words (int64 or uint64 [B][T]) and positions (int32 [B][T]) from parents; n_nodes may be None."""
    w = "oasis_tree_layout"
    dev = _device()
    _check_tree(n_tree, w)
    b = d.batch
    n = b * n_tree
    rc = lib().oasis_tree_layout(
        _byref(d), n_tree, _arg(parent, w, "parent", _I32, n, dev),
        None if n_nodes is None else _arg(n_nodes, w, "n_nodes", _I32, b, dev), _arg(ctx_len, w, "ctx_len", _I32, b, dev),
        _arg(mask, w, "mask", _word_type(mask), n, dev), _arg(pos, w, "pos", _I32, n, dev), _stream_of(stream, dev))
    if rc:
        raise _failed(rc, w)


def qk_norm_rope(d: Dims, n_tok, qkv, wq, wk, eps, inv_freq, pos, q, k, v, stream=None):
    """qkv: bf16 [B, n_tok, >= (Hq + 2 Hkv) * 128], rows evenly spaced (a slice of a wider projection will do);
    wq / wk None: no norm.  q: [B, n_tok, Hq, 128], k and v: [B, Hkv, n_tok, 128], bf16."""
    w = "oasis_qk_norm_rope"
    dev = _device()
    if n_tok < 1:
        raise _bad(w, f"n_tok must be >= 1 (got {n_tok})")
    n, hq, hkv = d.batch * n_tok, d.n_q_heads, d.n_kv_heads
    at, step = _rows(qkv, w, "qkv", _BF16, n, (hq + 2 * hkv) * 128, dev)
    kv = n * hkv * 128
    rc = lib().oasis_qk_norm_rope(
        _byref(d), n_tok, at, step, None if wq is None else _arg(wq, w, "wq", _BF16, 128, dev),
        None if wk is None else _arg(wk, w, "wk", _BF16, 128, dev), eps, _arg(inv_freq, w, "inv_freq", _F32, 64, dev),
        _arg(pos, w, "pos", _I32, n, dev), _arg(q, w, "q", _BF16, n * hq * 128, dev), _arg(k, w, "k", _BF16, kv, dev),
        _arg(v, w, "v", _BF16, kv, dev), _stream_of(stream, dev))
    if rc:
        raise _failed(rc, w)


def tree_workspace_bytes(d: Dims, n_tree) -> int:
    return lib().oasis_tree_workspace_bytes(_byref(d), n_tree)


def tree_attn(d: Dims, n_tree, q, pool, slot_table, ctx_len, k_tree, v_tree, mask, scale, out, lse, ws, stream=None):
    """out: bf16 [B, T, Hq, 128], lse: fp32 [B, T, Hq]; ws: any tensor of tree_workspace_bytes(d, n_tree) bytes."""
    w = "oasis_tree_attn"
    dev = _device()
    _check_tree(n_tree, w)
    b, hq, hkv = d.batch, d.n_q_heads, d.n_kv_heads
    n = b * n_tree
    slots = b * hkv * d.budget_blocks
    kv = n * hkv * 128
    if not isinstance(ws, torch.Tensor):
        raise _bad(w, "ws must be a tensor (its size is taken from it)")
    rc = lib().oasis_tree_attn(
        _byref(d), n_tree, _arg(q, w, "q", _BF16, n * hq * 128, dev), _arg(pool, w, "pool", _BF16, slots * 4096, dev),
        _arg(slot_table, w, "slot_table", _I32, slots, dev), _arg(ctx_len, w, "ctx_len", _I32, b, dev),
        _arg(k_tree, w, "k_tree", _BF16, kv, dev), _arg(v_tree, w, "v_tree", _BF16, kv, dev), _arg(mask, w, "mask", _word_type(mask), n, dev), scale,
        _arg(out, w, "out", _BF16, n * hq * 128, dev), _arg(lse, w, "lse", _F32, n * hq, dev),
        _arg(ws, w, "ws", ws.dtype, 1, dev), ws.numel() * ws.element_size(), _stream_of(stream, dev))
    if rc:
        raise _failed(rc, w)


def verify_tree(d: Dims, n_tree, probs, draft_probs, tokens, parent, n_nodes, u_accept, u_sample, path, n_accept, next_token,
                stream=None):
    """probs, draft_probs: fp32 [B, T, vocab], rows evenly spaced and alike (a slice of padded rows will do);
    draft_probs None: the drafts were not drawn at random; n_nodes may be None."""
    w = "oasis_verify_tree"
    dev = _device()
    _check_tree(n_tree, w)
    b = d.batch
    n = b * n_tree
    at, step = _rows(probs, w, "probs", _F32, n, 1, dev)
    vocab = probs.shape[-1]
    draft = None
    if draft_probs is not None:
        draft, dstep = _rows(draft_probs, w, "draft_probs", _F32, n, 1, dev)
        if draft_probs.shape[-1] != vocab or dstep != step:
            raise _bad(w, "draft_probs must have the vocabulary and the row stride of probs")
    rc = lib().oasis_verify_tree(
        _byref(d), n_tree, vocab, at, draft, step, _arg(tokens, w, "tokens", _I32, n, dev), _arg(parent, w, "parent", _I32, n, dev),
        None if n_nodes is None else _arg(n_nodes, w, "n_nodes", _I32, b, dev), _arg(u_accept, w, "u_accept", _F32, n, dev),
        _arg(u_sample, w, "u_sample", _F32, b, dev), _arg(path, w, "path", _I32, n, dev), _arg(n_accept, w, "n_accept", _I32, b, dev),
        _arg(next_token, w, "next_token", _I32, b, dev), _stream_of(stream, dev))
    if rc:
        raise _failed(rc, w)


def _stack(x, what, name, dtype, layers, each, dev):
    """_arg for a tensor stacked over layers, `each` elements a layer without a gap (further layers are not used)."""
    if isinstance(x, torch.Tensor) and x.numel() > layers * each and x.numel() != x.shape[0] * each:
        raise _bad(what, f"{name} must hold {each} elements a layer, got {tuple(x.shape)}")
    return _arg(x, what, name, dtype, layers * each, dev)


def make_cache_layers(d: Dims, host_kv, kmin, kmax, slot_table, pool):
    """oasis_layer table for commit_path from tensors stacked over layers: host_kv [L, B, Hkv, N, 2, 16, 128] (pinned; None
    where no host copy is kept), kmin / kmax [L, B, Hkv, N, 128], slot_table [L, B, Hkv, K], pool [L, B, Hkv, K, 2, 16, 128]
    (slot_table and pool None: no pool).  The table keeps the tensors alive."""
    w = "make_cache_layers"
    rc = lib().oasis_check_dims(_byref(d))
    if rc:
        raise _failed(rc, w)
    dev = _device()
    if not isinstance(kmin, torch.Tensor) or kmin.dim() < 2:
        raise _bad(w, "kmin must be a tensor with a leading layer dim")
    L, units = kmin.shape[0], d.batch * d.n_kv_heads
    if L < 1:
        raise _bad(w, "no layers")
    N, K = d.max_blocks, d.budget_blocks
    at = {"kmin": (_stack(kmin, w, "kmin", _BF16, L, units * N * 128, dev), units * N * 256),
          "kmax": (_stack(kmax, w, "kmax", _BF16, L, units * N * 128, dev), units * N * 256)}
    if host_kv is not None:
        if host_kv.is_cuda:
            raise _bad(w, "host_kv must be pinned host memory")
        at["host_kv"] = (_stack(host_kv, w, "host_kv", _BF16, L, units * N * 4096, -1), units * N * 8192)
    if pool is not None:
        at["pool"] = (_stack(pool, w, "pool", _BF16, L, units * K * 4096, dev), units * K * 8192)
        at["slot_table"] = (_stack(slot_table, w, "slot_table", _I32, L, units * K, dev), units * K * 4)
    table = (Layer * L)(*(Layer(**{name: base + i * step for name, (base, step) in at.items()}) for i in range(L)))
    table._keep = (host_kv, kmin, kmax, slot_table, pool)
    return table


def commit_path(d: Dims, n_tree, layers, k_tree, v_tree, path, n_accept, ctx_len, ctx_len_out, stream=None):
    """The accepted nodes' rows into every layer's cache.  layers: make_cache_layers(...), or a list of ``Layer`` from
    make_layer; k_tree, v_tree: bf16 [L, B, Hkv, T, 128]; ctx_len_out may be None."""
    w = "oasis_commit_path"
    dev = _device()
    _check_tree(n_tree, w)
    b = d.batch
    n = b * n_tree
    if not isinstance(layers, ctypes.Array):
        layers = (Layer * len(layers))(*layers)
    elif layers._type_ is not Layer:
        raise _bad(w, "layers must be a table of Layer")
    L = len(layers)
    kv = L * n * d.n_kv_heads * 128
    rc = lib().oasis_commit_path(
        _byref(d), n_tree, layers, L, _arg(k_tree, w, "k_tree", _BF16, kv, dev), _arg(v_tree, w, "v_tree", _BF16, kv, dev),
        _arg(path, w, "path", _I32, n, dev), _arg(n_accept, w, "n_accept", _I32, b, dev), _arg(ctx_len, w, "ctx_len", _I32, b, dev),
        None if ctx_len_out is None else _arg(ctx_len_out, w, "ctx_len_out", _I32, b, dev), _stream_of(stream, dev))
    if rc:
        raise _failed(rc, w)
