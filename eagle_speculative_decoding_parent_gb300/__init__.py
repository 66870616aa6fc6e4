"""Python binding of libtreeverify (EAGLE draft-tree verification on GB300).

Argument marshalling only: every step runs in the library's CUDA kernels.
The functions carry the C entry points' names and take torch CUDA tensors
(PyTorch is used for device memory and streams).  Each call is asynchronous
on the current torch stream (or ``stream``) and raises ``TreeVerifyError``
when the library returns a host-side error; per-sequence data errors are
reported in the ``status`` tensors, as the C header describes.

There is no CPU fallback: importing this package fails if the compiled
library is missing (run ``__graft_entry__.build()`` or ``python -m
eagle_speculative_decoding_parent_gb300._build``).
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

__all__ = ["TV_OK", "TV_ERR_BAD_TREE", "TV_ERR_OUT_OF_RANGE", "TV_ERR_UNSUPPORTED",
           "TV_ERR_TIMEOUT", "TV_ERR_BAD_VALUES", "TV_F32", "TV_BF16", "GREEDY", "STOCHASTIC",
           "GREEDY_MASKED",
           "TreeVerifyError", "library_path", "status_string", "tree_mask_build",
           "tree_verify_attention_workspace", "tree_verify_attention_kernels", "tree_kv_append",
           "tree_verify_attention",
           "tree_verify_attention_noalloc", "tree_verify_attention_noalloc_capacity",
           "tree_accept_workspace",
           "tree_accept", "kv_compact", "draft_tree_workspace", "draft_tree_expand",
           "RopeTable", "rope_table", "chunk_kv_append", "chunk_attention_workspace",
           "chunk_attention", "chunk_kv_append_q8", "chunk_attention_q8_workspace",
           "chunk_attention_q8", "kv_compact_q8", "logits_sample",
           "token_counts_update", "tree_logits_process"]

(TV_OK, TV_ERR_INVALID_ARG, TV_ERR_BAD_TREE, TV_ERR_OUT_OF_RANGE, TV_ERR_UNSUPPORTED,
 TV_ERR_CUDA, TV_ERR_TIMEOUT, TV_ERR_BAD_VALUES, TV_ERR_WORKSPACE) = range(9)
TV_F32, TV_BF16 = 0, 1
GREEDY, STOCHASTIC, GREEDY_MASKED = 0, 1, 2


class TreeVerifyError(RuntimeError):
    pass


def library_path() -> str:
    return _build.LIB


if not os.path.exists(_build.LIB):
    raise ImportError(f"libtreeverify is not built ({_build.LIB} missing); "
                      "run python -m eagle_speculative_decoding_parent_gb300._build")

_lib = ctypes.CDLL(_build.LIB)

_i, _u64, _i64, _f, _p, _sz = (ctypes.c_int, ctypes.c_uint64, ctypes.c_int64, ctypes.c_float,
                               ctypes.c_void_p, ctypes.c_size_t)


def _sig(name, res, args):
    fn = getattr(_lib, name)
    fn.restype = res
    fn.argtypes = args
    return fn


_status_string = _sig("tv_status_string", ctypes.c_char_p, [_i])
_abi = _sig("tv_abi_version", _i, [])
_mask = _sig("tree_mask_build", _i, [_p, _i, _i, _p, _p, _p, _p, _p])
_attn_ws = _sig("tree_verify_attention_workspace", _sz, [_i, _i, _i, _i, _i, _i, _i, _i])
_attn_nk = _sig("tree_verify_attention_kernels", _i, [_i, _i, _i, _i, _i, _i, _i, _i, _sz])
_append = _sig("tree_kv_append", _i, [_p, _p, _p, _i, _i, _p, _i, _i, _f, _p, _p, _p, _i, _p, _i,
                                      _i, _i, _p, _p])
_attn = _sig("tree_verify_attention", _i,
             [_p, _p, _p, _p, _i, _p, _p, _i, _i, _p, _i, _i, _i, _i, _i, _i, _f, _p, _p, _p, _sz,
              _p])
_attn_na = _sig("tree_verify_attention_noalloc", _i,
                [_p, _p, _p, _p, _i, _p, _p, _i, _i, _p, _i, _i, _i, _i, _i, _i, _f, _p, _p, _p])
_attn_na_cap = _sig("tree_verify_attention_noalloc_capacity", _sz, [])
_acc_ws = _sig("tree_accept_workspace", _sz, [_i, _i, _i, _i])
_acc = _sig("tree_accept", _i,
            [_i, _p, _p, _p, _p, _i, _i, _p, _i, _u64, _u64, _p, _p, _p, _i, _p, _p, _sz, _p])
_compact = _sig("kv_compact", _i,
                [_p, _p, _i, _i64, _p, _i, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _p, _p, _p,
                 _p, _p])

_draft_ws = _sig("draft_tree_workspace", _sz, [_i, _i, _i])
_draft_expand = _sig("draft_tree_expand", _i, [_p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p, _p,
                                               _p, _p, _p, _sz, _p])

_rope_init = _sig("rope_table_init", _i, [_p, _i, _i, ctypes.c_double, _i] + [ctypes.c_double] * 5)
_chunk_append = _sig("chunk_kv_append", _i, [_p, _i64, _p, _i64, _p, _i64, _p, _i, _p, _p, _i, _i,
                                             _i, _i, _p, _p, _i64, _p, _p, _p, _i, _i, _i, _i, _p,
                                             _p])
_chunk_attn_ws = _sig("chunk_attention_workspace", _sz, [_i, _i, _i, _i, _i, _i])
_chunk_attn = _sig("chunk_attention", _i, [_p, _i64, _p, _p, _p, _i, _p, _p, _i, _i, _i, _i, _i,
                                           _i, _i, _i, _f, _f, _i, _p, _i64, _p, _p, _sz, _p])
_chunk_attn_q8_ws = _sig("chunk_attention_q8_workspace", _sz, [_i, _i, _i, _i, _i])
_chunk_attn_q8 = _sig("chunk_attention_q8", _i, [_p, _i64, _p, _p, _p, _p, _p, _i, _p, _p, _p, _i, _i, _i,
                                                 _i, _i, _i, _i, _f, _f, _i, _i, _p, _i64, _p, _p,
                                                 _sz, _p])
_chunk_append_q8 = _sig("chunk_kv_append_q8", _i, [_p, _i64, _p, _i64, _p, _i64, _p, _i, _p, _p, _i, _i,
                                                   _i, _i, _p, _p, _i64, _p, _p, _p, _p, _p, _i, _i,
                                                   _i, _p, _p])
_compact_q8 = _sig("kv_compact_q8", _i, [_p, _p, _p, _p, _i, _i64, _i64, _p, _i, _p, _p, _p, _i, _i, _i, _i,
                                         _i, _i, _p, _p, _p, _p, _p])
_sample = _sig("logits_sample", _i, [_p, _i, _i, _i, _i] + [_p] * 10)
_token_counts = _sig("token_counts_update", _i, [_p, _p, _p, _i, _i, _i, _i, _i, _p, _p])
_tree_logits = _sig("tree_logits_process", _i, [_p, _i, _i, _i, _i] + [_p] * 10 + [_i, _p, _p, _p])

assert _abi() == 2, "header / library ABI mismatch"


def status_string(code: int) -> str:
    return _status_string(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc != TV_OK:
        raise TreeVerifyError(f"{what}: {status_string(rc)} ({rc})")


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("tensors passed to libtreeverify must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libtreeverify must be contiguous")
    return t.data_ptr()


def _want(t, dtype, name, shape=None):
    """Checks a tensor's dtype (and shape) before its pointer reaches the
    library: the kernels index every buffer by the sizes passed beside it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _counts(node_counts, B):
    """Optional per-sequence node counts: int32 [B] on the device (the tree of
    sequence b is its first node_counts[b] node slots); None for full trees."""
    if node_counts is None:
        return None
    _want(node_counts, torch.int32, "node_counts", (B,))
    return _ptr(node_counts)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return TV_BF16
    if t.dtype == torch.float32:
        return TV_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def tree_mask_build(parents, mask, depth, status, stream=None, *, node_counts=None) -> None:
    """parents int32 [B,N] -> mask int64 (uint64 bits) [B,N], depth int32 [B,N] or None,
    status [B]; node_counts int32 [B] or None (trees of N nodes)."""
    _want(parents, torch.int32, "parents")
    if parents.dim() != 2:
        raise ValueError("parents is int32 [B, N]")
    B, N = parents.shape
    _want(mask, torch.int64, "mask", (B, N))
    if depth is not None:
        _want(depth, torch.int32, "depth", (B, N))
    _want(status, torch.int32, "status", (B,))
    _check(_mask(_ptr(parents), B, N, _counts(node_counts, B), _ptr(mask), _ptr(depth),
                 _ptr(status), _stream(stream)), "tree_mask_build")


def tree_verify_attention_workspace(B, N, Hq, Hkv, d, max_blocks_per_seq, block_size,
                                    dtype=torch.bfloat16) -> int:
    dt = TV_BF16 if dtype == torch.bfloat16 else TV_F32
    return int(_attn_ws(B, N, Hq, Hkv, d, max_blocks_per_seq, block_size, dt))


def tree_verify_attention_kernels(B, N, Hq, Hkv, d, max_blocks_per_seq, block_size,
                                  dtype=torch.bfloat16, workspace_bytes: int = 0) -> int:
    """Kernels one tree_verify_attention call launches (launch accounting)."""
    dt = TV_BF16 if dtype == torch.bfloat16 else TV_F32
    return int(_attn_nk(B, N, Hq, Hkv, d, max_blocks_per_seq, block_size, dt, workspace_bytes))


def _attention_args(q, k_cache, v_cache, block_table, prefix_lens, mask, out, status):
    """Shape and dtype checks shared by both attention entry points."""
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q is [B,N,Hq,d] and the caches [num_blocks,Hkv,block_size,d]")
    B, N, Hq, d = q.shape
    num_blocks, Hkv, bs, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("q and the caches disagree on the head size")
    dt = _dtype_code(q)
    _want(k_cache, q.dtype, "k_cache")
    _want(v_cache, q.dtype, "v_cache", k_cache.shape)
    _want(out, q.dtype, "out", q.shape)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table is int32 [B, max_blocks_per_seq]")
    _want(block_table, torch.int32, "block_table")
    _want(prefix_lens, torch.int32, "prefix_lens", (B,))
    _want(mask, torch.int64, "mask", (B, N))
    _want(status, torch.int32, "status", (B,))
    return B, N, Hq, Hkv, d, bs, num_blocks, dt


def tree_verify_attention(q, k_cache, v_cache, block_table, prefix_lens, mask, out, status,
                          workspace=None, *, scale: float = 0.0, stream=None,
                          node_counts=None) -> None:
    """q [B,N,Hq,d]; caches [num_blocks,Hkv,bs,d]; block_table int32 [B,max_blocks];
    prefix_lens int32 [B]; mask int64 [B,N]; out like q; status int32 [B];
    workspace uint8 tensor (zero-filled before first use); node_counts int32 [B]
    or None (rows of absent nodes are not written)."""
    B, N, Hq, Hkv, d, bs, num_blocks, dt = _attention_args(q, k_cache, v_cache, block_table,
                                                           prefix_lens, mask, out, status)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1],
                 _ptr(prefix_lens), _ptr(mask), B, N, _counts(node_counts, B), Hq, Hkv, d, bs,
                 num_blocks, dt, scale, _ptr(out), _ptr(status), _ptr(workspace), ws_bytes,
                 _stream(stream)), "tree_verify_attention")


def tree_verify_attention_noalloc_capacity() -> int:
    return int(_attn_na_cap())


def tree_verify_attention_noalloc(q, k_cache, v_cache, block_table, prefix_lens, mask, out,
                                  status, *, scale: float = 0.0, stream=None,
                                  node_counts=None) -> None:
    """tree_verify_attention for callers that cannot hand the library a
    workspace: the scratch is a fixed array inside the library, shared by
    every call on a device (overlapping calls race on it; the C header gives
    the size limit)."""
    B, N, Hq, Hkv, d, bs, num_blocks, dt = _attention_args(q, k_cache, v_cache, block_table,
                                                           prefix_lens, mask, out, status)
    _check(_attn_na(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                    block_table.shape[1], _ptr(prefix_lens), _ptr(mask), B, N,
                    _counts(node_counts, B), Hq, Hkv, d, bs, num_blocks, dt, scale, _ptr(out),
                    _ptr(status), _stream(stream)), "tree_verify_attention_noalloc")


def tree_accept_workspace(mode, B, N, V) -> int:
    return int(_acc_ws(mode, B, N, V))


def tree_accept(mode, parents, draft_tokens, target, draft_probs, accept_len, path, out_tokens,
                status, *, seed: int = 0, offset: int = 0, workspace=None, stream=None,
                node_counts=None) -> None:
    """Greedy (target = logits) or stochastic (target = p, draft_probs = q) acceptance;
    node_counts int32 [B] or None."""
    if target.dim() != 3:
        raise ValueError("target is float32 [B, N, V]")
    B, N, V = target.shape
    _want(target, torch.float32, "target")
    if draft_probs is not None:
        _want(draft_probs, torch.float32, "draft_probs", target.shape)
    _want(parents, torch.int32, "parents", (B, N))
    _want(draft_tokens, torch.int32, "draft_tokens", (B, N))
    if path.dim() != 2 or path.shape[0] != B:
        raise ValueError("path is int32 [B, max_path]")
    _want(path, torch.int32, "path")
    _want(out_tokens, torch.int32, "out_tokens", path.shape)
    _want(accept_len, torch.int32, "accept_len", (B,))
    _want(status, torch.int32, "status", (B,))
    if workspace is not None:
        _want(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_acc(mode, _ptr(parents), _ptr(draft_tokens), _ptr(target), _ptr(draft_probs), B, N,
                _counts(node_counts, B), V, seed, offset, _ptr(accept_len), _ptr(path),
                _ptr(out_tokens), path.shape[1], _ptr(status), _ptr(workspace), ws_bytes,
                _stream(stream)), "tree_accept")


def tree_kv_append(k_new, v_new, depth, k_cache, v_cache, block_table, prefix_lens, status, *,
                   rope_theta: float = 0.0, stream=None, node_counts=None) -> None:
    """k_new / v_new [B,N,Hkv,d]; caches [num_blocks,Hkv,bs,d]; depth int32 [B,N]
    (needed when rope_theta > 0); status int32 [B]; node_counts int32 [B] or None."""
    if k_new.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("k_new is [B,N,Hkv,d] and the caches [num_blocks,Hkv,block_size,d]")
    B, N, Hkv, d = k_new.shape
    num_blocks, Hkv2, bs, d2 = k_cache.shape
    if (Hkv2, d2) != (Hkv, d):
        raise ValueError("k_new and the caches disagree on Hkv or the head size")
    _dtype_code(k_cache)
    _want(k_new, k_cache.dtype, "k_new")
    _want(v_new, k_cache.dtype, "v_new", k_new.shape)
    _want(v_cache, k_cache.dtype, "v_cache", k_cache.shape)
    if depth is not None:
        _want(depth, torch.int32, "depth", (B, N))
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table is int32 [B, max_blocks_per_seq]")
    _want(block_table, torch.int32, "block_table")
    _want(prefix_lens, torch.int32, "prefix_lens", (B,))
    _want(status, torch.int32, "status", (B,))
    _check(_append(_ptr(k_new), _ptr(v_new), _ptr(depth), B, N, _counts(node_counts, B), Hkv, d,
                   float(rope_theta),
                   _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1],
                   _ptr(prefix_lens), bs, num_blocks, _dtype_code(k_cache), _ptr(status), _stream(stream)),
           "tree_kv_append")


def kv_compact(k_cache, v_cache, block_table, prefix_lens, path, accept_len, new_lens, status,
               *, src_slots=None, dst_slots=None, num_layers: int = 1, layer_stride: int = 0,
               stream=None) -> None:
    """Caches [num_layers*][num_blocks,Hkv,bs,d] (layers back to back, ``layer_stride``
    elements apart); path int32 [B,max_path]; accept_len int32 [B]."""
    num_blocks, Hkv, bs, d = k_cache.shape[-4:]
    if path.dim() != 2:
        raise ValueError("path is int32 [B, max_path]")
    B, max_path = path.shape
    _dtype_code(k_cache)
    _want(v_cache, k_cache.dtype, "v_cache", k_cache.shape)
    _want(path, torch.int32, "path")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table is int32 [B, max_blocks_per_seq]")
    _want(block_table, torch.int32, "block_table")
    for t, n in ((prefix_lens, "prefix_lens"), (accept_len, "accept_len"),
                 (new_lens, "new_lens"), (status, "status")):
        _want(t, torch.int32, n, (B,))
    for t, n in ((src_slots, "src_slots"), (dst_slots, "dst_slots")):
        if t is not None:
            _want(t, torch.int64, n, (B, max_path))
    if num_layers < 1 or (num_layers > 1 and
                          k_cache.numel() < (num_layers - 1) * layer_stride + num_blocks * Hkv * bs * d):
        raise ValueError("the caches hold fewer than num_layers layers at layer_stride")
    _check(_compact(_ptr(k_cache), _ptr(v_cache), num_layers, layer_stride, _ptr(block_table),
                    block_table.shape[1], _ptr(prefix_lens), _ptr(path), _ptr(accept_len),
                    max_path, B, Hkv, d, bs, num_blocks, _dtype_code(k_cache), _ptr(new_lens),
                    _ptr(src_slots), _ptr(dst_slots), _ptr(status), _stream(stream)),
           "kv_compact")


def draft_tree_workspace(B, topk, layers) -> int:
    return int(_draft_ws(B, topk, layers))


def draft_tree_expand(logits, layer, layers, status, workspace, *, topk, root_tokens=None,
                      N=1, front_tokens=None, front_src=None, parents=None, tokens=None,
                      scores=None, stream=None) -> None:
    """One draft-tree layer: logits float32 [B, F, V] (F = 1 at layer 0, else
    topk); root_tokens int32 [B] (layer 0); front_tokens / front_src int32
    [B, topk]; on the last layer parents / tokens int32 [B, N] and scores
    float32 [B, N]; workspace uint8 (zero-filled before the first call)."""
    _want(logits, torch.float32, "logits")
    if logits.dim() != 3:
        raise ValueError("logits is float32 [B, F, V]")
    B, F, V = logits.shape
    _want(status, torch.int32, "status", (B,))
    for t, n, shp in ((root_tokens, "root_tokens", (B,)), (front_tokens, "front_tokens", (B, topk)),
                      (front_src, "front_src", (B, topk)), (parents, "parents", (B, N)),
                      (tokens, "tokens", (B, N))):
        if t is not None:
            _want(t, torch.int32, n, shp)
    if scores is not None:
        _want(scores, torch.float32, "scores", (B, N))
    _want(workspace, torch.uint8, "workspace")
    if F != (1 if layer == 0 else topk):
        raise ValueError(f"layer {layer} takes {1 if layer == 0 else topk} rows per sequence")
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(_draft_expand(_ptr(logits), _ptr(root_tokens), B, V, topk, layer, layers, N, _ptr(front_tokens),
               _ptr(front_src), _ptr(parents), _ptr(tokens), _ptr(scores), _ptr(status),
               _ptr(workspace), ws_bytes, _stream(stream)), "draft_tree_expand")


# ---------------------------------------------------------------------------
# chunks of new tokens, and the logits of a tree

ROPE_SCALINGS = {"none": 0, "linear": 1, "bands": 2, "ramp": 3}


class RopeTable(ctypes.Structure):
    """Rotary frequencies (plain host data, see rope_table); dim columns are rotated."""
    _fields_ = [("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("amplitude", ctypes.c_float), ("amplitude_rest", ctypes.c_float),
                ("turn", ctypes.c_uint64 * 128)]


def rope_table(dim, *, theta: float = 10000.0, interleaved: bool = False, scaling: str = "none",
               factor: float = 1.0, original_len: float = 0.0, low: float = 0.0,
               high: float = 0.0, amplitude: float = 0.0) -> RopeTable:
    """The rotary positions of one model, made once: dim rotated columns of a head, pairs
    (j, j + dim/2) or, interleaved, (2j, 2j + 1); scaling "none", "linear", "bands" or "ramp"
    with its factor and original context length (formulas in the C header)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling is one of {sorted(ROPE_SCALINGS)}")
    t = RopeTable()
    _check(_rope_init(ctypes.addressof(t), dim, int(bool(interleaved)), float(theta),
                      ROPE_SCALINGS[scaling], float(factor), float(original_len), float(low),
                      float(high), float(amplitude)), "rope_table")
    return t


def _fault(t, dtype, name, shape, dev):
    """Raises what is wrong with a tensor that failed a check of _arg or _rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensors passed to libtreeverify must live on the current CUDA device")
    raise ValueError(f"{name}: tensors passed to libtreeverify must be contiguous")


def _arg(t, dtype, name, shape, dev):
    """Address of a contiguous tensor of this type and shape on device dev; None for None.
    (One call per tensor: the marshalling of a small call costs as much as its kernel.)"""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _fault(t, dtype, name, shape, dev)


def _rows(t, dtype, name, shape, dev):
    """Address and row stride, in elements, of [T, heads, d] with contiguous heads and rows any
    stride apart."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            if t.is_contiguous():
                return t.data_ptr(), shape[1] * shape[2]
            s = t.stride()
            if (s[2] == 1 or shape[2] == 1) and (s[1] == shape[2] or shape[1] == 1):
                return t.data_ptr(), (s[0] if shape[0] > 1 else shape[1] * shape[2])
            raise ValueError(f"{name}: the heads of a row must be contiguous")
    except AttributeError:
        pass
    _fault(t, dtype, name, shape, dev)


def _stream_of(stream, dev):
    """The raw-stream query instead of torch's Stream object: that costs more than the rest of a
    small call's marshalling."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _paged(k_cache, v_cache, block_table, q_start, prefix_lens, status, dtype, Hkv, d, dev):
    """Checks shared by the chunk calls; returns (B, block size, blocks) and the addresses in
    the order of the arguments."""
    ks, ts = k_cache.shape, block_table.shape
    if len(ks) != 4 or ks[1] != Hkv or ks[3] != d:
        raise ValueError("the caches are [num_blocks, Hkv, block_size, d]")
    B = status.shape[0] if status.dim() == 1 else -1
    if len(ts) != 2 or ts[0] != B:
        raise ValueError("block_table is int32 [B, max_blocks_per_seq], status int32 [B]")
    i32 = torch.int32
    return (B, ks[2], ks[0], _arg(k_cache, dtype, "k_cache", ks, dev),
            _arg(v_cache, dtype, "v_cache", ks, dev),
            _arg(block_table, i32, "block_table", ts, dev),
            _arg(q_start, i32, "q_start", (B + 1,), dev),
            _arg(prefix_lens, i32, "prefix_lens", (B,), dev),
            _arg(status, i32, "status", (B,), dev))


def chunk_kv_append(q, k, v, k_cache, v_cache, block_table, q_start, prefix_lens, status, *,
                    q_out=None, rope=None, positions=None, stream=None) -> None:
    """A ragged batch of new tokens into the paged cache: k / v [T,Hkv,d] and (or None) q
    [T,Hq,d], rows any stride apart; queries and keys rotated by ``rope`` (a RopeTable, or
    None); q_out [T,Hq,d] (default: q in place); positions int32 [T] or None (prefix + row);
    q_start int32 [B+1]; caches [num_blocks,Hkv,bs,d]; prefix_lens, status int32 [B]."""
    shape = k.shape
    if len(shape) != 3:
        raise ValueError("k is [T, Hkv, d]")
    T, Hkv, d = shape
    dtype = k.dtype
    dt = _dtype_code(k)
    dev = torch._C._cuda_getDevice()
    k_at, ks = _rows(k, dtype, "k", shape, dev)
    v_at, vs = _rows(v, dtype, "v", shape, dev)
    Hq, q_at, qs, q_out_at, qos = 1, None, 0, None, 0
    if q is not None:
        q_shape = q.shape
        if len(q_shape) != 3 or q_shape[0] != T or q_shape[2] != d:
            raise ValueError("q is [T, Hq, d]")
        Hq = q_shape[1]
        q_at, qs = _rows(q, dtype, "q", q_shape, dev)
        q_out_at, qos = (q_at, qs) if q_out is None else _rows(q_out, dtype, "q_out", q_shape, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    B, bs, blocks, kc, vc, table, start, prefix, st = _paged(
        k_cache, v_cache, block_table, q_start, prefix_lens, status, dtype, Hkv, d, dev)
    if rope is not None and not isinstance(rope, RopeTable):
        raise TypeError("rope: expected a RopeTable")
    _check(_chunk_append(q_at, qs, k_at, ks, v_at, vs,
                         _arg(positions, torch.int32, "positions", (T,), dev), T, start, prefix, B,
                         Hq, Hkv, d, None if rope is None else ctypes.addressof(rope), q_out_at,
                         qos, kc, vc, table, block_table.shape[1], bs, blocks, dt, st,
                         _stream_of(stream, dev)), "chunk_kv_append")


def chunk_attention_workspace(T, B, Hq, Hkv, d, dtype=torch.bfloat16) -> int:
    return int(_chunk_attn_ws(T, B, Hq, Hkv, d, TV_BF16 if dtype == torch.bfloat16 else TV_F32))


def chunk_attention(q, k_cache, v_cache, block_table, q_start, prefix_lens, out, status,
                    workspace=None, *, scale: float = 0.0, softcap: float = 0.0, window: int = 0,
                    stream=None) -> None:
    """Causal attention of a ragged batch of new tokens over the paged cache (prefix and the
    chunk itself): q / out [T,Hq,d], rows any stride apart; caches [num_blocks,Hkv,bs,d];
    q_start int32 [B+1]; prefix_lens, status int32 [B]; softcap > 0 caps the scores, window > 0
    limits the keys of a token to itself and the window - 1 before it; workspace uint8 of
    chunk_attention_workspace() bytes."""
    shape = q.shape
    if len(shape) != 3 or k_cache.dim() != 4:
        raise ValueError("q is [T, Hq, d] and the caches [num_blocks, Hkv, block_size, d]")
    T, Hq, d = shape
    Hkv = k_cache.shape[1]
    dtype = q.dtype
    dt = _dtype_code(q)
    dev = torch._C._cuda_getDevice()
    q_at, qs = _rows(q, dtype, "q", shape, dev)
    out_at, os_ = _rows(out, dtype, "out", shape, dev)
    B, bs, blocks, kc, vc, table, start, prefix, st = _paged(
        k_cache, v_cache, block_table, q_start, prefix_lens, status, dtype, Hkv, d, dev)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.nbytes
        ws = _arg(workspace, workspace.dtype, "workspace", workspace.shape, dev)
    if not 0 < window < 1 << 31:                # (the C argument has 32 bits)
        window = 0
    _check(_chunk_attn(q_at, qs, kc, vc, table, block_table.shape[1], start, prefix, T, B, Hq, Hkv,
                       d, bs, blocks, dt, scale, softcap, window, out_at, os_, st, ws, ws_bytes,
                       _stream_of(stream, dev)), "chunk_attention")


def _paged_q8(k_cache, v_cache, k_scale, v_scale, block_table, q_start, prefix_lens, status, Hkv,
              d, dev):
    """_paged for an 8-bit cache: e4m3 codes and their scales float32 [num_blocks, Hkv]."""
    paged = _paged(k_cache, v_cache, block_table, q_start, prefix_lens, status, torch.float8_e4m3fn,
                   Hkv, d, dev)
    shape = (paged[2], Hkv)
    return paged + (_arg(k_scale, torch.float32, "k_scale", shape, dev),
                    _arg(v_scale, torch.float32, "v_scale", shape, dev))


def chunk_kv_append_q8(q, k, v, k_cache, v_cache, k_scale, v_scale, block_table, q_start,
                       prefix_lens, status, *, q_out=None, rope=None, positions=None,
                       stream=None) -> None:
    """chunk_kv_append into an 8-bit cache: q, k, v, q_out bfloat16; caches float8_e4m3fn
    [num_blocks,Hkv,bs,d] with scales float32 [num_blocks,Hkv], powers of two that grow with
    what is appended to a block."""
    shape = k.shape
    if len(shape) != 3:
        raise ValueError("k is [T, Hkv, d]")
    T, Hkv, d = shape
    bf16 = torch.bfloat16
    dev = torch._C._cuda_getDevice()
    k_at, ks = _rows(k, bf16, "k", shape, dev)
    v_at, vs = _rows(v, bf16, "v", shape, dev)
    Hq, q_at, qs, q_out_at, qos = 1, None, 0, None, 0
    if q is not None:
        q_shape = q.shape
        if len(q_shape) != 3 or q_shape[0] != T or q_shape[2] != d:
            raise ValueError("q is [T, Hq, d]")
        Hq = q_shape[1]
        q_at, qs = _rows(q, bf16, "q", q_shape, dev)
        q_out_at, qos = (q_at, qs) if q_out is None else _rows(q_out, bf16, "q_out", q_shape, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    B, bs, blocks, kc, vc, table, start, prefix, st, ksc, vsc = _paged_q8(
        k_cache, v_cache, k_scale, v_scale, block_table, q_start, prefix_lens, status, Hkv, d, dev)
    if rope is not None and not isinstance(rope, RopeTable):
        raise TypeError("rope: expected a RopeTable")
    _check(_chunk_append_q8(q_at, qs, k_at, ks, v_at, vs,
                            _arg(positions, torch.int32, "positions", (T,), dev), T, start, prefix,
                            B, Hq, Hkv, d, None if rope is None else ctypes.addressof(rope),
                            q_out_at, qos, kc, vc, ksc, vsc, table, block_table.shape[1], bs,
                            blocks, st, _stream_of(stream, dev)), "chunk_kv_append_q8")


def chunk_attention_q8_workspace(T, B, Hq, Hkv, d) -> int:
    return int(_chunk_attn_q8_ws(T, B, Hq, Hkv, d))


def chunk_attention_q8(q, k_cache, v_cache, k_scale, v_scale, block_table, q_start, prefix_lens,
                       out, status, workspace=None, *, scale: float = 0.0, softcap: float = 0.0,
                       window: int = 0, sinks: int = 0, mask=None, stream=None) -> None:
    """chunk_attention over an 8-bit cache: q / out bfloat16 [T,Hq,d]; caches float8_e4m3fn
    [num_blocks,Hkv,bs,d] with scales float32 [num_blocks,Hkv]; window > 0 limits the keys of a
    token to itself, the window - 1 before it and the first ``sinks`` (at most 64) of its
    sequence; mask int64 [T] (rows of tree_mask_build's masks) makes a sequence's rows the nodes
    of a tree; workspace uint8 of chunk_attention_q8_workspace() bytes."""
    shape = q.shape
    if len(shape) != 3 or k_cache.dim() != 4:
        raise ValueError("q is [T, Hq, d] and the caches [num_blocks, Hkv, block_size, d]")
    T, Hq, d = shape
    Hkv = k_cache.shape[1]
    bf16 = torch.bfloat16
    dev = torch._C._cuda_getDevice()
    q_at, qs = _rows(q, bf16, "q", shape, dev)
    out_at, os_ = _rows(out, bf16, "out", shape, dev)
    B, bs, blocks, kc, vc, table, start, prefix, st, ksc, vsc = _paged_q8(
        k_cache, v_cache, k_scale, v_scale, block_table, q_start, prefix_lens, status, Hkv, d, dev)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.nbytes
        ws = _arg(workspace, workspace.dtype, "workspace", workspace.shape, dev)
    if not 0 < window < 1 << 31:                # (the C argument has 32 bits)
        window = 0
    if not 0 <= sinks <= 64:
        raise ValueError("sinks is 0 to 64")
    _check(_chunk_attn_q8(q_at, qs, kc, vc, ksc, vsc, table, block_table.shape[1], start, prefix,
                          _arg(mask, torch.int64, "mask", (T,), dev), T, B, Hq, Hkv, d, bs, blocks,
                          scale, softcap, window, sinks, out_at, os_, st, ws, ws_bytes,
                          _stream_of(stream, dev)), "chunk_attention_q8")


def kv_compact_q8(k_cache, v_cache, k_scale, v_scale, block_table, prefix_lens, path, accept_len,
                  new_lens, status, *, src_slots=None, dst_slots=None, stream=None) -> None:
    """kv_compact on 8-bit caches: float8_e4m3fn [num_blocks,Hkv,bs,d] with scales float32
    [num_blocks,Hkv], or both with the layers in front; path int32 [B,max_path]; accept_len,
    new_lens, status int32 [B]; src_slots, dst_slots int64 [B,max_path] or None."""
    shape, where = k_cache.shape, path.shape
    if len(shape) not in (4, 5):
        raise ValueError("the caches are [num_blocks, Hkv, block_size, d], or layers of them")
    if len(where) != 2:
        raise ValueError("path is int32 [B, max_path]")
    layers = shape[0] if len(shape) == 5 else 1
    num_blocks, Hkv, bs, d = shape[-4:]
    B, max_path = where
    ts = block_table.shape
    if len(ts) != 2 or ts[0] != B:
        raise ValueError("block_table is int32 [B, max_blocks_per_seq]")
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    dev = torch._C._cuda_getDevice()
    f8 = torch.float8_e4m3fn
    _check(_compact_q8(_arg(k_cache, f8, "k_cache", shape, dev), _arg(v_cache, f8, "v_cache", shape, dev),
                       _arg(k_scale, f32, "k_scale", shape[:-2], dev),
                       _arg(v_scale, f32, "v_scale", shape[:-2], dev), layers,
                       num_blocks * Hkv * bs * d, num_blocks * Hkv,
                       _arg(block_table, i32, "block_table", ts, dev), ts[1],
                       _arg(prefix_lens, i32, "prefix_lens", (B,), dev),
                       _arg(path, i32, "path", where, dev),
                       _arg(accept_len, i32, "accept_len", (B,), dev), max_path, B, Hkv, d, bs,
                       num_blocks, _arg(new_lens, i32, "new_lens", (B,), dev),
                       _arg(src_slots, i64, "src_slots", where, dev),
                       _arg(dst_slots, i64, "dst_slots", where, dev),
                       _arg(status, i32, "status", (B,), dev), _stream_of(stream, dev)),
           "kv_compact_q8")


def logits_sample(logits, uniform, tokens, status, *, temperature=None, top_k=None, top_p=None,
                  min_p=None, probs=None, node_counts=None, stream=None) -> None:
    """Samples rows of logits, float32 or bfloat16 [B,N,V], with the given uniform numbers float32
    [B,N] into tokens int32 [B,N], and writes the filtered distributions to probs float32
    [B,N,V] if given; temperature (0: the best entry), top_p, min_p float32 [B] and top_k int32
    [B], each optional; status int32 [B,N]."""
    shape = logits.shape
    if len(shape) != 3:
        raise ValueError("logits is [B, N, V]")
    B, N, V = shape
    dt = _dtype_code(logits)
    f32, i32 = torch.float32, torch.int32
    dev = torch._C._cuda_getDevice()
    _check(_sample(_arg(logits, logits.dtype, "logits", shape, dev), dt, B, N, V,
                   _arg(node_counts, i32, "node_counts", (B,), dev),
                   _arg(uniform, f32, "uniform", (B, N), dev),
                   _arg(temperature, f32, "temperature", (B,), dev),
                   _arg(top_k, i32, "top_k", (B,), dev), _arg(top_p, f32, "top_p", (B,), dev),
                   _arg(min_p, f32, "min_p", (B,), dev), _arg(tokens, i32, "tokens", (B, N), dev),
                   _arg(probs, f32, "probs", shape, dev), _arg(status, i32, "status", (B, N), dev),
                   _stream_of(stream, dev)), "logits_sample")


def token_counts_update(counts, tokens, status, *, starts=None, clear: bool = False,
                        prompt: bool = False, stream=None) -> None:
    """Token histories counts int32 [B,V] (bit 31: in the prompt; below: times emitted):
    tokens int32, [total] with starts int32 [B+1], or [B,W] without (-1 entries are skipped);
    clear zeroes the rows first; prompt marks instead of counting; status int32 [B]."""
    shape = counts.shape
    if len(shape) != 2:
        raise ValueError("counts is int32 [B, V]")
    B, V = shape
    i32 = torch.int32
    dev = torch._C._cuda_getDevice()
    words = tokens.shape
    if starts is None:
        if len(words) != 2 or words[0] != B:
            raise ValueError("tokens is int32 [B, W], or [total] with starts")
    elif len(words) != 1:
        raise ValueError("tokens is int32 [total] with starts")
    _check(_token_counts(_arg(counts, i32, "counts", shape, dev), _arg(tokens, i32, "tokens", words, dev),
                         _arg(starts, i32, "starts", (B + 1,), dev), tokens.numel(), B, V,
                         1 if clear else 0, 1 if prompt else 0,
                         _arg(status, i32, "status", (B,), dev), _stream_of(stream, dev)),
           "token_counts_update")


def tree_logits_process(logits, out, status, *, probs: bool, mask=None, draft_tokens=None,
                        counts=None, bias=None, grammar=None, repetition=None, frequency=None,
                        presence=None, temperature=None, node_counts=None, stream=None) -> None:
    """The target model's rows of a tree, logits float32 or bfloat16 [B,N,V], into what
    tree_accept reads, out float32 [B,N,V]: probabilities (probs) or logits, after bias
    [B,V], the penalties float32 [B] for tokens of the history (counts int32 [B,V]) and of
    each node's path (mask int64 [B,N], draft_tokens int32 [B,N]), the temperature float32 [B]
    and the grammar bits int32 [B,N,ceil(V/32)]; all of them optional; status int32 [B]."""
    shape = logits.shape
    if len(shape) != 3:
        raise ValueError("logits is [B, N, V]")
    B, N, V = shape
    dt = _dtype_code(logits)
    f32, i32 = torch.float32, torch.int32
    dev = torch._C._cuda_getDevice()
    _check(_tree_logits(_arg(logits, logits.dtype, "logits", shape, dev), dt, B, N, V,
                        _arg(node_counts, i32, "node_counts", (B,), dev),
                        _arg(mask, torch.int64, "mask", (B, N), dev),
                        _arg(draft_tokens, i32, "draft_tokens", (B, N), dev),
                        _arg(counts, i32, "counts", (B, V), dev),
                        _arg(bias, f32, "bias", (B, V), dev),
                        _arg(grammar, i32, "grammar", (B, N, (V + 31) // 32), dev),
                        _arg(repetition, f32, "repetition", (B,), dev),
                        _arg(frequency, f32, "frequency", (B,), dev),
                        _arg(presence, f32, "presence", (B,), dev),
                        _arg(temperature, f32, "temperature", (B,), dev), 1 if probs else 0,
                        _arg(out, f32, "out", shape, dev), _arg(status, i32, "status", (B,), dev),
                        _stream_of(stream, dev)), "tree_logits_process")
