"""Thin ctypes binding over libjf.so (declared in include/jf.h).

The functions named ``jf_*`` mirror the C entry points one to one: they take torch tensors
that already live on the GPU, check dtype/shape/contiguity, and pass raw pointers and the
current CUDA stream.  All computation happens in the library's kernels; there is no
fallback of any kind -- if libjf.so is missing or fails to load, importing this module
raises.  ``build_tree_mask``, ``tree_attention`` and ``tree_verify`` are conveniences that
also allocate the outputs (with torch) before calling the same entry points.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libjf.so")

JF_OK = 0
STATUS_NAMES = {0: "JF_OK", 1: "JF_ERR_INVALID_ARGUMENT", 2: "JF_ERR_INVALID_TREE",
                3: "JF_ERR_UNSUPPORTED", 4: "JF_ERR_WORKSPACE_TOO_SMALL", 5: "JF_ERR_CUDA",
                6: "JF_ERR_TIMEOUT", 7: "JF_ERR_MISALIGNED", 8: "JF_ERR_SCRATCH_CAPACITY"}
JF_DTYPE_BF16, JF_DTYPE_F32 = 0, 1
DEVERR_BAD_PARENT, DEVERR_BAD_PAGE, DEVERR_BAD_PREFIX = 0x1, 0x2, 0x4
DEVERR_BAD_TOKEN, DEVERR_TIMEOUT, DEVERR_BAD_PATH = 0x8, 0x10, 0x20
DEVERR_BAD_TREE_LEN, DEVERR_BAD_GROUP = 0x40, 0x80
MAX_NODES = 4096
PAGE_SIZE = 16
COUNT_PROMPT = 1 << 30
_Tensor, _bf16, _f32, _i32 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32


class JFError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m tree_speculative_decoding_jf_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    lib.jf_status_string.argtypes = [ctypes.c_int]
    lib.jf_status_string.restype = ctypes.c_char_p
    lib.jf_version.restype = ctypes.c_int
    lib.jf_build_tree_mask.argtypes = [P, P, i32, i32, P, P, P, P, P]
    lib.jf_build_tree_mask.restype = ctypes.c_int
    lib.jf_tree_attention_workspace_size.argtypes = [i32] * 7
    lib.jf_tree_attention_workspace_size.restype = sz
    lib.jf_tree_attention.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                                      f32, P, P, P, sz, P, P]
    lib.jf_tree_attention.restype = ctypes.c_int
    lib.jf_tree_verify_workspace_size.argtypes = [i32, i32, i32]
    lib.jf_tree_verify_workspace_size.restype = sz
    lib.jf_tree_verify.argtypes = [P, i32, P, P, i32, i32, i32, P, P, P, P, P, sz, P, P]
    lib.jf_tree_verify.restype = ctypes.c_int
    lib.jf_tree_verify_static.argtypes = [P, i32, P, P, i32, i32, i32, P, P, P, P, P, P]
    lib.jf_tree_verify_static.restype = ctypes.c_int
    lib.jf_compact_accepted_kv.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                           P, P, P]
    lib.jf_compact_accepted_kv.restype = ctypes.c_int
    lib.jf_build_draft_tree.argtypes = [P, i32, P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P]
    lib.jf_build_draft_tree_ragged.argtypes = [P, i32, P, P, i32, i32, i32, i32, i32, P, P, P, P,
                                               P, P, P, P]
    lib.jf_build_draft_tree_ragged.restype = ctypes.c_int
    lib.jf_build_draft_tree.restype = ctypes.c_int
    lib.jf_build_tree_mask_ragged.argtypes = [P, P, P, i32, i32, P, P, P, P, P]
    lib.jf_build_tree_mask_ragged.restype = ctypes.c_int
    lib.jf_tree_attention_ragged.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                             i32, i32, f32, P, P, P, sz, P, P]
    lib.jf_tree_attention_ragged.restype = ctypes.c_int
    lib.jf_tree_verify_ragged.argtypes = [P, i32, P, P, P, i32, i32, i32, P, P, P, P, P, sz, P, P]
    lib.jf_tree_verify_ragged.restype = ctypes.c_int
    lib.jf_debug_set_wait_limit_ns.argtypes = [ctypes.c_uint64, ctypes.c_int32]
    lib.jf_tree_verify_sampled.argtypes = [P, i32, P, P, P, P, f32, i32, i32, i32, P, P, P, P, sz,
                                           P, P]
    lib.jf_tree_verify_sampled.restype = ctypes.c_int
    lib.jf_debug_set_wait_limit_ns.restype = ctypes.c_int
    lib.jf_tree_verify_shard_chunks.argtypes = [i32, i32, i32]
    lib.jf_tree_verify_shard_chunks.restype = ctypes.c_int32
    lib.jf_tree_verify_shard_keys.argtypes = [P, i32, i32, i32, i32, i32, i32, P, P]
    lib.jf_tree_verify_shard_keys.restype = ctypes.c_int
    lib.jf_tree_verify_from_keys.argtypes = [P, i32, i32, P, P, i32, i32, i32, P, P, P, P, P, sz,
                                             P, P]
    lib.jf_tree_verify_from_keys.restype = ctypes.c_int
    lib.jf_build_tree_mask_packed.argtypes = [P, P, P, i32, i32, i32, P, P, P, P, P]
    lib.jf_build_tree_mask_packed.restype = ctypes.c_int
    lib.jf_tree_attention_packed.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                             i32, i32, i32, f32, P, P, P, sz, P, P]
    lib.jf_tree_attention_packed.restype = ctypes.c_int
    lib.jf_tree_verify_packed_workspace_size.argtypes = [i32, i32]
    lib.jf_tree_verify_packed_workspace_size.restype = sz
    lib.jf_tree_verify_packed.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, P, P, P, P, P, sz,
                                          P, P]
    lib.jf_tree_verify_packed.restype = ctypes.c_int
    lib.jf_tree_verify_sampled_ragged.argtypes = [P, i32, P, P, P, P, P, f32, i32, i32, i32, P, P,
                                                  P, P, sz, P, P]
    lib.jf_tree_verify_sampled_ragged.restype = ctypes.c_int
    lib.jf_tree_verify_sampled_packed.argtypes = [P, i32, P, P, P, P, P, f32, i32, i32, i32, i32,
                                                  P, P, P, P, sz, P, P]
    lib.jf_tree_verify_sampled_packed.restype = ctypes.c_int
    lib.jf_attention_weight.argtypes = [P, P, P, P, P, P, P, P] + [i32] * 8 + [f32, P, P, P]
    lib.jf_attention_weight.restype = ctypes.c_int
    lib.jf_attention_weight_packed.argtypes = [P] * 9 + [i32] * 9 + [f32, P, P, P]
    lib.jf_attention_weight_packed.restype = ctypes.c_int
    lib.jf_select_kept.argtypes = [P, P] + [i32] * 6 + [P, P, P, P]
    lib.jf_select_kept.restype = ctypes.c_int
    lib.jf_evict_kv.argtypes = [P, P, P, P, P, P, P, P, P] + [i32] * 7 + [P, P]
    lib.jf_evict_kv.restype = ctypes.c_int
    lib.jf_beam_select_workspace_size.argtypes = [i32] * 5
    lib.jf_beam_select_workspace_size.restype = sz
    lib.jf_beam_select.argtypes = [P, i32, P, P, i32, i32, i32, i32, i32, P, P, P, P, P, sz, P]
    lib.jf_beam_select.restype = ctypes.c_int
    lib.jf_beam_fork_kv.argtypes = [P, P, P, P, P, P] + [i32] * 8 + [P, P, P, P]
    lib.jf_beam_fork_kv.restype = ctypes.c_int
    i64 = ctypes.c_int64
    rotate = [P, i64, P, i64, P, i64, P, P, i32, i32, f32, P, P, f32, P, P, P]
    lib.jf_rotate_append_kv.argtypes = rotate + [i32] * 8 + [P, P, P, P, P]
    lib.jf_rotate_append_kv.restype = ctypes.c_int
    lib.jf_rotate_append_kv_packed.argtypes = rotate + [i32] * 9 + [P, P, P, P, P]
    lib.jf_rotate_append_kv_packed.restype = ctypes.c_int
    lib.jf_tree_attention_shared_workspace_size.argtypes = [i32] * 9
    lib.jf_tree_attention_shared_workspace_size.restype = sz
    lib.jf_tree_attention_shared.argtypes = [P] * 9 + [i32] * 9 + [f32, P, P, P, sz, P, P]
    lib.jf_tree_attention_shared.restype = ctypes.c_int
    lib.jf_tree_attention_shared_packed.argtypes = [P] * 9 + [i32] * 10 + [f32, P, P, P, sz, P, P]
    lib.jf_tree_attention_shared_packed.restype = ctypes.c_int
    adjust = [P, i32, P, P, P, P, P, P, i32, P, P, P, f32, P]
    lib.jf_adjust_logits.argtypes = adjust + [i32] * 3 + [P, i32, P, P]
    lib.jf_adjust_logits.restype = ctypes.c_int
    lib.jf_adjust_logits_packed.argtypes = adjust + [i32] * 4 + [P, i32, P, P]
    lib.jf_adjust_logits_packed.restype = ctypes.c_int
    lib.jf_count_tokens.argtypes = [P, P, i32, P, P, P, P, i32, i32, i32, i32, P, P, P]
    lib.jf_count_tokens.restype = ctypes.c_int
    return lib


_lib = _load()
SIZE_MAX = ctypes.c_size_t(-1).value


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check(fn: str, status: int):
    if status != JF_OK:
        raise JFError(fn, status)


def jf_status_string(status: int) -> str:
    return _lib.jf_status_string(status).decode()


def jf_version() -> int:
    return _lib.jf_version()


def jf_debug_set_wait_limit_ns(limit_ns: int, withhold_arrivals: bool = False) -> None:
    """Test hook: time limit of the attention kernels' pipeline waits on the current device,
    optionally with the data-arrival signals withheld so a wait can never complete
    ((0, False) restores normal operation).  See include/jf.h."""
    _check("jf_debug_set_wait_limit_ns",
           _lib.jf_debug_set_wait_limit_ns(int(limit_ns), 1 if withhold_arrivals else 0))


def jf_build_tree_mask(parent, prefix_len, mask, depth=None, pos=None, dev_err=None,
                       stream=None) -> None:
    _mask_call(parent, prefix_len, None, mask, depth, pos, dev_err, stream)


def jf_build_tree_mask_ragged(parent, prefix_len, tree_len, mask, depth=None, pos=None,
                              dev_err=None, stream=None) -> None:
    """Per-sequence tree sizes: nodes i >= tree_len[b] are padding (see include/jf.h)."""
    _need(tree_len, "tree_len", torch.int32, (parent.shape[0],))
    _mask_call(parent, prefix_len, tree_len, mask, depth, pos, dev_err, stream)


def _mask_call(parent, prefix_len, tree_len, mask, depth, pos, dev_err, stream) -> None:
    B, N = parent.shape
    W = (N + 63) // 64
    _need(parent, "parent", torch.int32)
    _need(prefix_len, "prefix_len", torch.int32, (B,))
    _need(mask, "mask", torch.int64, (B, N, W))
    for name, t in (("depth", depth), ("pos", pos)):
        if t is not None:
            _need(t, name, torch.int32, (B, N))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    if tree_len is None:
        _check("jf_build_tree_mask", _lib.jf_build_tree_mask(
            _ptr(parent), _ptr(prefix_len), B, N, _ptr(mask), _ptr(depth), _ptr(pos),
            _ptr(dev_err), _stream(stream)))
    else:
        _check("jf_build_tree_mask_ragged", _lib.jf_build_tree_mask_ragged(
            _ptr(parent), _ptr(prefix_len), _ptr(tree_len), B, N, _ptr(mask), _ptr(depth),
            _ptr(pos), _ptr(dev_err), _stream(stream)))


def jf_tree_attention_workspace_size(B, N, Hq, Hkv, D, max_pages, page_size=PAGE_SIZE) -> int:
    n = _lib.jf_tree_attention_workspace_size(B, N, Hq, Hkv, D, max_pages, page_size)
    if n == SIZE_MAX:
        raise JFError("jf_tree_attention_workspace_size", 3)
    return int(n)


def jf_tree_attention(q, k_cache, v_cache, block_table, prefix_len, mask, scale, out, lse=None,
                      workspace=None, dev_err=None, stream=None) -> None:
    _attention_call(q, k_cache, v_cache, block_table, prefix_len, None, mask, scale, out, lse,
                    workspace, dev_err, stream)


def jf_tree_attention_ragged(q, k_cache, v_cache, block_table, prefix_len, tree_len, mask,
                             scale, out, lse=None, workspace=None, dev_err=None,
                             stream=None) -> None:
    """Per-sequence tree sizes: sequence b's tree keys are P_b .. P_b + tree_len[b] - 1."""
    _need(tree_len, "tree_len", torch.int32, (q.shape[0],))
    _attention_call(q, k_cache, v_cache, block_table, prefix_len, tree_len, mask, scale, out,
                    lse, workspace, dev_err, stream)


def _attention_call(q, k_cache, v_cache, block_table, prefix_len, tree_len, mask, scale, out,
                    lse, workspace, dev_err, stream) -> None:
    B, N, Hq, D = q.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    max_pages = block_table.shape[1]
    W = (N + 63) // 64
    _need(q, "q", torch.bfloat16)
    _need(k_cache, "k_cache", torch.bfloat16)
    _need(v_cache, "v_cache", torch.bfloat16, k_cache.shape)
    _need(block_table, "block_table", torch.int32, (B, max_pages))
    _need(prefix_len, "prefix_len", torch.int32, (B,))
    _need(mask, "mask", torch.int64, (B, N, W))
    _need(out, "out", torch.bfloat16, (B, N, Hq, D))
    if D2 != D:
        raise ValueError("q and k_cache head dims differ")
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq, N))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    ws_bytes = 0
    if workspace is not None:
        if workspace.device.type != "cuda" or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    if tree_len is None:
        _check("jf_tree_attention", _lib.jf_tree_attention(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(prefix_len),
            _ptr(mask), B, N, Hq, Hkv, D, page, max_pages, num_pages, float(scale), _ptr(out),
            _ptr(lse), _ptr(workspace), ws_bytes, _ptr(dev_err), _stream(stream)))
    else:
        _check("jf_tree_attention_ragged", _lib.jf_tree_attention_ragged(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(prefix_len),
            _ptr(tree_len), _ptr(mask), B, N, Hq, Hkv, D, page, max_pages, num_pages,
            float(scale), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _ptr(dev_err),
            _stream(stream)))


def jf_tree_verify_workspace_size(B, N, V) -> int:
    n = _lib.jf_tree_verify_workspace_size(B, N, V)
    if n == SIZE_MAX:
        raise JFError("jf_tree_verify_workspace_size", 3)
    return int(n)


def jf_tree_verify(logits, draft, parent, accept_len, path, bonus, argmax=None, workspace=None,
                   dev_err=None, stream=None) -> None:
    _verify_call(logits, draft, parent, None, accept_len, path, bonus, argmax, workspace,
                 dev_err, stream)


def jf_tree_verify_ragged(logits, draft, parent, tree_len, accept_len, path, bonus, argmax=None,
                          workspace=None, dev_err=None, stream=None) -> None:
    """Per-sequence tree sizes: nodes i >= tree_len[b] are never accepted."""
    _need(tree_len, "tree_len", torch.int32, (logits.shape[0],))
    _verify_call(logits, draft, parent, tree_len, accept_len, path, bonus, argmax, workspace,
                 dev_err, stream)


def jf_tree_verify_sampled(logits, draft, parent, uniform, bonus_uniform, temperature,
                           accept_len, path, bonus, workspace, dev_err=None, stream=None) -> None:
    """Lossless (stochastic) verification; uniform float32 [B][N] and bonus_uniform float32
    [B] are the random numbers in [0, 1) (see include/jf.h).  The workspace is sized by
    jf_tree_verify_workspace_size."""
    B, N, V = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = JF_DTYPE_BF16
    elif logits.dtype == torch.float32:
        dt = JF_DTYPE_F32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    _need(logits, "logits", logits.dtype)
    _need(draft, "draft", torch.int32, (B, N))
    _need(parent, "parent", torch.int32, (B, N))
    _need(uniform, "uniform", torch.float32, (B, N))
    _need(bonus_uniform, "bonus_uniform", torch.float32, (B,))
    _need(accept_len, "accept_len", torch.int32, (B,))
    _need(path, "path", torch.int32, (B, N))
    _need(bonus, "bonus", torch.int32, (B,))
    _need(workspace, "workspace", torch.uint8)
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    _check("jf_tree_verify_sampled", _lib.jf_tree_verify_sampled(
        _ptr(logits), dt, _ptr(draft), _ptr(parent), _ptr(uniform), _ptr(bonus_uniform),
        float(temperature), B, N, V, _ptr(accept_len), _ptr(path), _ptr(bonus), _ptr(workspace),
        workspace.numel(), _ptr(dev_err), _stream(stream)))


def _verify_call(logits, draft, parent, tree_len, accept_len, path, bonus, argmax, workspace,
                 dev_err, stream) -> None:
    B, N, V = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = JF_DTYPE_BF16
    elif logits.dtype == torch.float32:
        dt = JF_DTYPE_F32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    _need(logits, "logits", logits.dtype)
    _need(draft, "draft", torch.int32, (B, N))
    _need(parent, "parent", torch.int32, (B, N))
    _need(accept_len, "accept_len", torch.int32, (B,))
    _need(path, "path", torch.int32, (B, N))
    _need(bonus, "bonus", torch.int32, (B,))
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, (B, N))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
    if tree_len is None:
        _check("jf_tree_verify", _lib.jf_tree_verify(
            _ptr(logits), dt, _ptr(draft), _ptr(parent), B, N, V, _ptr(argmax),
            _ptr(accept_len), _ptr(path), _ptr(bonus), _ptr(workspace), ws_bytes, _ptr(dev_err),
            _stream(stream)))
    else:
        _check("jf_tree_verify_ragged", _lib.jf_tree_verify_ragged(
            _ptr(logits), dt, _ptr(draft), _ptr(parent), _ptr(tree_len), B, N, V, _ptr(argmax),
            _ptr(accept_len), _ptr(path), _ptr(bonus), _ptr(workspace), ws_bytes, _ptr(dev_err),
            _stream(stream)))


def jf_tree_verify_static(logits, draft, parent, accept_len, path, bonus, argmax=None,
                          dev_err=None, stream=None) -> None:
    """jf_tree_verify without a workspace: the library's fixed scratch array is used
    (see include/jf.h for its capacity and the rules for concurrent calls)."""
    B, N, V = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = JF_DTYPE_BF16
    elif logits.dtype == torch.float32:
        dt = JF_DTYPE_F32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    _need(logits, "logits", logits.dtype)
    for name, t, shape in (("draft", draft, (B, N)), ("parent", parent, (B, N)),
                           ("accept_len", accept_len, (B,)), ("path", path, (B, N)),
                           ("bonus", bonus, (B,))):
        _need(t, name, torch.int32, shape)
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, (B, N))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    _check("jf_tree_verify_static", _lib.jf_tree_verify_static(
        _ptr(logits), dt, _ptr(draft), _ptr(parent), B, N, V, _ptr(argmax), _ptr(accept_len),
        _ptr(path), _ptr(bonus), _ptr(dev_err), _stream(stream)))


def jf_tree_verify_shard_chunks(B, N, V_shard) -> int:
    n = _lib.jf_tree_verify_shard_chunks(B, N, V_shard)
    if n < 0:
        raise JFError("jf_tree_verify_shard_chunks", 3)
    return int(n)


def jf_tree_verify_shard_keys(logits_shard, vocab_offset, keys, stream=None) -> None:
    """Argmax keys of one vocabulary range: logits_shard [B][N][V_shard] (bf16 or f32) holds
    the tokens vocab_offset .. vocab_offset + V_shard - 1; keys is int64 [B][N][chunks]
    (the uint64 keys' bits).  See include/jf.h."""
    B, N, Vs = logits_shard.shape
    if logits_shard.dtype == torch.bfloat16:
        dt = JF_DTYPE_BF16
    elif logits_shard.dtype == torch.float32:
        dt = JF_DTYPE_F32
    else:
        raise TypeError("logits_shard must be bfloat16 or float32")
    _need(logits_shard, "logits_shard", logits_shard.dtype)
    _need(keys, "keys", torch.int64)
    if keys.dim() != 3 or tuple(keys.shape[:2]) != (B, N):
        raise ValueError(f"keys has shape {tuple(keys.shape)}, expected ({B}, {N}, chunks)")
    _check("jf_tree_verify_shard_keys", _lib.jf_tree_verify_shard_keys(
        _ptr(logits_shard), dt, B, N, Vs, int(vocab_offset), keys.shape[2], _ptr(keys),
        _stream(stream)))


def jf_tree_verify_from_keys(keys, V, draft, parent, accept_len, path, bonus, workspace,
                             argmax=None, dev_err=None, stream=None) -> None:
    """The greedy walk on every range's keys, int64 [S][B][N][chunks] (an all-gather of
    jf_tree_verify_shard_keys' outputs); workspace uint8 of at least 8*B*N bytes."""
    S, B, N, chunks = keys.shape
    _need(keys, "keys", torch.int64)
    for name, t, shape in (("draft", draft, (B, N)), ("parent", parent, (B, N)),
                           ("accept_len", accept_len, (B,)), ("path", path, (B, N)),
                           ("bonus", bonus, (B,))):
        _need(t, name, torch.int32, shape)
    _need(workspace, "workspace", torch.uint8)
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, (B, N))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    _check("jf_tree_verify_from_keys", _lib.jf_tree_verify_from_keys(
        _ptr(keys), S, chunks, _ptr(draft), _ptr(parent), B, N, int(V), _ptr(argmax),
        _ptr(accept_len), _ptr(path), _ptr(bonus), _ptr(workspace), workspace.numel(),
        _ptr(dev_err), _stream(stream)))


def jf_build_tree_mask_packed(parent, prefix_len, cu_seqlens, N_max, mask, depth=None, pos=None,
                              dev_err=None, stream=None) -> None:
    """Packed trees: parent int32 [T] (ids within each sequence), cu_seqlens int32 [B + 1],
    mask int64 [T][ceil(N_max / 64)] (see include/jf.h)."""
    (T,) = parent.shape
    B = cu_seqlens.shape[0] - 1
    W = (N_max + 63) // 64
    _need(parent, "parent", torch.int32)
    _need(prefix_len, "prefix_len", torch.int32, (B,))
    _need(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,))
    _need(mask, "mask", torch.int64, (T, W))
    for name, t in (("depth", depth), ("pos", pos)):
        if t is not None:
            _need(t, name, torch.int32, (T,))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    _check("jf_build_tree_mask_packed", _lib.jf_build_tree_mask_packed(
        _ptr(parent), _ptr(prefix_len), _ptr(cu_seqlens), B, N_max, T, _ptr(mask), _ptr(depth),
        _ptr(pos), _ptr(dev_err), _stream(stream)))


def jf_tree_attention_packed(q, k_cache, v_cache, block_table, prefix_len, cu_seqlens, N_max,
                             mask, scale, out, lse=None, workspace=None, dev_err=None,
                             stream=None) -> None:
    """Packed trees: q and out bf16 [T][Hq][D], mask int64 [T][W], lse float32 [Hq][T];
    the workspace is sized by jf_tree_attention_workspace_size with N = N_max."""
    T, Hq, D = q.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    B = cu_seqlens.shape[0] - 1
    max_pages = block_table.shape[1]
    W = (N_max + 63) // 64
    _need(q, "q", torch.bfloat16)
    _need(k_cache, "k_cache", torch.bfloat16)
    _need(v_cache, "v_cache", torch.bfloat16, k_cache.shape)
    _need(block_table, "block_table", torch.int32, (B, max_pages))
    _need(prefix_len, "prefix_len", torch.int32, (B,))
    _need(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,))
    _need(mask, "mask", torch.int64, (T, W))
    _need(out, "out", torch.bfloat16, (T, Hq, D))
    if D2 != D:
        raise ValueError("q and k_cache head dims differ")
    if lse is not None:
        _need(lse, "lse", torch.float32, (Hq, T))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    ws_bytes = 0
    if workspace is not None:
        if workspace.device.type != "cuda" or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    _check("jf_tree_attention_packed", _lib.jf_tree_attention_packed(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(prefix_len),
        _ptr(cu_seqlens), _ptr(mask), B, N_max, T, Hq, Hkv, D, page, max_pages, num_pages,
        float(scale), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _ptr(dev_err),
        _stream(stream)))


def jf_tree_verify_packed_workspace_size(T, V) -> int:
    n = _lib.jf_tree_verify_packed_workspace_size(T, V)
    if n == SIZE_MAX:
        raise JFError("jf_tree_verify_packed_workspace_size", 3)
    return int(n)


def jf_tree_verify_packed(logits, draft, parent, cu_seqlens, N_max, accept_len, path, bonus,
                          argmax=None, workspace=None, dev_err=None, stream=None) -> None:
    """Packed trees: logits [T][V] (bf16 or f32), draft/parent/argmax int32 [T], path int32
    [B][N_max]; the workspace is sized by jf_tree_verify_packed_workspace_size(T, V)."""
    T, V = logits.shape
    B = cu_seqlens.shape[0] - 1
    if logits.dtype == torch.bfloat16:
        dt = JF_DTYPE_BF16
    elif logits.dtype == torch.float32:
        dt = JF_DTYPE_F32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    _need(logits, "logits", logits.dtype)
    for name, t, shape in (("draft", draft, (T,)), ("parent", parent, (T,)),
                           ("cu_seqlens", cu_seqlens, (B + 1,)), ("accept_len", accept_len, (B,)),
                           ("path", path, (B, N_max)), ("bonus", bonus, (B,))):
        _need(t, name, torch.int32, shape)
    if argmax is not None:
        _need(argmax, "argmax", torch.int32, (T,))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("jf_tree_verify_packed", _lib.jf_tree_verify_packed(
        _ptr(logits), dt, _ptr(draft), _ptr(parent), _ptr(cu_seqlens), B, N_max, T, V,
        _ptr(argmax), _ptr(accept_len), _ptr(path), _ptr(bonus), _ptr(workspace), ws_bytes,
        _ptr(dev_err), _stream(stream)))


def jf_tree_verify_sampled_ragged(logits, draft, parent, tree_len, uniform, bonus_uniform,
                                  temperature, accept_len, path, bonus, workspace, dev_err=None,
                                  stream=None) -> None:
    """Lossless verification with per-sequence tree sizes (padded [B][N] arrays, tree_len
    int32 [B]); the workspace is sized by jf_tree_verify_workspace_size."""
    B, N, V = logits.shape
    dt = _logit_dtype(logits)
    _need(logits, "logits", logits.dtype)
    for name, t, shape in (("draft", draft, (B, N)), ("parent", parent, (B, N)),
                           ("tree_len", tree_len, (B,)), ("accept_len", accept_len, (B,)),
                           ("path", path, (B, N)), ("bonus", bonus, (B,))):
        _need(t, name, torch.int32, shape)
    _need(uniform, "uniform", torch.float32, (B, N))
    _need(bonus_uniform, "bonus_uniform", torch.float32, (B,))
    _need(workspace, "workspace", torch.uint8)
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    _check("jf_tree_verify_sampled_ragged", _lib.jf_tree_verify_sampled_ragged(
        _ptr(logits), dt, _ptr(draft), _ptr(parent), _ptr(tree_len), _ptr(uniform),
        _ptr(bonus_uniform), float(temperature), B, N, V, _ptr(accept_len), _ptr(path),
        _ptr(bonus), _ptr(workspace), workspace.numel(), _ptr(dev_err), _stream(stream)))


def jf_tree_verify_sampled_packed(logits, draft, parent, cu_seqlens, N_max, uniform,
                                  bonus_uniform, temperature, accept_len, path, bonus, workspace,
                                  dev_err=None, stream=None) -> None:
    """Lossless verification of packed trees: logits [T][V], draft/parent int32 [T], uniform
    float32 [T], path int32 [B][N_max]; the workspace is sized by
    jf_tree_verify_packed_workspace_size(T, V)."""
    T, V = logits.shape
    B = cu_seqlens.shape[0] - 1
    dt = _logit_dtype(logits)
    _need(logits, "logits", logits.dtype)
    for name, t, shape in (("draft", draft, (T,)), ("parent", parent, (T,)),
                           ("cu_seqlens", cu_seqlens, (B + 1,)), ("accept_len", accept_len, (B,)),
                           ("path", path, (B, N_max)), ("bonus", bonus, (B,))):
        _need(t, name, torch.int32, shape)
    _need(uniform, "uniform", torch.float32, (T,))
    _need(bonus_uniform, "bonus_uniform", torch.float32, (B,))
    _need(workspace, "workspace", torch.uint8)
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    _check("jf_tree_verify_sampled_packed", _lib.jf_tree_verify_sampled_packed(
        _ptr(logits), dt, _ptr(draft), _ptr(parent), _ptr(cu_seqlens), _ptr(uniform),
        _ptr(bonus_uniform), float(temperature), B, N_max, T, V, _ptr(accept_len), _ptr(path),
        _ptr(bonus), _ptr(workspace), workspace.numel(), _ptr(dev_err), _stream(stream)))


def _logit_dtype(logits) -> int:
    if logits.dtype == torch.bfloat16:
        return JF_DTYPE_BF16
    if logits.dtype == torch.float32:
        return JF_DTYPE_F32
    raise TypeError("logits must be bfloat16 or float32")


def jf_compact_accepted_kv(k_cache, v_cache, block_table, prefix_len, path, accept_len,
                           new_prefix_len, dev_err=None, stream=None) -> None:
    """Moves the accepted path's K/V next to the prefix, in place (see include/jf.h)."""
    num_pages, page, Hkv, D = k_cache.shape
    B, N = path.shape
    _need(k_cache, "k_cache", torch.bfloat16)
    _need(v_cache, "v_cache", torch.bfloat16, tuple(k_cache.shape))
    _need(block_table, "block_table", torch.int32)
    for name, t, shape in (("prefix_len", prefix_len, (B,)), ("accept_len", accept_len, (B,)),
                           ("new_prefix_len", new_prefix_len, (B,))):
        _need(t, name, torch.int32, shape)
    _need(path, "path", torch.int32, (B, N))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    _check("jf_compact_accepted_kv", _lib.jf_compact_accepted_kv(
        _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(prefix_len), _ptr(path),
        _ptr(accept_len), B, N, Hkv, D, page, block_table.shape[1], num_pages,
        _ptr(new_prefix_len), _ptr(dev_err), _stream(stream)))


def jf_build_draft_tree(draft_logits, K, N, cand_token, cand_logp, parent, draft, depth,
                        root_token=None, score=None, stream=None) -> None:
    """Best-first draft tree from per-depth draft logits (see include/jf.h)."""
    B, Dmax, V = draft_logits.shape
    if draft_logits.dtype == torch.bfloat16:
        dt = JF_DTYPE_BF16
    elif draft_logits.dtype == torch.float32:
        dt = JF_DTYPE_F32
    else:
        raise TypeError("draft_logits must be bfloat16 or float32")
    _need(draft_logits, "draft_logits", draft_logits.dtype)
    _need(cand_token, "cand_token", torch.int32, (B, Dmax, K))
    _need(cand_logp, "cand_logp", torch.float32, (B, Dmax, K))
    for name, t in (("parent", parent), ("draft", draft), ("depth", depth)):
        _need(t, name, torch.int32, (B, N))
    if score is not None:
        _need(score, "score", torch.float32, (B, N))
    if root_token is not None:
        _need(root_token, "root_token", torch.int32, (B,))
    _check("jf_build_draft_tree", _lib.jf_build_draft_tree(
        _ptr(draft_logits), dt, _ptr(root_token), B, Dmax, V, K, N, _ptr(cand_token),
        _ptr(cand_logp), _ptr(parent), _ptr(draft), _ptr(depth), _ptr(score), _stream(stream)))


def jf_build_draft_tree_ragged(draft_logits, K, N, budget, cand_token, cand_logp, parent, draft,
                               depth, root_token=None, score=None, dev_err=None,
                               stream=None) -> None:
    """Best-first draft trees with a budget per sequence (budget int32 [B], clamped to
    [1, N]); entries past a sequence's budget are padding (see include/jf.h)."""
    B, Dmax, V = draft_logits.shape
    dt = _logit_dtype(draft_logits)
    _need(draft_logits, "draft_logits", draft_logits.dtype)
    _need(budget, "budget", torch.int32, (B,))
    _need(cand_token, "cand_token", torch.int32, (B, Dmax, K))
    _need(cand_logp, "cand_logp", torch.float32, (B, Dmax, K))
    for name, t in (("parent", parent), ("draft", draft), ("depth", depth)):
        _need(t, name, torch.int32, (B, N))
    if score is not None:
        _need(score, "score", torch.float32, (B, N))
    if root_token is not None:
        _need(root_token, "root_token", torch.int32, (B,))
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
    _check("jf_build_draft_tree_ragged", _lib.jf_build_draft_tree_ragged(
        _ptr(draft_logits), dt, _ptr(root_token), _ptr(budget), B, Dmax, V, K, N,
        _ptr(cand_token), _ptr(cand_logp), _ptr(parent), _ptr(draft), _ptr(depth), _ptr(score),
        _ptr(dev_err), _stream(stream)))


def _on_stream(specs, dev_err, stream) -> int:
    """Checks of the cache and beam calls, quick where all is well: (name, tensor, dtype,
    shape) of every tensor given, and one device, the current one, for all of them (an error
    says what _need says).  Returns the stream's handle."""
    cur = torch.cuda.current_device()
    for name, t, dtype, shape in specs:
        if t is None:
            continue
        if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == cur and
                t.is_contiguous() and (shape is None or t.shape == shape)):
            continue
        _need(t, name, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{cur}")
    if dev_err is not None:
        _need(dev_err, "dev_err", torch.int32, (1,))
        if dev_err.get_device() != cur:
            raise ValueError(f"dev_err is on {dev_err.device}, the current device is cuda:{cur}")
    if stream is None:        # the handle of torch.cuda.current_stream(), without the object
        return torch._C._cuda_getCurrentRawStream(cur)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _as_current(stream):
    """The context in which stream is the current one.  Calls that make tensors run in it:
    their memory's earlier users, a fill and the kernels then follow each other."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _pointers(specs, dev_err, stream) -> list:
    """_on_stream's checks for calls of many small arguments, with the addresses taken in the same
    round: those of the tensors (None where none is given), dev_err's and the stream's handle."""
    cur = torch._C._cuda_getDevice()
    out = []
    for name, t, dtype, shape in specs:
        if t is None:
            out.append(None)
        elif (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == cur and t.is_contiguous() and
              (shape is None or t.shape == shape)):
            out.append(t.data_ptr())
        else:
            _need(t, name, dtype, shape)
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{cur}")
    if dev_err is None and stream is None:
        out += (None, torch._C._cuda_getCurrentRawStream(cur))
    else:
        on = _on_stream((), dev_err, stream)
        out += (_at(dev_err), on)
    return out


def _at(t):
    """Address of an optional tensor for a call whose arguments are declared as pointers."""
    return None if t is None else t.data_ptr()


def jf_attention_weight(q, k_cache, block_table, prefix_len, lse, weight_out, scale, path=None,
                        accept_len=None, weight=None, dev_err=None, stream=None) -> None:
    """Adds the attention probabilities that every cached key received (see include/jf.h)."""
    B, N, Hq, D = q.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    max_pages = block_table.shape[1]
    if D2 != D:
        raise ValueError("q and k_cache head dims differ")
    wshape = (B, Hkv, max_pages * page)
    on = _on_stream((("q", q, torch.bfloat16, None), ("k_cache", k_cache, torch.bfloat16, None),
                     ("block_table", block_table, torch.int32, (B, max_pages)),
                     ("prefix_len", prefix_len, torch.int32, (B,)),
                     ("lse", lse, torch.float32, (B, Hq, N)), ("path", path, torch.int32, (B, N)),
                     ("accept_len", accept_len, torch.int32, (B,)),
                     ("weight", weight, torch.float32, wshape),
                     ("weight_out", weight_out, torch.float32, wshape)), dev_err, stream)
    _check("jf_attention_weight", _lib.jf_attention_weight(
        _at(q), _at(k_cache), _at(block_table), _at(prefix_len), _at(path), _at(accept_len),
        _at(lse), _at(weight), B, N, Hq, Hkv, D, page, max_pages, num_pages, float(scale),
        _at(weight_out), _at(dev_err), on))


def jf_attention_weight_packed(q, k_cache, block_table, prefix_len, cu_seqlens, lse, weight_out,
                               scale, N_max, path=None, accept_len=None, weight=None,
                               dev_err=None, stream=None) -> None:
    """jf_attention_weight on packed rows: q [T][Hq][D], lse [Hq][T], path [B][N_max]."""
    T, Hq, D = q.shape
    B, max_pages = block_table.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    if D2 != D:
        raise ValueError("q and k_cache head dims differ")
    wshape = (B, Hkv, max_pages * page)
    on = _on_stream((("q", q, torch.bfloat16, None), ("k_cache", k_cache, torch.bfloat16, None),
                     ("block_table", block_table, torch.int32, None),
                     ("prefix_len", prefix_len, torch.int32, (B,)),
                     ("cu_seqlens", cu_seqlens, torch.int32, (B + 1,)),
                     ("lse", lse, torch.float32, (Hq, T)), ("path", path, torch.int32, (B, N_max)),
                     ("accept_len", accept_len, torch.int32, (B,)),
                     ("weight", weight, torch.float32, wshape),
                     ("weight_out", weight_out, torch.float32, wshape)), dev_err, stream)
    _check("jf_attention_weight_packed", _lib.jf_attention_weight_packed(
        _at(q), _at(k_cache), _at(block_table), _at(prefix_len), _at(cu_seqlens), _at(path),
        _at(accept_len), _at(lse), _at(weight), B, N_max, T, Hq, Hkv, D, page, max_pages,
        num_pages, float(scale), _at(weight_out), _at(dev_err), on))


def jf_select_kept(weight, seq_len, keep, kept_len, sink=0, recent=0, dev_err=None,
                   stream=None) -> None:
    """The positions a cache of keep.shape[-1] keys keeps (see include/jf.h)."""
    B, Hkv, capacity = weight.shape
    budget = keep.shape[-1]
    on = _on_stream((("weight", weight, torch.float32, None),
                     ("seq_len", seq_len, torch.int32, (B,)),
                     ("keep", keep, torch.int32, (B, Hkv, budget)),
                     ("kept_len", kept_len, torch.int32, (B,))), dev_err, stream)
    _check("jf_select_kept", _lib.jf_select_kept(
        _at(weight), _at(seq_len), B, Hkv, capacity, int(sink), int(recent), budget, _at(keep),
        _at(kept_len), _at(dev_err), on))


def jf_evict_kv(k_cache, v_cache, block_table, seq_len, keep, kept_len, new_block_table=None,
                weight=None, weight_out=None, dev_err=None, stream=None) -> None:
    """Moves the kept rows to the front of the cache (see include/jf.h)."""
    num_pages, page, Hkv, D = k_cache.shape
    B, max_pages = block_table.shape
    budget = keep.shape[-1]
    wshape = (B, Hkv, max_pages * page)
    on = _on_stream((("k_cache", k_cache, torch.bfloat16, None),
                     ("v_cache", v_cache, torch.bfloat16, k_cache.shape),
                     ("block_table", block_table, torch.int32, None),
                     ("seq_len", seq_len, torch.int32, (B,)),
                     ("keep", keep, torch.int32, (B, Hkv, budget)),
                     ("kept_len", kept_len, torch.int32, (B,)),
                     ("new_block_table", new_block_table, torch.int32, (B, max_pages)),
                     ("weight", weight, torch.float32, wshape),
                     ("weight_out", weight_out, torch.float32, wshape)), dev_err, stream)
    _check("jf_evict_kv", _lib.jf_evict_kv(
        _at(k_cache), _at(v_cache), _at(block_table), _at(seq_len), _at(keep), _at(kept_len),
        _at(new_block_table), _at(weight), _at(weight_out), B, Hkv, D, budget, page, max_pages,
        num_pages, _at(dev_err), on))


def jf_beam_select_workspace_size(B, W, V, K, dtype) -> int:
    n = _lib.jf_beam_select_workspace_size(B, W, V, K, dtype)
    if n == SIZE_MAX:
        raise JFError("jf_beam_select_workspace_size", 3)
    return int(n)


def jf_beam_select(logits, score, parent, token, new_score, workspace, finished=None,
                   eos_token=-1, new_finished=None, stream=None) -> None:
    """The best (beam, token) pairs of every prompt (see include/jf.h)."""
    B, W, V = logits.shape
    K = parent.shape[-1]
    dt = _logit_dtype(logits)
    on = _on_stream((("logits", logits, logits.dtype, None),
                     ("score", score, torch.float32, (B, W)),
                     ("finished", finished, torch.int32, (B, W)),
                     ("parent", parent, torch.int32, (B, K)), ("token", token, torch.int32, (B, K)),
                     ("new_score", new_score, torch.float32, (B, K)),
                     ("new_finished", new_finished, torch.int32, (B, K)),
                     ("workspace", workspace, torch.uint8, None)), None, stream)
    _check("jf_beam_select", _lib.jf_beam_select(
        _at(logits), dt, _at(score), _at(finished), int(eos_token), B, W, V, K, _at(parent),
        _at(token), _at(new_score), _at(new_finished), _at(workspace), workspace.numel(),
        on))


def jf_beam_fork_kv(k_cache, v_cache, block_table, prefix_len, parent, fresh_page,
                    new_block_table, new_prefix_len, dev_err=None, stream=None) -> None:
    """Block tables of the new beams, with their partial pages copied (see include/jf.h)."""
    num_pages, page, Hkv, D = k_cache.shape
    rows, max_pages = block_table.shape
    B, K = parent.shape
    if B < 1 or rows % B != 0:
        raise ValueError(f"block_table has {rows} rows, not a multiple of {B} prompts")
    W = rows // B
    on = _on_stream((("k_cache", k_cache, torch.bfloat16, None),
                     ("v_cache", v_cache, torch.bfloat16, k_cache.shape),
                     ("block_table", block_table, torch.int32, None),
                     ("prefix_len", prefix_len, torch.int32, (B * W,)),
                     ("parent", parent, torch.int32, (B, K)),
                     ("fresh_page", fresh_page, torch.int32, (B, K)),
                     ("new_block_table", new_block_table, torch.int32, (B * K, max_pages)),
                     ("new_prefix_len", new_prefix_len, torch.int32, (B * K,))), dev_err, stream)
    _check("jf_beam_fork_kv", _lib.jf_beam_fork_kv(
        _at(k_cache), _at(v_cache), _at(block_table), _at(prefix_len), _at(parent),
        _at(fresh_page), B, W, K, Hkv, D, page, max_pages, num_pages, _at(new_block_table),
        _at(new_prefix_len), _at(dev_err), on))


def _token_rows(name, t, lead) -> int:
    """Elements between consecutive tokens of a bf16 [..., H, D] tensor whose heads are
    contiguous and whose token rows lie evenly apart (a slice of a projection's output)."""
    H, D = t.shape[-2:]
    strides = t.stride()
    if D > 1 and strides[-1] != 1 or H > 1 and strides[-2] != D:
        raise ValueError(f"{name} must have contiguous heads")
    if len(lead) == 1:
        return strides[0] if lead[0] > 1 else H * D
    B, N = lead
    if N == 1:
        return strides[0] if B > 1 else H * D
    if B > 1 and strides[0] != N * strides[1]:
        raise ValueError(f"the token rows of {name} must lie evenly apart")
    return strides[1]


def _heads(name, t, lead, H, D, cur) -> int:
    """Checks one of q, k and v, quickly where all is well; the elements between its tokens."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.get_device() == cur and t.shape == lead + (H, D):
        s = t.stride()
        if s[-1] == 1 and s[-2] == D:
            if len(s) == 3:
                if lead[0] > 1:
                    return s[0]
            elif lead[1] > 1 and (lead[0] == 1 or s[0] == lead[1] * s[1]):
                return s[1]
        return _token_rows(name, t, lead)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != lead + (H, D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {lead + (H, D)}")
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{cur}")


def _rotate_call(q, k, v, k_cache, v_cache, block_table, prefix_len, lead, q_out, pos, freq, interleaved,
                 rotary_scale, q_norm, k_norm, norm_eps, tree_len, cu_seqlens, N_max, dev_err, stream):
    num_pages, page, Hkv, D = k_cache.shape
    B, max_pages = block_table.shape
    cur = torch._C._cuda_getDevice()
    k_stride = _heads("k", k, lead, Hkv, D, cur)
    v_stride = _heads("v", v, lead, Hkv, D, cur)
    Hq = q_stride = R = 0
    q_at = None
    if q is not None:
        Hq = q.shape[-2]
        q_stride = _heads("q", q, lead, Hq, D, cur)
        q_at = q.data_ptr()
    if freq is not None:
        R = 2 * freq.numel()
    batch = (B,)
    (k_to, v_to, table, lens, pos_at, freq_at, qn, kn, out, tl, cu, err, on) = _pointers(
        (("k_cache", k_cache, _bf16, None), ("v_cache", v_cache, _bf16, k_cache.shape),
         ("block_table", block_table, _i32, None), ("prefix_len", prefix_len, _i32, batch),
         ("pos", pos, _i32, lead), ("freq", freq, torch.float64, None if freq is None else (R // 2,)),
         ("q_norm", q_norm, _bf16, (D,)), ("k_norm", k_norm, _bf16, (D,)),
         ("q_out", q_out, _bf16, None if q_out is None else lead + (Hq, D)), ("tree_len", tree_len, _i32, batch),
         ("cu_seqlens", cu_seqlens, _i32, None if cu_seqlens is None else (B + 1,))), dev_err, stream)
    if cu is None:
        status = _lib.jf_rotate_append_kv(
            q_at, q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride, pos_at, freq_at, R, 1 if interleaved else 0,
            rotary_scale, qn, kn, norm_eps, table, lens, tl, B, lead[1], Hq, Hkv, D, page, max_pages, num_pages, out, k_to,
            v_to, err, on)
        if status:
            _check("jf_rotate_append_kv", status)
    else:
        _check("jf_rotate_append_kv_packed", _lib.jf_rotate_append_kv_packed(
            q_at, q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride, pos_at, freq_at, R, 1 if interleaved else 0,
            rotary_scale, qn, kn, norm_eps, table, lens, cu, B, N_max, lead[0], Hq, Hkv, D, page, max_pages, num_pages,
            out, k_to, v_to, err, on))


def jf_rotate_append_kv(q, k, v, k_cache, v_cache, block_table, prefix_len, q_out, pos=None, freq=None,
                        interleaved=False, rotary_scale=1.0, q_norm=None, k_norm=None, norm_eps=1e-6,
                        tree_len=None, dev_err=None, stream=None) -> None:
    """Rotates a step's queries [B][N][Hq][D] and keys [B][N][Hkv][D] and appends its keys and
    values to the paged cache (see include/jf.h).  q, k and v may be slices of one projection's
    output; q and q_out may be None."""
    B = block_table.shape[0]
    if k.dim() != 4 or k.shape[0] != B:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected ({B}, N, Hkv, D)")
    _rotate_call(q, k, v, k_cache, v_cache, block_table, prefix_len, k.shape[:2], q_out, pos, freq,
                 interleaved, rotary_scale, q_norm, k_norm, norm_eps, tree_len, None, None, dev_err, stream)


def jf_rotate_append_kv_packed(q, k, v, k_cache, v_cache, block_table, prefix_len, cu_seqlens, N_max, q_out,
                               pos=None, freq=None, interleaved=False, rotary_scale=1.0, q_norm=None,
                               k_norm=None, norm_eps=1e-6, dev_err=None, stream=None) -> None:
    """jf_rotate_append_kv on packed rows: q [T][Hq][D], k and v [T][Hkv][D], pos [T]."""
    if k.dim() != 3:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected (T, Hkv, D)")
    _rotate_call(q, k, v, k_cache, v_cache, block_table, prefix_len, k.shape[:1], q_out, pos, freq,
                 interleaved, rotary_scale, q_norm, k_norm, norm_eps, None, cu_seqlens, int(N_max), dev_err, stream)


def jf_tree_attention_shared_workspace_size(B, N, n_groups, Hq, Hkv, D, max_pages, T=0, page_size=PAGE_SIZE) -> int:
    """T: the rows of a packed call, 0 for a padded one."""
    n = _lib.jf_tree_attention_shared_workspace_size(B, N, T, n_groups, Hq, Hkv, D, max_pages, page_size)
    if n == SIZE_MAX:
        raise JFError("jf_tree_attention_shared_workspace_size", 3)
    return int(n)


@functools.lru_cache(maxsize=512)
def _shared_workspace(device, *sizes) -> int:
    """A workspace's bytes: they follow from the sizes and the current device alone."""
    return jf_tree_attention_shared_workspace_size(*sizes)


def jf_tree_attention_shared(q, k_cache, v_cache, block_table, prefix_len, mask, group_start, shared_pages, scale,
                             out, workspace, lse=None, tree_len=None, dev_err=None, stream=None) -> None:
    """jf_tree_attention with each group's shared prefix read once (see include/jf.h)."""
    B, N, Hq, D = q.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    max_pages = block_table.shape[1]
    n_groups = shared_pages.shape[0]
    if D2 != D:
        raise ValueError("q and k_cache head dims differ")
    (q_at, k_at, v_at, table, lens, tl, bits, starts, shared, o_at, l_at, ws, err, on) = _pointers(
        (("q", q, _bf16, None), ("k_cache", k_cache, _bf16, None), ("v_cache", v_cache, _bf16, k_cache.shape),
         ("block_table", block_table, _i32, (B, max_pages)), ("prefix_len", prefix_len, _i32, (B,)),
         ("tree_len", tree_len, _i32, (B,)), ("mask", mask, torch.int64, (B, N, (N + 63) // 64)),
         ("group_start", group_start, _i32, (n_groups + 1,)), ("shared_pages", shared_pages, _i32, None),
         ("out", out, _bf16, q.shape), ("lse", lse, _f32, (B, Hq, N)), ("workspace", workspace, torch.uint8, None)),
        dev_err, stream)
    _check("jf_tree_attention_shared", _lib.jf_tree_attention_shared(
        q_at, k_at, v_at, table, lens, tl, bits, starts, shared, n_groups, B, N, Hq, Hkv, D, page, max_pages, num_pages,
        scale, o_at, l_at, ws, workspace.numel(), err, on))


def jf_tree_attention_shared_packed(q, k_cache, v_cache, block_table, prefix_len, cu_seqlens, N_max, mask,
                                    group_start, shared_pages, scale, out, workspace, lse=None, dev_err=None,
                                    stream=None) -> None:
    """jf_tree_attention_shared on packed rows: q and out [T][Hq][D], mask [T][W], lse [Hq][T]."""
    T, Hq, D = q.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    B, max_pages = block_table.shape
    n_groups = shared_pages.shape[0]
    if D2 != D:
        raise ValueError("q and k_cache head dims differ")
    (q_at, k_at, v_at, table, lens, cu, bits, starts, shared, o_at, l_at, ws, err, on) = _pointers(
        (("q", q, _bf16, None), ("k_cache", k_cache, _bf16, None), ("v_cache", v_cache, _bf16, k_cache.shape),
         ("block_table", block_table, _i32, None), ("prefix_len", prefix_len, _i32, (B,)),
         ("cu_seqlens", cu_seqlens, _i32, (B + 1,)), ("mask", mask, torch.int64, (T, (N_max + 63) // 64)),
         ("group_start", group_start, _i32, (n_groups + 1,)), ("shared_pages", shared_pages, _i32, None),
         ("out", out, _bf16, q.shape), ("lse", lse, _f32, (Hq, T)), ("workspace", workspace, torch.uint8, None)),
        dev_err, stream)
    _check("jf_tree_attention_shared_packed", _lib.jf_tree_attention_shared_packed(
        q_at, k_at, v_at, table, lens, cu, bits, starts, shared, n_groups, B, N_max, T, Hq, Hkv, D, page, max_pages,
        num_pages, scale, o_at, l_at, ws, workspace.numel(), err, on))


def jf_adjust_logits(logits, out, count=None, draft=None, mask=None, bias=None, allowed=None, allowed_row=None,
                     repetition=None, presence=None, frequency=None, masked=float("-inf"), tree_len=None,
                     dev_err=None, stream=None) -> None:
    """Penalties, biases and grammar masks on logits [B][N][V] (see include/jf.h); out has their
    type or float32 and may be logits."""
    B, N, V = logits.shape
    _adjust_call(logits, out, count, draft, mask, bias, allowed, allowed_row, repetition, presence, frequency,
                 masked, tree_len, None, B, N, dev_err, stream)


def jf_adjust_logits_packed(logits, out, cu_seqlens, N_max, count=None, draft=None, mask=None, bias=None,
                            allowed=None, allowed_row=None, repetition=None, presence=None, frequency=None,
                            masked=float("-inf"), dev_err=None, stream=None) -> None:
    """jf_adjust_logits on packed rows: logits [T][V], draft and allowed_row [T], mask [T][W]."""
    T, V = logits.shape
    _adjust_call(logits, out, count, draft, mask, bias, allowed, allowed_row, repetition, presence, frequency,
                 masked, None, cu_seqlens, cu_seqlens.shape[0] - 1, int(N_max), dev_err, stream)


def _adjust_call(logits, out, count, draft, mask, bias, allowed, allowed_row, repetition, presence, frequency,
                 masked, tree_len, cu_seqlens, B, N, dev_err, stream):
    shape = logits.shape
    V, lead = shape[-1], shape[:-1]
    dt, odt = _logit_dtype(logits), _logit_dtype(out)
    n_allowed = 0
    if allowed is not None:
        n_allowed = allowed.shape[0]
        if allowed_row is None and n_allowed != lead.numel():
            raise ValueError(f"allowed has {n_allowed} rows, one for each of {lead.numel()} nodes is expected")
    batch = (B,)
    (x, o, c, d, m, bi, al, ar, rep, pres, freq, tl, cu, err, on) = _pointers(
        (("logits", logits, logits.dtype, None), ("out", out, out.dtype, shape), ("count", count, _i32, (B, V)),
         ("draft", draft, _i32, lead), ("mask", mask, torch.int64, None if mask is None else lead + ((N + 63) // 64,)),
         ("bias", bias, _f32, (B, V)), ("allowed", allowed, _i32, (n_allowed, (V + 31) // 32)),
         ("allowed_row", allowed_row, _i32, lead), ("repetition", repetition, _f32, batch),
         ("presence", presence, _f32, batch), ("frequency", frequency, _f32, batch), ("tree_len", tree_len, _i32, batch),
         ("cu_seqlens", cu_seqlens, _i32, (B + 1,))), dev_err, stream)
    if cu is None:
        _check("jf_adjust_logits", _lib.jf_adjust_logits(
            x, dt, c, d, m, bi, al, ar, n_allowed, rep, pres, freq, masked, tl, B, N, V, o, odt, err, on))
    else:
        _check("jf_adjust_logits_packed", _lib.jf_adjust_logits_packed(
            x, dt, c, d, m, bi, al, ar, n_allowed, rep, pres, freq, masked, cu, B, N, lead[0], V, o, odt, err, on))


def jf_count_tokens(count, token, count_out, path=None, length=None, extra=None, row=None, prompt=False,
                    dev_err=None, stream=None) -> None:
    """Adds a step's tokens to the counts that jf_adjust_logits reads (see include/jf.h)."""
    B, N = token.shape
    V = count_out.shape[-1]
    rows_in = 0 if count is None else count.shape[0]
    batch = (B,)
    (c, t, o, pa, le, ex, ro, err, on) = _pointers(
        (("count", count, _i32, (rows_in, V)), ("token", token, _i32, None), ("count_out", count_out, _i32, (B, V)),
         ("path", path, _i32, (B, N)), ("length", length, _i32, batch), ("extra", extra, _i32, batch),
         ("row", row, _i32, batch)), dev_err, stream)
    _check("jf_count_tokens", _lib.jf_count_tokens(c, ro, rows_in, t, pa, le, ex, 1 if prompt else 0, B, N, V, o, err, on))


# ----------------------------------------------------------------------------- conveniences

def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    return torch.empty((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)


def build_tree_mask(parent: torch.Tensor, prefix_len: torch.Tensor, dev_err=None, stream=None,
                    tree_len=None):
    B, N = parent.shape
    W = (N + 63) // 64
    mask = torch.empty((B, N, W), dtype=torch.int64, device=parent.device)
    depth = torch.empty((B, N), dtype=torch.int32, device=parent.device)
    pos = torch.empty((B, N), dtype=torch.int32, device=parent.device)
    if tree_len is None:
        jf_build_tree_mask(parent, prefix_len, mask, depth, pos, dev_err, stream)
    else:
        jf_build_tree_mask_ragged(parent, prefix_len, tree_len, mask, depth, pos, dev_err, stream)
    return mask, depth, pos


def tree_attention(q, k_cache, v_cache, block_table, prefix_len, mask, scale=None,
                   with_lse=False, dev_err=None, stream=None, tree_len=None):
    B, N, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    if scale is None:
        scale = D ** -0.5
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if with_lse else None
    ws = _workspace(jf_tree_attention_workspace_size(B, N, Hq, Hkv, D, block_table.shape[1],
                                                     k_cache.shape[1]), q.device)
    if tree_len is None:
        jf_tree_attention(q, k_cache, v_cache, block_table, prefix_len, mask, scale, out, lse, ws,
                          dev_err, stream)
    else:
        jf_tree_attention_ragged(q, k_cache, v_cache, block_table, prefix_len, tree_len, mask,
                                 scale, out, lse, ws, dev_err, stream)
    return (out, lse) if with_lse else out


def tree_verify(logits, draft, parent, dev_err=None, stream=None, tree_len=None):
    B, N, V = logits.shape
    dev = logits.device
    argmax = torch.empty((B, N), dtype=torch.int32, device=dev)
    accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    path = torch.empty((B, N), dtype=torch.int32, device=dev)
    bonus = torch.empty((B,), dtype=torch.int32, device=dev)
    ws = _workspace(jf_tree_verify_workspace_size(B, N, V), dev)
    if tree_len is None:
        jf_tree_verify(logits, draft, parent, accept_len, path, bonus, argmax, ws, dev_err, stream)
    else:
        jf_tree_verify_ragged(logits, draft, parent, tree_len, accept_len, path, bonus, argmax, ws,
                              dev_err, stream)
    return argmax, accept_len, path, bonus


def tree_verify_sampled(logits, draft, parent, uniform, bonus_uniform, temperature=1.0,
                        dev_err=None, stream=None):
    """Allocating wrapper of jf_tree_verify_sampled: (accept_len, path, bonus)."""
    B, N, V = logits.shape
    dev = logits.device
    accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    path = torch.empty((B, N), dtype=torch.int32, device=dev)
    bonus = torch.empty((B,), dtype=torch.int32, device=dev)
    ws = _workspace(jf_tree_verify_workspace_size(B, N, V), dev)
    jf_tree_verify_sampled(logits, draft, parent, uniform, bonus_uniform, temperature, accept_len,
                           path, bonus, ws, dev_err, stream)
    return accept_len, path, bonus


def tree_verify_shard_keys(logits_shard, vocab_offset, chunks=None, stream=None):
    """Allocating wrapper of jf_tree_verify_shard_keys: int64 keys [B][N][chunks].  Every
    range must use the same chunks (by default the planned count for this range's size:
    pass the largest range's count when the ranges differ in size)."""
    B, N, Vs = logits_shard.shape
    if chunks is None:
        chunks = jf_tree_verify_shard_chunks(B, N, Vs)
    keys = torch.empty((B, N, chunks), dtype=torch.int64, device=logits_shard.device)
    jf_tree_verify_shard_keys(logits_shard, vocab_offset, keys, stream)
    return keys


def tree_verify_from_keys(keys, V, draft, parent, dev_err=None, stream=None):
    """Allocating wrapper of jf_tree_verify_from_keys on gathered keys [S][B][N][chunks]:
    (argmax, accept_len, path, bonus) as tree_verify returns them."""
    S, B, N, _ = keys.shape
    dev = keys.device
    argmax = torch.empty((B, N), dtype=torch.int32, device=dev)
    accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    path = torch.empty((B, N), dtype=torch.int32, device=dev)
    bonus = torch.empty((B,), dtype=torch.int32, device=dev)
    ws = torch.empty((8 * B * N,), dtype=torch.uint8, device=dev)
    jf_tree_verify_from_keys(keys, V, draft, parent, accept_len, path, bonus, ws, argmax,
                             dev_err, stream)
    return argmax, accept_len, path, bonus


def compact_accepted_kv(k_cache, v_cache, block_table, prefix_len, path, accept_len,
                        dev_err=None, stream=None):
    """In-place KV compaction after verification; returns the new prefix lengths."""
    new_prefix_len = torch.empty_like(prefix_len)
    jf_compact_accepted_kv(k_cache, v_cache, block_table, prefix_len, path, accept_len,
                           new_prefix_len, dev_err, stream)
    return new_prefix_len


def build_draft_tree(draft_logits, K, N, root_token=None, stream=None):
    """Returns (parent, draft, depth, score, cand_token, cand_logp)."""
    B, Dmax, V = draft_logits.shape
    dev = draft_logits.device
    cand_token = torch.empty((B, Dmax, K), dtype=torch.int32, device=dev)
    cand_logp = torch.empty((B, Dmax, K), dtype=torch.float32, device=dev)
    parent = torch.empty((B, N), dtype=torch.int32, device=dev)
    draft = torch.empty((B, N), dtype=torch.int32, device=dev)
    depth = torch.empty((B, N), dtype=torch.int32, device=dev)
    score = torch.empty((B, N), dtype=torch.float32, device=dev)
    jf_build_draft_tree(draft_logits, K, N, cand_token, cand_logp, parent, draft, depth,
                        root_token, score, stream)
    return parent, draft, depth, score, cand_token, cand_logp


def accumulate_attention_weight(q, k_cache, block_table, prefix_len, lse, path=None,
                                accept_len=None, weight=None, scale=None, cu_seqlens=None,
                                out=None, dev_err=None, stream=None):
    """Accumulated attention weight [B][Hkv][max_pages * page] after this step: weight (zeros
    if None) plus what the step's rows gave every key.  Written to out if given (out may be
    weight), else to a new tensor.  With cu_seqlens, q and lse are packed; N_max is then the
    path's width, or without a path the number of packed rows."""
    D = q.shape[-1]
    Hkv, page = k_cache.shape[2], k_cache.shape[1]
    B, max_pages = block_table.shape
    if scale is None:
        scale = D ** -0.5
    if out is None:
        if stream is not None:
            with _as_current(stream):
                return accumulate_attention_weight(q, k_cache, block_table, prefix_len, lse, path,
                                                   accept_len, weight, scale, cu_seqlens, None,
                                                   dev_err)
        out = torch.zeros((B, Hkv, max_pages * page), dtype=torch.float32, device=q.device)
    if cu_seqlens is None:
        jf_attention_weight(q, k_cache, block_table, prefix_len, lse, out, scale, path, accept_len,
                            weight, dev_err, stream)
    else:
        N_max = path.shape[1] if path is not None else min(q.shape[0], MAX_NODES)
        jf_attention_weight_packed(q, k_cache, block_table, prefix_len, cu_seqlens, lse, out, scale,
                                   N_max, path, accept_len, weight, dev_err, stream)
    return out


def select_kept_keys(weight, seq_len, budget, sink=0, recent=0, dev_err=None, stream=None):
    """(keep [B][Hkv][budget], kept_len [B]): the positions that stay, by weight."""
    if stream is not None:
        with _as_current(stream):
            return select_kept_keys(weight, seq_len, budget, sink, recent, dev_err)
    B, Hkv, _ = weight.shape
    keep = torch.empty((B, Hkv, budget), dtype=torch.int32, device=weight.device)
    kept_len = torch.empty((B,), dtype=torch.int32, device=weight.device)
    jf_select_kept(weight, seq_len, keep, kept_len, sink, recent, dev_err)
    return keep, kept_len


def evict_kv(k_cache, v_cache, block_table, seq_len, keep, kept_len, new_block_table=None,
             weight=None, weight_out=None, dev_err=None, stream=None):
    """Moves the kept rows to the front, in place or into new_block_table's pages; the weights
    likewise (in place if weight_out is None).  Returns kept_len, the new lengths."""
    if weight is not None and weight_out is None:
        weight_out = weight
    jf_evict_kv(k_cache, v_cache, block_table, seq_len, keep, kept_len, new_block_table, weight,
                weight_out, dev_err, stream)
    return kept_len


def beam_select(logits, score, K, finished=None, eos_token=-1, stream=None):
    """(parent, token, score, finished), each [B][K]: the K best continuations of every prompt."""
    if stream is not None:
        with _as_current(stream):
            return beam_select(logits, score, K, finished, eos_token)
    B, W, V = logits.shape
    dev = logits.device
    parent = torch.empty((B, K), dtype=torch.int32, device=dev)
    token = torch.empty((B, K), dtype=torch.int32, device=dev)
    new_finished = torch.empty((B, K), dtype=torch.int32, device=dev)
    new_score = torch.empty((B, K), dtype=torch.float32, device=dev)
    ws = _workspace(jf_beam_select_workspace_size(B, W, V, K, _logit_dtype(logits)), dev)
    jf_beam_select(logits, score, parent, token, new_score, ws, finished, eos_token, new_finished)
    return parent, token, new_score, new_finished


def beam_fork_kv(k_cache, v_cache, block_table, prefix_len, parent, fresh_page, dev_err=None,
                 stream=None):
    """(block_table [B * K][max_pages], prefix_len [B * K]) of the new beams."""
    if stream is not None:
        with _as_current(stream):
            return beam_fork_kv(k_cache, v_cache, block_table, prefix_len, parent, fresh_page, dev_err)
    B, K = parent.shape
    new_table = torch.empty((B * K, block_table.shape[1]), dtype=torch.int32,
                            device=block_table.device)
    new_len = torch.empty((B * K,), dtype=torch.int32, device=block_table.device)
    jf_beam_fork_kv(k_cache, v_cache, block_table, prefix_len, parent, fresh_page, new_table,
                    new_len, dev_err)
    return new_table, new_len


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, device="cuda"):
    """(freq, rotary_scale) for rotate_append_kv: float64 [rotary_dim / 2] radians per position,
    base^(-2 f / rotary_dim), and the factor on the rotated elements.  scaling for contexts longer
    than the model was trained on: None; ("linear", factor), every frequency divided by factor; or
    ("yarn", factor, trained_length), which divides the frequencies that turn less than once in
    trained_length positions, keeps those that turn more than 32 times, goes over between them in a
    linear ramp over the pair's index, and scales by 0.1 ln(factor) + 1."""
    f = torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim
    freq = float(base) ** -f
    if scaling is None:
        return freq.to(device), 1.0
    kind, factor = scaling[0], float(scaling[1])
    if not factor >= 1.0:
        raise ValueError(f"the scaling factor must be at least 1, got {factor}")
    if kind == "linear":
        return (freq / factor).to(device), 1.0
    if kind != "yarn":
        raise ValueError(f"unknown rotary scaling {kind!r}")
    length = float(scaling[2])

    def pair_of(turns):        # the (fractional) pair that turns so often in trained_length positions
        return rotary_dim * math.log(length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

    low = max(math.floor(pair_of(32.0)), 0)
    high = min(math.ceil(pair_of(1.0)), rotary_dim - 1)
    ramp = ((torch.arange(rotary_dim // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
    return (freq / factor * ramp + freq * (1.0 - ramp)).to(device), 0.1 * math.log(factor) + 1.0


def rotate_append_kv(q, k, v, k_cache, v_cache, block_table, prefix_len, pos=None, freq=None, interleaved=False,
                     rotary_scale=1.0, q_norm=None, k_norm=None, norm_eps=1e-6, tree_len=None, cu_seqlens=None,
                     N_max=None, out=None, dev_err=None, stream=None):
    """Appends the step's keys and values to the cache and returns its rotated queries (written to
    out if given; padding rows of a new tensor are zero).  q [B][N][Hq][D], or [T][Hq][D] with
    cu_seqlens (N_max: the longest sequence's rows, by default T)."""
    if out is None and q is not None:
        if stream is not None:
            with _as_current(stream):
                return rotate_append_kv(q, k, v, k_cache, v_cache, block_table, prefix_len, pos, freq, interleaved,
                                        rotary_scale, q_norm, k_norm, norm_eps, tree_len, cu_seqlens, N_max, None,
                                        dev_err)
        make = torch.empty if tree_len is None and cu_seqlens is None else torch.zeros
        out = make(q.shape, dtype=q.dtype, device=q.device)
    if cu_seqlens is None:
        if k.dim() != 4 or k.shape[0] != block_table.shape[0]:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected ({block_table.shape[0]}, N, Hkv, D)")
        lead = k.shape[:2]
    else:
        if k.dim() != 3:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected (T, Hkv, D)")
        lead = k.shape[:1]
        N_max = int(lead[0] if N_max is None else N_max)
    _rotate_call(q, k, v, k_cache, v_cache, block_table, prefix_len, lead, out, pos, freq, interleaved, rotary_scale,
                 q_norm, k_norm, norm_eps, tree_len, cu_seqlens, N_max, dev_err, stream)
    return out


def _largest_tree(T, B, max_pages, words) -> int:
    """The most nodes that one of B sequences in T packed rows can have: every other one has a row, the
    block table holds them, and the mask has `words` words a row (which says at least 64 (words - 1) + 1)."""
    return max(64 * (words - 1) + 1, min(64 * words, T - B + 1, PAGE_SIZE * max_pages))


def tree_attention_shared(q, k_cache, v_cache, block_table, prefix_len, mask, group_start, shared_pages, scale=None,
                          with_lse=False, tree_len=None, cu_seqlens=None, N_max=None, out=None, lse=None,
                          workspace=None, dev_err=None, stream=None):
    """Attention of sequences in groups that share a prefix; out, or (out, lse) with with_lse or a
    given lse.  New tensors' padding rows are zero.  With cu_seqlens the rows are packed; N_max is then
    the largest tree (by default the largest that mask's width, the table's and the number of rows,
    one at least a sequence, allow)."""
    with_lse = with_lse or lse is not None
    if stream is not None and (out is None or workspace is None or (with_lse and lse is None)):
        with _as_current(stream):
            return tree_attention_shared(q, k_cache, v_cache, block_table, prefix_len, mask, group_start,
                                         shared_pages, scale, with_lse, tree_len, cu_seqlens, N_max, out, lse,
                                         workspace, dev_err)
    shape = q.shape
    Hq, D = shape[-2:]
    B, max_pages = block_table.shape
    if scale is None:
        scale = D ** -0.5
    packed = cu_seqlens is not None
    if packed and N_max is None:
        N_max = _largest_tree(shape[0], B, max_pages, mask.shape[-1])
    if out is None or (with_lse and lse is None):
        make = torch.zeros if packed or tree_len is not None else torch.empty
        if out is None:
            out = make(shape, dtype=q.dtype, device=q.device)
        if with_lse and lse is None:
            lse = make((Hq, shape[0]) if packed else (B, Hq, shape[1]), dtype=torch.float32, device=q.device)
    if workspace is None:
        page, Hkv = k_cache.shape[1:3]
        N, T = (N_max, shape[0]) if packed else (shape[1], 0)
        workspace = q.new_empty(_shared_workspace(torch._C._cuda_getDevice(), B, N, shared_pages.shape[0], Hq, Hkv, D,
                                                  max_pages, T, page), dtype=torch.uint8)
    if packed:
        jf_tree_attention_shared_packed(q, k_cache, v_cache, block_table, prefix_len, cu_seqlens, N_max, mask,
                                        group_start, shared_pages, scale, out, workspace, lse, dev_err, stream)
    else:
        jf_tree_attention_shared(q, k_cache, v_cache, block_table, prefix_len, mask, group_start, shared_pages, scale,
                                 out, workspace, lse, tree_len, dev_err, stream)
    return (out, lse) if with_lse else out


def adjust_logits(logits, count=None, draft=None, mask=None, bias=None, allowed=None, allowed_row=None,
                  repetition=None, presence=None, frequency=None, masked=float("-inf"), tree_len=None,
                  cu_seqlens=None, N_max=None, out=None, dev_err=None, stream=None):
    """The logits under penalties, biases and grammar masks: written to out if given (out may be
    logits), else to a new tensor, whose padding rows are zero.  With cu_seqlens the rows are packed;
    N_max is then the largest tree (by default what mask's width allows, or without one the rows)."""
    if out is None:
        if stream is not None:
            with _as_current(stream):
                return adjust_logits(logits, count, draft, mask, bias, allowed, allowed_row, repetition, presence,
                                     frequency, masked, tree_len, cu_seqlens, N_max, None, dev_err)
        make = torch.empty if tree_len is None and cu_seqlens is None else torch.zeros
        out = make(logits.shape, dtype=logits.dtype, device=logits.device)
    if cu_seqlens is None:
        B, N, _ = logits.shape
        _adjust_call(logits, out, count, draft, mask, bias, allowed, allowed_row, repetition, presence, frequency, masked,
                     tree_len, None, B, N, dev_err, stream)
    else:
        if N_max is None:
            N_max = min(logits.shape[0], MAX_NODES) if mask is None else 64 * mask.shape[-1]
        jf_adjust_logits_packed(logits, out, cu_seqlens, N_max, count, draft, mask, bias, allowed, allowed_row,
                                repetition, presence, frequency, masked, dev_err, stream)
    return out


def count_tokens(count, token, path=None, length=None, extra=None, row=None, prompt=False, V=None, out=None,
                 dev_err=None, stream=None):
    """The counts with a step's tokens added, in place (out=count), in out, or in a new tensor.
    count None: zeros, over a vocabulary of V tokens (or out's)."""
    if out is None:
        if stream is not None:
            with _as_current(stream):
                return count_tokens(count, token, path, length, extra, row, prompt, V, None, dev_err)
        size = count.shape[-1] if count is not None else int(V)
        out = torch.empty((token.shape[0], size), dtype=torch.int32, device=token.device)
    jf_count_tokens(count, token, out, path, length, extra, row, prompt, dev_err, stream)
    return out
