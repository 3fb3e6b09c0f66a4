"""ctypes binding of libkdverify.so (declared in include/kd_verify.h).

Argument marshalling only: shape/dtype checks, ``data_ptr()``s, the current
CUDA stream.  Every step of the verify path runs in the library's kernels.
Importing this module raises if the library has not been built.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkdverify.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m tree_speculative_decoding_kd_b200.build`")

lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64
_f = ctypes.c_float
_sz = ctypes.c_size_t

_SIGS = {
    "kd_tree_build_mask": (_i, [_p, _i, _i, _p, _p, _p, _p]),
    "kd_verify_workspace_bytes": (_sz, [_i, _i, _i, _i64, _i]),
    "kd_tree_verify_attn": (_i, [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _p, _i, _i, _i, _f,
                                 _p, _p, _p, _sz, _i, _p]),
    "kd_tree_verify_attn_simt": (_i, [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _p, _i, _i, _i,
                                      _f, _p, _p, _p, _p]),
    "kd_tree_verify_attn_noalloc": (_i, [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _p, _i, _i, _i,
                                         _f, _p, _p, _i, _p, _p]),
    "kd_tree_accept": (_i, [_p, _p, _p, _i, _i, _p, _p, _p, _p, _p]),
    "kd_accept_workspace_bytes": (_sz, [_i, _i]),
    "kd_tree_build": (_i, [_p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p, _p]),
    "kd_tree_verify_attn_paged": (_i, [_p, _p, _p, _p, _i64, _i64, _i, _p, _i64, _i64, _p, _p, _p, _i,
                                       _i, _i, _f, _p, _p, _p, _sz, _i, _p]),
    "kd_kv_write_nodes_paged": (_i, [_p, _p, _i64, _i64, _i, _p, _i64, _i64, _p, _p, _p, _i, _i, _p,
                                     _p]),
    "kd_kv_compact_paged": (_i, [_p, _p, _i64, _i64, _i, _p, _i64, _i64, _p, _p, _p, _i, _i, _p, _p]),
    "kd_tree_accept_logits": (_i, [_p, _p, _p, _i, _i, _i64, _p, _p, _p, _p, _p, _sz, _p, _p]),
    "kd_kv_compact": (_i, [_p, _p, _i64, _i64, _i64, _p, _p, _p, _i, _i, _p, _p]),
    "kd_kv_write_nodes": (_i, [_p, _p, _i64, _i64, _i64, _p, _p, _p, _i, _i, _p, _p]),
    "kd_qk_norm_rope": (_i, [_p, _i64, _i64, _p, _i64, _i64, _p, _p, _f, _p, _i64, _p, _i, _i, _i, _i, _i, _i,
                             _i, _p, _i64, _i64, _p, _i64, _i64, _p, _p]),
    "kd_kv_norm_rope_write": (_i, [_p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _f, _p, _i64, _p, _i, _p, _i, _i,
                                   _p, _i64, _i64, _i, _p, _p, _p]),
    "kd_kv_norm_rope_write_paged": (_i, [_p, _p, _i64, _i64, _i, _p, _i64, _i64, _p, _p, _i64, _p, _f, _p, _i64,
                                         _p, _i, _p, _i, _i, _p, _i64, _i64, _i, _p, _p, _p]),
    "kd_prompt_attn": (_i, [_p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _p,
                            _i, _i, _i, _i, _i, _f, _p, _p, _p, _p]),
    "kd_kv_attn_weights": (_i, [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p, _i, _i, _i, _f, _p, _i64, _p,
                                _i64, _p, _p]),
    "kd_kv_attn_weights_paged": (_i, [_p, _p, _p, _p, _i64, _i64, _i, _p, _i64, _i64, _p, _p, _p, _p, _p, _i, _i,
                                      _i, _f, _p, _i64, _p, _i64, _p, _p]),
    "kd_kv_evict": (_i, [_p, _p, _i64, _i64, _i64, _p, _p, _i64, _i, _i, _i, _i, _p, _p, _i64, _i64, _i64, _p, _i64,
                         _p, _p, _p, _p]),
    "kd_kv_evict_paged": (_i, [_p, _p, _i64, _i64, _i, _p, _i64, _i64, _p, _p, _i64, _i, _i, _i, _i, _p, _p, _i64,
                               _i64, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p]),
    "kd_call_packed": (_i, [_i, ctypes.c_char_p, _i]),
    "kd_read_device_error": (_i, [_p, _i, _p]),
    "kd_strerror": (ctypes.c_char_p, [_i]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

# Calls made through kd_call_packed, in the order of their op codes.
_PACKED = ("kd_qk_norm_rope", "kd_kv_norm_rope_write", "kd_kv_norm_rope_write_paged", "kd_prompt_attn",
           "kd_kv_attn_weights", "kd_kv_attn_weights_paged", "kd_kv_evict", "kd_kv_evict_paged")


def _packed(name):
    """The call `name` with its arguments (integers, addresses with 0 for none, floats) packed into
    one buffer: converting them one by one costs ctypes more than the launch of a small call."""
    op, types = _PACKED.index(name), _SIGS[name][1]
    pack, count = struct.Struct("".join("d" if t is _f else "q" for t in types)).pack, len(types)

    def call(*args):
        rc = lib.kd_call_packed(op, pack(*args), count)
        if rc:
            _check(rc, name)
    return call


D_C, D_R = 512, 64
KD_DEV_BITS = {0x01: "BAD_PARENT", 0x02: "CACHE_FULL", 0x04: "BAD_PATH",
               0x08: "BAD_POSITION", 0x10: "TIMEOUT", 0x20: "BAD_MASK", 0x40: "BAD_PAGE",
               0x80: "BAD_SEQLENS"}


class KdError(RuntimeError):
    pass


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise KdError(f"{what}: {lib.kd_strerror(rc).decode()} (code {rc})")


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _stream_of(stream, device) -> int:
    """_stream for the calls whose host time counts: the current stream's handle without a Stream object."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _addr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _need(t, dtype, name, contiguous=True):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dts = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in dts:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dts}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _cache_strides(c_kv, k_rope):
    """Row strides (elements) of [B][cap][512] / [B][cap][64] cache views."""
    _need(c_kv, torch.bfloat16, "c_kv", contiguous=False)
    _need(k_rope, torch.bfloat16, "k_rope", contiguous=False)
    B, cap, dc = c_kv.shape
    if dc != D_C or tuple(k_rope.shape) != (B, cap, D_R):
        raise ValueError("c_kv must be [B][cap][512] and k_rope [B][cap][64]")
    for t in (c_kv, k_rope):
        if t.stride(2) != 1 or t.stride(0) != cap * t.stride(1):
            raise ValueError("cache rows must be unit-stride with uniform row pitch")
    return c_kv.stride(1), k_rope.stride(1), cap


def new_error_word(device=None) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def kd_tree_build_mask(parents, vis=None, depth=None, dev_error=None, stream=None):
    _need(parents, torch.int32, "parents")
    B, n = parents.shape
    W = (n + 31) // 32
    if vis is None:
        vis = torch.empty(B, n, W, dtype=torch.int32, device=parents.device)
    if depth is None:
        depth = torch.empty(B, n, dtype=torch.int32, device=parents.device)
    _check(lib.kd_tree_build_mask(_ptr(parents), B, n, _ptr(vis), _ptr(depth), _ptr(dev_error),
                                  _stream(stream)), "kd_tree_build_mask")
    return vis, depth


def kd_verify_workspace_bytes(B, n, H, cap, kv_splits=0) -> int:
    return int(lib.kd_verify_workspace_bytes(B, n, H, cap, kv_splits))


def new_workspace(B, n, H, cap, kv_splits=0, device=None) -> torch.Tensor:
    """Zeroed workspace (its first int32 is the device error word)."""
    nbytes = kd_verify_workspace_bytes(B, n, H, cap, kv_splits)
    if nbytes == 0:
        raise ValueError("invalid shape for the verify workspace")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


def _attn_args(q_abs, q_rope, c_kv, k_rope, cache_lens, vis, positions, out, lse):
    _need(q_abs, torch.bfloat16, "q_abs")
    _need(q_rope, torch.bfloat16, "q_rope")
    _need(cache_lens, torch.int32, "cache_lens")
    _need(vis, (torch.int32, torch.uint32), "vis")
    B, n, H, dc = q_abs.shape
    if dc != D_C or tuple(q_rope.shape) != (B, n, H, D_R):
        raise ValueError("q_abs must be [B][n][H][512] and q_rope [B][n][H][64]")
    if positions is not None:
        _need(positions, torch.int32, "positions")
    sc, sr, cap = _cache_strides(c_kv, k_rope)
    if out is None:
        out = torch.empty(B, n, H, D_C, dtype=torch.bfloat16, device=q_abs.device)
    if lse is None:
        lse = torch.empty(B, n, H, dtype=torch.float32, device=q_abs.device)
    _need(out, torch.bfloat16, "out")
    _need(lse, torch.float32, "lse")
    return B, n, H, sc, sr, cap, out, lse


def kd_tree_verify_attn(q_abs, q_rope, c_kv, k_rope, cache_lens, vis, positions=None,
                        scale=1.0 / math.sqrt(192.0), out=None, lse=None, workspace=None,
                        kv_splits=0, stream=None):
    B, n, H, sc, sr, cap, out, lse = _attn_args(q_abs, q_rope, c_kv, k_rope, cache_lens, vis,
                                                positions, out, lse)
    if workspace is None:
        workspace = new_workspace(B, n, H, cap, kv_splits, q_abs.device)
    _check(lib.kd_tree_verify_attn(_ptr(q_abs), _ptr(q_rope), _ptr(c_kv), _ptr(k_rope), sc, sr,
                                   cap, _ptr(cache_lens), _ptr(vis), _ptr(positions), B, n, H,
                                   float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), int(kv_splits),
                                   _stream(stream)), "kd_tree_verify_attn")
    return out, lse


def kd_tree_verify_attn_noalloc(q_abs, q_rope, c_kv, k_rope, cache_lens, vis, positions=None,
                                scale=1.0 / math.sqrt(192.0), out=None, lse=None, kv_splits=0,
                                dev_error=None, stream=None):
    """kd_tree_verify_attn with the library's fixed workspace.

    The C call allocates no device memory.  This wrapper does when `out` or `lse`
    is None (it creates them with torch); under CUDA graph capture or on an
    allocation-free path pass both, and `dev_error`, preallocated.  With
    `dev_error` None the call's device errors are discarded."""
    B, n, H, sc, sr, cap, out, lse = _attn_args(q_abs, q_rope, c_kv, k_rope, cache_lens, vis,
                                                positions, out, lse)
    _check(lib.kd_tree_verify_attn_noalloc(_ptr(q_abs), _ptr(q_rope), _ptr(c_kv), _ptr(k_rope), sc,
                                           sr, cap, _ptr(cache_lens), _ptr(vis), _ptr(positions),
                                           B, n, H, float(scale), _ptr(out), _ptr(lse),
                                           int(kv_splits), _ptr(dev_error), _stream(stream)),
           "kd_tree_verify_attn_noalloc")
    return out, lse


def kd_tree_verify_attn_simt(q_abs, q_rope, c_kv, k_rope, cache_lens, vis, positions=None,
                             scale=1.0 / math.sqrt(192.0), out=None, lse=None, dev_error=None,
                             stream=None):
    B, n, H, sc, sr, cap, out, lse = _attn_args(q_abs, q_rope, c_kv, k_rope, cache_lens, vis,
                                                positions, out, lse)
    _check(lib.kd_tree_verify_attn_simt(_ptr(q_abs), _ptr(q_rope), _ptr(c_kv), _ptr(k_rope), sc,
                                        sr, cap, _ptr(cache_lens), _ptr(vis), _ptr(positions), B,
                                        n, H, float(scale), _ptr(out), _ptr(lse),
                                        _ptr(dev_error), _stream(stream)),
           "kd_tree_verify_attn_simt")
    return out, lse


def kd_tree_build(logp, cand_tokens, root_tokens, n, parents=None, tokens=None, depth=None, score=None,
                  stream=None):
    """Best-first draft trees: logp fp32 [B][D][K] (sorted per depth), cand_tokens int32
    [B][D][K], root_tokens int32 [B] -> (parents, tokens, depth, score), each [B][n]
    (allocated here unless given)."""
    _need(logp, torch.float32, "logp")
    _need(cand_tokens, torch.int32, "cand_tokens")
    _need(root_tokens, torch.int32, "root_tokens")
    B, D, K = logp.shape
    if tuple(cand_tokens.shape) != (B, D, K) or tuple(root_tokens.shape) != (B,):
        raise ValueError("cand_tokens must be [B][D][K] and root_tokens [B]")
    dev = logp.device
    if parents is None:
        parents = torch.empty(B, n, dtype=torch.int32, device=dev)
    if tokens is None:
        tokens = torch.empty(B, n, dtype=torch.int32, device=dev)
    if depth is None:
        depth = torch.empty(B, n, dtype=torch.int32, device=dev)
    if score is None:
        score = torch.empty(B, n, dtype=torch.float32, device=dev)
    for t, dt, name in ((parents, torch.int32, "parents"), (tokens, torch.int32, "tokens"),
                        (depth, torch.int32, "depth"), (score, torch.float32, "score")):
        _need(t, dt, name)
        if tuple(t.shape) != (B, n):
            raise ValueError(f"{name} must be [B][n]")
    _check(lib.kd_tree_build(_ptr(logp), _ptr(cand_tokens), _ptr(root_tokens), B, D, K, n,
                             _ptr(parents), _ptr(tokens), _ptr(depth), _ptr(score), _stream(stream)),
           "kd_tree_build")
    return parents, tokens, depth, score


def new_accept_workspace(B, n, device=None) -> torch.Tensor:
    nbytes = int(lib.kd_accept_workspace_bytes(B, n))
    if nbytes == 0:
        raise KdError("kd_accept_workspace_bytes: invalid shapes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def kd_tree_accept_logits(node_tokens, parents, logits, target_argmax=None, path=None,
                          length=None, bonus=None, workspace=None, dev_error=None, stream=None):
    """Target argmax of fp32 logits [B][n][V] fused with greedy acceptance.
    Returns (target_argmax, path, len, bonus)."""
    for t, nm in ((node_tokens, "node_tokens"), (parents, "parents")):
        _need(t, torch.int32, nm)
    _need(logits, torch.float32, "logits")
    B, n = parents.shape
    if logits.dim() != 3 or tuple(logits.shape[:2]) != (B, n):
        raise ValueError("logits must be [B][n][V]")
    V = logits.shape[2]
    dev = parents.device
    if target_argmax is None:
        target_argmax = torch.empty(B, n, dtype=torch.int32, device=dev)
    path = torch.empty(B, n, dtype=torch.int32, device=dev) if path is None else path
    length = torch.empty(B, dtype=torch.int32, device=dev) if length is None else length
    bonus = torch.empty(B, dtype=torch.int32, device=dev) if bonus is None else bonus
    workspace = new_accept_workspace(B, n, dev) if workspace is None else workspace
    _check(lib.kd_tree_accept_logits(_ptr(node_tokens), _ptr(parents), _ptr(logits), B, n, V,
                                     _ptr(target_argmax), _ptr(path), _ptr(length), _ptr(bonus),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _ptr(dev_error), _stream(stream)), "kd_tree_accept_logits")
    return target_argmax, path, length, bonus


def kd_tree_accept(node_tokens, parents, target_argmax, path=None, length=None, bonus=None,
                   dev_error=None, stream=None):
    for t, nm in ((node_tokens, "node_tokens"), (parents, "parents"), (target_argmax, "target_argmax")):
        _need(t, torch.int32, nm)
    B, n = parents.shape
    dev = parents.device
    path = torch.empty(B, n, dtype=torch.int32, device=dev) if path is None else path
    length = torch.empty(B, dtype=torch.int32, device=dev) if length is None else length
    bonus = torch.empty(B, dtype=torch.int32, device=dev) if bonus is None else bonus
    _check(lib.kd_tree_accept(_ptr(node_tokens), _ptr(parents), _ptr(target_argmax), B, n,
                              _ptr(path), _ptr(length), _ptr(bonus), _ptr(dev_error),
                              _stream(stream)), "kd_tree_accept")
    return path, length, bonus


def kd_kv_compact(c_kv, k_rope, path, length, cache_lens, dev_error=None, stream=None):
    sc, sr, cap = _cache_strides(c_kv, k_rope)
    _need(path, torch.int32, "path")
    _need(length, torch.int32, "len")
    _need(cache_lens, torch.int32, "cache_lens")
    B, n = path.shape
    _check(lib.kd_kv_compact(_ptr(c_kv), _ptr(k_rope), sc, sr, cap, _ptr(path), _ptr(length),
                             _ptr(cache_lens), B, n, _ptr(dev_error), _stream(stream)),
           "kd_kv_compact")


def kd_kv_write_nodes(c_kv, k_rope, cache_lens, node_ckv, node_krope, dev_error=None, stream=None):
    sc, sr, cap = _cache_strides(c_kv, k_rope)
    _need(node_ckv, torch.bfloat16, "node_ckv")
    _need(node_krope, torch.bfloat16, "node_krope")
    _need(cache_lens, torch.int32, "cache_lens")
    B, n, _ = node_ckv.shape
    _check(lib.kd_kv_write_nodes(_ptr(c_kv), _ptr(k_rope), sc, sr, cap, _ptr(cache_lens),
                                 _ptr(node_ckv), _ptr(node_krope), B, n, _ptr(dev_error),
                                 _stream(stream)), "kd_kv_write_nodes")


def _page_args(c_pages, r_pages, page_table, page_size):
    """Strides, pages per request and pool size of a paged cache: pools [rows][512] /
    [rows][64] bf16 (rows = num_pages * page_size), page_table int32 [B][M]."""
    _need(c_pages, torch.bfloat16, "c_pages", contiguous=False)
    _need(r_pages, torch.bfloat16, "r_pages", contiguous=False)
    _need(page_table, torch.int32, "page_table")
    rows = c_pages.shape[0]
    if c_pages.dim() != 2 or c_pages.shape[1] != D_C or tuple(r_pages.shape) != (rows, D_R):
        raise ValueError("c_pages must be [rows][512] and r_pages [rows][64]")
    if rows % page_size:
        raise ValueError("pool rows must be a multiple of page_size")
    for t in (c_pages, r_pages):
        if t.stride(1) != 1:
            raise ValueError("pool rows must be unit-stride")
    return c_pages.stride(0), r_pages.stride(0), page_table.shape[1], rows // page_size


def kd_tree_verify_attn_paged(q_abs, q_rope, c_pages, r_pages, page_table, page_size, cache_lens, vis,
                              positions=None, scale=1.0 / math.sqrt(192.0), out=None, lse=None,
                              workspace=None, kv_splits=0, stream=None):
    sc, sr, M, N = _page_args(c_pages, r_pages, page_table, page_size)
    _need(q_abs, torch.bfloat16, "q_abs")
    _need(q_rope, torch.bfloat16, "q_rope")
    _need(cache_lens, torch.int32, "cache_lens")
    _need(vis, (torch.int32, torch.uint32), "vis")
    B, n, H, _ = q_abs.shape
    if positions is not None:
        _need(positions, torch.int32, "positions")
    out = torch.empty(B, n, H, D_C, dtype=torch.bfloat16, device=q_abs.device) if out is None else out
    lse = torch.empty(B, n, H, dtype=torch.float32, device=q_abs.device) if lse is None else lse
    if workspace is None:
        workspace = new_workspace(B, n, H, M * page_size, kv_splits, q_abs.device)
    _check(lib.kd_tree_verify_attn_paged(_ptr(q_abs), _ptr(q_rope), _ptr(c_pages), _ptr(r_pages), sc, sr,
                                         int(page_size), _ptr(page_table), M, N, _ptr(cache_lens),
                                         _ptr(vis), _ptr(positions), B, n, H, float(scale), _ptr(out),
                                         _ptr(lse), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), int(kv_splits),
                                         _stream(stream)), "kd_tree_verify_attn_paged")
    return out, lse


def kd_kv_write_nodes_paged(c_pages, r_pages, page_table, page_size, cache_lens, node_ckv, node_krope,
                            dev_error=None, stream=None):
    sc, sr, M, N = _page_args(c_pages, r_pages, page_table, page_size)
    _need(node_ckv, torch.bfloat16, "node_ckv")
    _need(node_krope, torch.bfloat16, "node_krope")
    _need(cache_lens, torch.int32, "cache_lens")
    B, n, _ = node_ckv.shape
    _check(lib.kd_kv_write_nodes_paged(_ptr(c_pages), _ptr(r_pages), sc, sr, int(page_size),
                                       _ptr(page_table), M, N, _ptr(cache_lens), _ptr(node_ckv),
                                       _ptr(node_krope), B, n, _ptr(dev_error), _stream(stream)),
           "kd_kv_write_nodes_paged")


def kd_kv_compact_paged(c_pages, r_pages, page_table, page_size, path, length, cache_lens, dev_error=None,
                        stream=None):
    sc, sr, M, N = _page_args(c_pages, r_pages, page_table, page_size)
    _need(path, torch.int32, "path")
    _need(length, torch.int32, "len")
    _need(cache_lens, torch.int32, "cache_lens")
    B, n = path.shape
    _check(lib.kd_kv_compact_paged(_ptr(c_pages), _ptr(r_pages), sc, sr, int(page_size), _ptr(page_table),
                                   M, N, _ptr(path), _ptr(length), _ptr(cache_lens), B, n,
                                   _ptr(dev_error), _stream(stream)), "kd_kv_compact_paged")


# ------------------------------------------------------------------ operators next to the verify step
_call_qk_norm_rope = _packed("kd_qk_norm_rope")
_call_kv_norm_rope_write = _packed("kd_kv_norm_rope_write")
_call_kv_norm_rope_write_paged = _packed("kd_kv_norm_rope_write_paged")
_call_prompt_attn = _packed("kd_prompt_attn")
_call_kv_attn_weights = _packed("kd_kv_attn_weights")
_call_kv_attn_weights_paged = _packed("kd_kv_attn_weights_paged")
_call_kv_evict = _packed("kd_kv_evict")
_call_kv_evict_paged = _packed("kd_kv_evict_paged")


def _on_device(*tensors) -> int:
    """Index of the current CUDA device, on which every tensor given (None skipped) has to lie."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError("every tensor must be a CUDA tensor")
                if dev is not None:
                    raise ValueError(f"tensors on cuda:{dev} and cuda:{d}")
                dev = d
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{dev}, the current device is cuda:{torch._C._cuda_getDevice()}")
    return dev


def _new(stream, make, *shape, dtype, device):
    """A result tensor by make (torch.empty, torch.zeros), allocated and filled on the call's stream."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _typed(t, dtype, name, shape=None):
    """Contiguous tensor of `dtype` and, when given, of `shape`."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, has {tuple(t.shape)}")


def _heads(t, name, tokens=None, heads=None, width=None):
    """Shape and token and head strides of a bf16 [tokens][heads][width] view (unit stride inside a head;
    0 for an axis of length 1, whose stride torch leaves arbitrary)."""
    if t.dtype is not torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{name} must be bf16 [tokens][heads][width]")
    T, H, D = t.shape
    if (tokens is not None and T != tokens) or (heads is not None and H != heads) or (width is not None and D != width):
        raise ValueError(f"{name} must be {[tokens, heads, width]} (None: any), is {[T, H, D]}")
    if T == 0 or H == 0:
        return T, H, D, 0, 0
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must have unit stride inside a head")
    return T, H, D, st if T > 1 else 0, sh if H > 1 else 0


def _cache(c, r):
    """Requests, row strides and capacity of a contiguous cache [B][cap][512] / [B][cap][64]."""
    if c.dtype is not torch.bfloat16 or r.dtype is not torch.bfloat16:
        raise ValueError("caches must be bf16")
    B, cap, dc = c.shape
    if dc != D_C or r.shape != (B, cap, D_R):
        raise ValueError("c_kv must be [B][cap][512] and k_rope [B][cap][64]")
    cb, sc, c1 = c.stride()
    rb, sr, r1 = r.stride()
    if c1 != 1 or r1 != 1 or cb != cap * sc or rb != cap * sr:
        raise ValueError("cache rows must be unit-stride with uniform row pitch")
    return B, sc, sr, cap


def _pages(c, r, page_table, page_size, B):
    """Row strides, pages per request and pool size of a paged cache of B requests."""
    if c.dtype is not torch.bfloat16 or r.dtype is not torch.bfloat16:
        raise ValueError("page pools must be bf16")
    rows, dc = c.shape
    if dc != D_C or r.shape != (rows, D_R):
        raise ValueError("c_pages must be [rows][512] and r_pages [rows][64]")
    if page_size < 1 or rows % page_size:
        raise ValueError("pool rows must be a multiple of page_size")
    sc, c1 = c.stride()
    sr, r1 = r.stride()
    if c1 != 1 or r1 != 1:
        raise ValueError("pool rows must be unit-stride")
    _typed(page_table, torch.int32, "page_table")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B][pages per request]")
    return sc, sr, page_table.shape[1], rows // page_size


def _rope_table(table, rot):
    _typed(table, torch.float32, "rope_table")
    if table.dim() != 2 or (rot is not None and table.shape[1] != rot):
        raise ValueError("rope_table must be [max_pos][rot]")
    return table.shape


def kd_qk_norm_rope(q, k, positions, rope_table, q_weight=None, k_weight=None, eps=1e-6, rot_offset=0,
                    interleaved=False, q_out=None, k_out=None, dev_error=None, stream=None):
    """RMS norm of every head of q [T][H][D] and k [T][Hk][D] (k None: queries alone; a weight
    None: no norm) and the rotation of its elements [rot_offset, rot_offset + rot) by
    positions [T] int32; rope_table fp32 [max_pos][rot], cos | sin.  Returns (q_out, k_out),
    allocated contiguous unless given (not cleared: a bad position's rows hold what was in
    memory); q_out=q, k_out=k works in place."""
    dev = _on_device(q, k, positions, rope_table, q_weight, k_weight, q_out, k_out, dev_error)
    T, H, D, qt, qh = _heads(q, "q")
    _typed(positions, torch.int32, "positions", (T,))
    max_pos, rot = _rope_table(rope_table, None)
    if q_weight is not None:
        _typed(q_weight, torch.bfloat16, "q_weight", (D,))
    if q_out is None:
        q_out = _new(stream, torch.empty, T, H, D, dtype=torch.bfloat16, device=q.device)
    _, _, _, qot, qoh = _heads(q_out, "q_out", T, H, D)
    Hk = kt = kh = kot = koh = 0
    if k is not None:
        _, Hk, _, kt, kh = _heads(k, "k", T, None, D)
        if k_weight is not None:
            _typed(k_weight, torch.bfloat16, "k_weight", (D,))
        if k_out is None:
            k_out = _new(stream, torch.empty, T, Hk, D, dtype=torch.bfloat16, device=q.device)
        _, _, _, kot, koh = _heads(k_out, "k_out", T, Hk, D)
    _call_qk_norm_rope(q.data_ptr(), qt, qh, _addr(k), kt, kh, _addr(q_weight), _addr(k_weight), eps,
        rope_table.data_ptr(), max_pos, positions.data_ptr(), T, H, Hk, D, rot, rot_offset, interleaved,
        q_out.data_ptr(), qot, qoh, _addr(k_out), kot, koh, _addr(dev_error), _stream_of(stream, dev))
    return q_out, k_out


def _write_args(cache_lens, kv, positions, rope_table, kv_weight, cu_seqlens, B, q_rope_in, q_rope_out, stream):
    _typed(cache_lens, torch.int32, "cache_lens")
    if B is None:
        B = cache_lens.shape[0]
    if cache_lens.shape[0] != B:
        raise ValueError("cache_lens must be [B]")
    if kv.dtype is not torch.bfloat16 or kv.dim() != 2 or kv.shape[1] != D_C + D_R or kv.stride(1) != 1:
        raise ValueError("kv must be bf16 [T][576] with unit-stride rows")
    T = kv.shape[0]
    row = kv.stride(0) if T > 1 else D_C + D_R
    max_pos, _ = _rope_table(rope_table, D_R)
    if positions is not None:
        _typed(positions, torch.int32, "positions", (T,))
    if kv_weight is not None:
        _typed(kv_weight, torch.bfloat16, "kv_weight", (D_C,))
    if cu_seqlens is not None:
        _typed(cu_seqlens, torch.int32, "cu_seqlens", (B + 1,))
    elif B < 1 or T % B:
        raise ValueError("without cu_seqlens the tokens must divide evenly among the requests")
    H = qt = qh = 0
    if q_rope_in is not None:
        _, H, _, qt, qh = _heads(q_rope_in, "q_rope_in", T, None, D_R)
        if q_rope_out is None:
            q_rope_out = _new(stream, torch.empty, T, H, D_R, dtype=torch.bfloat16, device=kv.device)
        _typed(q_rope_out, torch.bfloat16, "q_rope_out", (T, H, D_R))
    elif q_rope_out is not None:
        raise ValueError("q_rope_out without q_rope_in")
    return B, T, row, max_pos, H, qt, qh, q_rope_out


def kd_kv_norm_rope_write(c_kv, k_rope, cache_lens, kv, positions, rope_table, cu_seqlens=None, B=None,
                          kv_weight=None, eps=1e-6, interleaved=True, q_rope_in=None, q_rope_out=None,
                          dev_error=None, stream=None):
    """Cache rows of new tokens from the down-projection's output kv [T][576]: the latent
    normed, the rope key rotated, both stored at slots cache_lens[b] + i; the queries' rope
    part q_rope_in [T][H][64] rotated beside them.  positions None: cache_lens[b] + i;
    cu_seqlens None: T / B tokens per request.  Returns q_rope_out (None without queries;
    allocated unless given, and then not cleared: rows of bad positions or lengths, or behind
    the last sequence, hold what was in memory)."""
    dev = _on_device(c_kv, k_rope, cache_lens, kv, positions, rope_table, cu_seqlens, kv_weight, q_rope_in, q_rope_out,
               dev_error)
    rows, sc, sr, cap = _cache(c_kv, k_rope)
    B, T, row, max_pos, H, qt, qh, q_rope_out = _write_args(cache_lens, kv, positions, rope_table, kv_weight, cu_seqlens,
                                                            B, q_rope_in, q_rope_out, stream)
    if rows != B:
        raise ValueError("the cache must hold B requests")
    _call_kv_norm_rope_write(c_kv.data_ptr(), k_rope.data_ptr(), sc, sr, cap, cache_lens.data_ptr(), kv.data_ptr(),
        row, _addr(kv_weight), eps, rope_table.data_ptr(), max_pos, _addr(positions), interleaved,
        _addr(cu_seqlens), B, T, _addr(q_rope_in), qt, qh, H, _addr(q_rope_out), _addr(dev_error),
        _stream_of(stream, dev))
    return q_rope_out


def kd_kv_norm_rope_write_paged(c_pages, r_pages, page_table, page_size, cache_lens, kv, positions, rope_table,
                                cu_seqlens=None, B=None, kv_weight=None, eps=1e-6, interleaved=True, q_rope_in=None,
                                q_rope_out=None, dev_error=None, stream=None):
    """kd_kv_norm_rope_write through a page table."""
    dev = _on_device(c_pages, r_pages, page_table, cache_lens, kv, positions, rope_table, cu_seqlens, kv_weight, q_rope_in,
               q_rope_out, dev_error)
    B, T, row, max_pos, H, qt, qh, q_rope_out = _write_args(cache_lens, kv, positions, rope_table, kv_weight, cu_seqlens,
                                                            B, q_rope_in, q_rope_out, stream)
    sc, sr, M, N = _pages(c_pages, r_pages, page_table, page_size, B)
    _call_kv_norm_rope_write_paged(c_pages.data_ptr(), r_pages.data_ptr(), sc, sr, int(page_size),
        page_table.data_ptr(), M, N, cache_lens.data_ptr(), kv.data_ptr(), row, _addr(kv_weight), eps,
        rope_table.data_ptr(), max_pos, _addr(positions), interleaved, _addr(cu_seqlens), B, T, _addr(q_rope_in), qt,
        qh, H, _addr(q_rope_out), _addr(dev_error), _stream_of(stream, dev))
    return q_rope_out


def kd_prompt_attn(q_nope, k_nope, v, cu_seqlens_q, q_rope=None, k_rope=None, cu_seqlens_k=None, scale=None, out=None,
                   lse=None, dev_error=None, stream=None):
    """Causal attention of packed prompts: q_nope [T][H][128], k_nope and v [Tk][Hk][128], and
    with a rope part q_rope [T][H][64] and k_rope [Tk][Hk][64] (or [Tk][64]: one for all
    heads), any token and head strides; sequence b is rows cu_seqlens_q[b] .. [b + 1] of the
    queries and of the keys (cu_seqlens_k when those differ: the queries are the last
    positions).  scale None: 1 / sqrt(192) with a rope part, else 1 / sqrt(128).
    Returns (out [T][H][128] bf16, lse [T][H] fp32), allocated unless given (not cleared: rows
    behind the last sequence, and all with bad lengths, hold what was in memory)."""
    dev = _on_device(q_nope, k_nope, v, cu_seqlens_q, q_rope, k_rope, cu_seqlens_k, out, lse, dev_error)
    T, H, _, qnt, qnh = _heads(q_nope, "q_nope", None, None, 128)
    Tk, Hk, _, knt, knh = _heads(k_nope, "k_nope", None, None, 128)
    _, _, _, vt, vh = _heads(v, "v", Tk, Hk, 128)
    if (q_rope is None) != (k_rope is None):
        raise ValueError("q_rope and k_rope go together")
    qrt = qrh = krt = krh = 0
    if q_rope is not None:
        _, _, _, qrt, qrh = _heads(q_rope, "q_rope", T, H, D_R)
        if k_rope.dim() == 2:
            krt = _heads(k_rope.unsqueeze(1), "k_rope", Tk, 1, D_R)[3]
        else:
            _, _, _, krt, krh = _heads(k_rope, "k_rope", Tk, Hk, D_R)
    _typed(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    if cu_seqlens_q.dim() != 1 or cu_seqlens_q.shape[0] < 2:
        raise ValueError("cu_seqlens_q must be [B + 1]")
    B = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k is not None:
        _typed(cu_seqlens_k, torch.int32, "cu_seqlens_k", (B + 1,))
    if scale is None:
        scale = 1.0 / math.sqrt(128.0 if q_rope is None else 192.0)
    if out is None:
        out = _new(stream, torch.empty, T, H, 128, dtype=torch.bfloat16, device=q_nope.device)
    if lse is None:
        lse = _new(stream, torch.empty, T, H, dtype=torch.float32, device=q_nope.device)
    _typed(out, torch.bfloat16, "out", (T, H, 128))
    _typed(lse, torch.float32, "lse", (T, H))
    _call_prompt_attn(q_nope.data_ptr(), qnt, qnh, _addr(q_rope), qrt, qrh, k_nope.data_ptr(), knt, knh,
        _addr(k_rope), krt, krh, v.data_ptr(), vt, vh, cu_seqlens_q.data_ptr(), _addr(cu_seqlens_k), B, T, Tk, H, Hk,
        scale, out.data_ptr(), lse.data_ptr(), _addr(dev_error), _stream_of(stream, dev))
    return out, lse


def _weight_rows(w, B, cap, name):
    if w.dtype is not torch.float32 or w.dim() != 2 or w.shape[0] != B or w.shape[1] < cap or w.stride(1) != 1:
        raise ValueError(f"{name} must be fp32 [{B}][at least {cap}] with unit-stride rows")
    return w.stride(0) if B > 1 else max(w.stride(0), w.shape[1])


def _weights_args(q_abs, q_rope, cache_lens, vis, lse, path, length, weights_in, weights_out, cap, stream):
    _typed(q_abs, torch.bfloat16, "q_abs")
    if q_abs.dim() != 4 or q_abs.shape[3] != D_C:
        raise ValueError("q_abs must be [B][n][H][512]")
    B, n, H, _ = q_abs.shape
    _typed(q_rope, torch.bfloat16, "q_rope", (B, n, H, D_R))
    _typed(cache_lens, torch.int32, "cache_lens", (B,))
    if (vis.dtype is not torch.int32 and vis.dtype is not torch.uint32) or not vis.is_contiguous() or \
            vis.shape != (B, n, (n + 31) // 32):
        raise ValueError("vis must be contiguous int32 or uint32 [B][n][ceil(n / 32)]")
    _typed(lse, torch.float32, "lse", (B, n, H))
    if (path is None) != (length is None):
        raise ValueError("path and length go together")
    if path is not None:
        _typed(path, torch.int32, "path", (B, n))
        _typed(length, torch.int32, "length", (B,))
    if weights_out is None:
        weights_out = _new(stream, torch.zeros, B, cap, dtype=torch.float32, device=q_abs.device)
    wi = _weight_rows(weights_in, B, cap, "weights_in") if weights_in is not None else 0
    return B, n, H, wi, _weight_rows(weights_out, B, cap, "weights_out"), weights_out


def kd_kv_attn_weights(q_abs, q_rope, c_kv, k_rope, cache_lens, vis, lse, path=None, length=None,
                       scale=1.0 / math.sqrt(192.0), weights_in=None, weights_out=None, dev_error=None, stream=None):
    """Attention weight each cache slot receives from the accepted nodes (path, length of
    kd_tree_accept; None: every node), added to weights_in [B][>= cap] fp32 (None: zeros).
    lse is kd_tree_verify_attn's.  Call it before kd_kv_compact: the new slots' weights are
    stored in compacted order.  Returns weights_out (weights_out=weights_in accumulates)."""
    dev = _on_device(q_abs, q_rope, c_kv, k_rope, cache_lens, vis, lse, path, length, weights_in, weights_out, dev_error)
    rows, sc, sr, cap = _cache(c_kv, k_rope)
    B, n, H, wi, wo, weights_out = _weights_args(q_abs, q_rope, cache_lens, vis, lse, path, length, weights_in,
                                                 weights_out, cap, stream)
    if rows != B:
        raise ValueError("the cache must hold B requests")
    _call_kv_attn_weights(q_abs.data_ptr(), q_rope.data_ptr(), c_kv.data_ptr(), k_rope.data_ptr(), sc, sr, cap,
        cache_lens.data_ptr(), vis.data_ptr(), lse.data_ptr(), _addr(path), _addr(length), B, n, H, scale,
        _addr(weights_in), wi, weights_out.data_ptr(), wo, _addr(dev_error), _stream_of(stream, dev))
    return weights_out


def kd_kv_attn_weights_paged(q_abs, q_rope, c_pages, r_pages, page_table, page_size, cache_lens, vis, lse, path=None,
                             length=None, scale=1.0 / math.sqrt(192.0), weights_in=None, weights_out=None,
                             dev_error=None, stream=None):
    """kd_kv_attn_weights over a paged cache (page_size 64, 128 or 256)."""
    dev = _on_device(q_abs, q_rope, c_pages, r_pages, page_table, cache_lens, vis, lse, path, length, weights_in,
               weights_out, dev_error)
    sc, sr, M, N = _pages(c_pages, r_pages, page_table, page_size, cache_lens.shape[0])
    B, n, H, wi, wo, weights_out = _weights_args(q_abs, q_rope, cache_lens, vis, lse, path, length, weights_in,
                                                 weights_out, M * page_size, stream)
    _call_kv_attn_weights_paged(q_abs.data_ptr(), q_rope.data_ptr(), c_pages.data_ptr(), r_pages.data_ptr(), sc, sr,
        int(page_size), page_table.data_ptr(), M, N, cache_lens.data_ptr(), vis.data_ptr(), lse.data_ptr(),
        _addr(path), _addr(length), B, n, H, scale, _addr(weights_in), wi, weights_out.data_ptr(), wo,
        _addr(dev_error), _stream_of(stream, dev))
    return weights_out


def _evict_args(cache_lens, weights_in, cap, dst_cap, keep, inplace, weights_out, lens_out, kept, stream):
    _typed(cache_lens, torch.int32, "cache_lens")
    B, dev = cache_lens.shape[0], cache_lens.device
    wi = _weight_rows(weights_in, B, cap, "weights_in")
    rows = min(dst_cap, max(int(keep), 1))
    if weights_out is None:
        weights_out = weights_in if inplace else _new(stream, torch.zeros, B, dst_cap, dtype=torch.float32, device=dev)
    wo = _weight_rows(weights_out, B, rows, "weights_out")
    if lens_out is None:
        # (zeros: a request that fails is not written, and holds nothing at its destination)
        lens_out = cache_lens if inplace else _new(stream, torch.zeros, B, dtype=torch.int32, device=dev)
    _typed(lens_out, torch.int32, "lens_out", (B,))
    if kept is None:
        kept = _new(stream, torch.empty, B, max(int(keep), 1), dtype=torch.int32, device=dev)
    _typed(kept, torch.int32, "kept", (B, max(int(keep), 1)))
    return B, wi, wo, weights_out, lens_out, kept


def kd_kv_evict(c_kv, k_rope, cache_lens, weights_in, keep, sink=0, recent=0, c_dst=None, r_dst=None,
                weights_out=None, lens_out=None, kept=None, dev_error=None, stream=None):
    """Cuts every request's cache to at most `keep` slots: its first `sink`, its last `recent`
    and those of the largest weights between.  Without c_dst, r_dst it works in place (cache,
    cache_lens and weights_in are updated); with them the kept rows go to another cache.
    Returns (kept [B][keep] int32, weights_out, lens_out); in another cache the length of a
    request that fails is 0 (one given is left as it was)."""
    dev = _on_device(c_kv, k_rope, cache_lens, weights_in, c_dst, r_dst, weights_out, lens_out, kept, dev_error)
    rows, sc, sr, cap = _cache(c_kv, k_rope)
    if (c_dst is None) != (r_dst is None):
        raise ValueError("c_dst and r_dst go together")
    inplace = c_dst is None
    if inplace:
        c_dst, r_dst = c_kv, k_rope
    drows, dc, dr, dcap = _cache(c_dst, r_dst)
    B, wi, wo, weights_out, lens_out, kept = _evict_args(cache_lens, weights_in, cap, dcap, keep, inplace, weights_out,
                                                         lens_out, kept, stream)
    if rows != B or drows != B:
        raise ValueError("the caches must hold B requests")
    _call_kv_evict(c_kv.data_ptr(), k_rope.data_ptr(), sc, sr, cap, cache_lens.data_ptr(), weights_in.data_ptr(), wi,
        int(keep), int(sink), int(recent), B, c_dst.data_ptr(), r_dst.data_ptr(), dc, dr, dcap,
        weights_out.data_ptr(), wo, lens_out.data_ptr(), kept.data_ptr(), _addr(dev_error), _stream_of(stream, dev))
    return kept, weights_out, lens_out


def kd_kv_evict_paged(c_pages, r_pages, page_table, page_size, cache_lens, weights_in, keep, sink=0, recent=0,
                      c_dst=None, r_dst=None, dst_page_table=None, weights_out=None, lens_out=None, kept=None,
                      dev_error=None, stream=None):
    """kd_kv_evict through page tables: in place without dst_page_table (the request's tail
    pages are then free), else into the pages of dst_page_table (of c_dst, r_dst, or of the
    same pool), which must be none of the source's.  Requests that share pages (a common prefix)
    are evicted into pages of their own, not in place."""
    dev = _on_device(c_pages, r_pages, page_table, cache_lens, weights_in, c_dst, r_dst, dst_page_table, weights_out,
               lens_out, kept, dev_error)
    sc, sr, M, N = _pages(c_pages, r_pages, page_table, page_size, cache_lens.shape[0])
    if (c_dst is None) != (r_dst is None) or (c_dst is not None and dst_page_table is None):
        raise ValueError("c_dst, r_dst and dst_page_table go together")
    inplace = dst_page_table is None
    if inplace:
        dst_page_table = page_table
    if c_dst is None:
        c_dst, r_dst = c_pages, r_pages
    dc, dr, DM, DN = _pages(c_dst, r_dst, dst_page_table, page_size, cache_lens.shape[0])
    B, wi, wo, weights_out, lens_out, kept = _evict_args(cache_lens, weights_in, M * page_size, DM * page_size, keep,
                                                         inplace, weights_out, lens_out, kept, stream)
    _call_kv_evict_paged(c_pages.data_ptr(), r_pages.data_ptr(), sc, sr, int(page_size), page_table.data_ptr(), M, N,
        cache_lens.data_ptr(), weights_in.data_ptr(), wi, int(keep), int(sink), int(recent), B, c_dst.data_ptr(),
        r_dst.data_ptr(), dc, dr, dst_page_table.data_ptr(), DM, DN, weights_out.data_ptr(), wo, lens_out.data_ptr(),
        kept.data_ptr(), _addr(dev_error), _stream_of(stream, dev))
    return kept, weights_out, lens_out


def kd_read_device_error(word, clear=True, stream=None) -> int:
    """Device error bits from an error word or a verify workspace (its first int32)."""
    rc = lib.kd_read_device_error(_ptr(word), int(bool(clear)), _stream(stream))
    if rc < 0:
        _check(rc, "kd_read_device_error")
    return rc


def decode_device_error(bits: int) -> list:
    return [name for bit, name in KD_DEV_BITS.items() if bits & bit]


# ------------------------------------------------------------------ host <-> device helpers
def bf16_from_bits(u16, device="cuda") -> torch.Tensor:
    """numpy uint16 bf16 bit patterns -> bf16 tensor on ``device``."""
    import numpy as np
    t = torch.from_numpy(np.ascontiguousarray(u16).view(np.int16))
    return t.to(device).view(torch.bfloat16)


def bits_from_bf16(t: torch.Tensor):
    """bf16 tensor -> numpy uint16 bit patterns (on the host)."""
    import numpy as np
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
