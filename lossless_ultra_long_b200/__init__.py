"""B200-native TokenSwift verification path: thin ctypes binding of libtsverify.so.

The three calls mirror the C ABI in ``include/ts_verify.h``; every step of
the path runs in the library's CUDA kernels.  This module only checks
tensor dtypes/devices, passes raw pointers and the current CUDA stream, and
turns non-zero status codes into exceptions.  torch supplies device memory
and streams.  There is no CPU fallback: if the library is not built, every
call raises.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtsverify.so")

TS_MAX_TREE = 64
STATUS = {0: "TS_OK", 1: "TS_ERR_INVALID_ARG", 2: "TS_ERR_UNSUPPORTED", 3: "TS_ERR_WORKSPACE",
          4: "TS_ERR_CUDA", 5: "TS_ERR_TIMEOUT", 6: "TS_ERR_DEVICE_ARG"}

EXPORTS = ("ts_status_string", "ts_version", "ts_tree_verify_attn_workspace_size",
           "ts_tree_verify_attn", "ts_kv_importance_select_workspace_size",
           "ts_kv_importance_select", "ts_penalize_accept_workspace_size", "ts_penalize_accept",
           "ts_workspace_status", "ts_kernel_launch_count", "ts_tree_verify_attn_root_scores",
           "ts_kv_select_from_scores_workspace_size", "ts_kv_select_from_scores",
           "ts_ngram_table_bytes", "ts_ngram_init", "ts_ngram_update", "ts_ngram_topk",
           "ts_ngram_topk_prefix",
           "ts_ngram_count", "ts_ngram_size", "ts_selftest_bounded_wait",
           "ts_penalize_accept_ex", "ts_penalize_sample_accept", "ts_kv_commit_path",
           "ts_kv_quantize_q8", "ts_tree_verify_attn_q8_workspace_size",
           "ts_tree_verify_attn_q8", "ts_kv_gather_q8", "ts_kv_select_from_scores_q8",
           "ts_rope_append", "ts_rope_inv_freq")

TS_Q8_BLOCK = 64
ROPE_KINDS = {"plain": 0, "linear": 1, "wavelength": 2, "yarn": 3}

TS_PENALIZE_PATH_TOKENS = 1
TS_ACCEPT_RANDOM_TIE = 2


class _Q8Cache(ctypes.Structure):
    """``ts_q8_cache``."""
    _fields_ = [("k8", ctypes.c_void_p), ("v8", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("q8_cap", ctypes.c_int64),
                ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p),
                ("tail_cap", ctypes.c_int64), ("tail_row0", ctypes.c_int64),
                ("n_heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("n_q8", ctypes.c_int), ("n_tail", ctypes.c_int)]


class TsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} "
                         f"({_lib().ts_status_string(status).decode()})")


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtsverify.so is not built ({LIB_PATH}); run "
                               "`python -m lossless_ultra_long_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                ctypes.c_size_t)
        lib.ts_status_string.restype = ctypes.c_char_p
        lib.ts_status_string.argtypes = [i32]
        lib.ts_version.restype = i32
        lib.ts_tree_verify_attn_workspace_size.restype = sz
        lib.ts_tree_verify_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.ts_tree_verify_attn.restype = i32
        lib.ts_tree_verify_attn.argtypes = [P, P, P, i64, i32, i32, i32, i32, i32, P, f32, P, P,
                                            sz, P]
        lib.ts_tree_verify_attn_root_scores.restype = i32
        lib.ts_tree_verify_attn_root_scores.argtypes = [P, P, P, i64, i32, i32, i32, i32, i32, P,
                                                        f32, P, P, P, sz, P]
        lib.ts_kv_select_from_scores_workspace_size.restype = sz
        lib.ts_kv_select_from_scores_workspace_size.argtypes = [i32, i32, i32]
        lib.ts_kv_select_from_scores.restype = i32
        lib.ts_kv_select_from_scores.argtypes = [P, P, P, i64, i32, i32, i32, i32, i32, i32, P, P,
                                                 P, P, i64, P, sz, P]
        lib.ts_kv_importance_select_workspace_size.restype = sz
        lib.ts_kv_importance_select_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.ts_kv_importance_select.restype = i32
        lib.ts_kv_importance_select.argtypes = [P, P, P, i64, i32, i32, i32, i32, i32, i32, f32,
                                                P, P, P, P, i64, P, sz, P]
        lib.ts_penalize_accept_workspace_size.restype = sz
        lib.ts_penalize_accept_workspace_size.argtypes = [i32, i32]
        lib.ts_penalize_accept.restype = i32
        lib.ts_penalize_accept.argtypes = [P, i32, i32, P, i32, f32, P, P, P, P, P, sz, P]
        lib.ts_penalize_accept_ex.restype = i32
        lib.ts_penalize_accept_ex.argtypes = [P, i32, i32, P, i32, f32, P, P, ctypes.c_uint,
                                              ctypes.c_uint64, P, P, P, sz, P]
        lib.ts_penalize_sample_accept.restype = i32
        lib.ts_penalize_sample_accept.argtypes = [P, P, f32, i32, i32, P, i32, f32, P, P,
                                                  ctypes.c_uint, ctypes.c_uint64, P, P, P, sz, P]
        lib.ts_kv_commit_path.restype = i32
        lib.ts_kv_commit_path.argtypes = [P, P, i64, i32, i32, i32, i32, P, P, sz, P]
        lib.ts_kv_quantize_q8.restype = i32
        lib.ts_kv_quantize_q8.argtypes = [P, P, i64, i32, i32, i64, i32, P, P, P, P, i64, i64, P]
        lib.ts_tree_verify_attn_q8_workspace_size.restype = sz
        lib.ts_tree_verify_attn_q8_workspace_size.argtypes = [i32] * 6
        lib.ts_tree_verify_attn_q8.restype = i32
        lib.ts_tree_verify_attn_q8.argtypes = [P, P, i32, i32, P, f32, P, P, P, sz, P]
        lib.ts_kv_gather_q8.restype = i32
        lib.ts_kv_gather_q8.argtypes = [P, P, i32, P, P, i64, P, sz, P]
        lib.ts_kv_select_from_scores_q8.restype = i32
        lib.ts_kv_select_from_scores_q8.argtypes = [P, P, i32, i32, i32, P, P, P, P, i64, P, sz, P]
        lib.ts_rope_append.restype = i32
        lib.ts_rope_append.argtypes = [P, i64, P, i64, P, i64, i32, i32, i32, i32, P, i64, P, i32,
                                       i32, f32, P, P, P, i64, i64, P]
        lib.ts_rope_inv_freq.restype = i32
        lib.ts_rope_inv_freq.argtypes = [P, i32, ctypes.c_double, i32, P, P]
        lib.ts_kernel_launch_count.restype = ctypes.c_ulonglong
        lib.ts_kernel_launch_count.argtypes = []
        lib.ts_workspace_status.restype = i32
        lib.ts_workspace_status.argtypes = [P, P, i32]
        lib.ts_selftest_bounded_wait.restype = i32
        lib.ts_selftest_bounded_wait.argtypes = [P, sz, P]
        lib.ts_ngram_table_bytes.restype = sz
        lib.ts_ngram_table_bytes.argtypes = [i32, i64]
        lib.ts_ngram_init.restype = i32
        lib.ts_ngram_init.argtypes = [P, sz, i32, i64]
        lib.ts_ngram_update.restype = i32
        lib.ts_ngram_update.argtypes = [P, sz, P, i64, i64]
        lib.ts_ngram_topk.restype = i32
        lib.ts_ngram_topk.argtypes = [P, sz, ctypes.c_int32, i32, P, P, P]
        lib.ts_ngram_topk_prefix.restype = i32
        lib.ts_ngram_topk_prefix.argtypes = [P, sz, P, i32, i32, P, P, P]
        lib.ts_ngram_count.restype = i32
        lib.ts_ngram_count.argtypes = [P, sz, P, P]
        lib.ts_ngram_size.restype = i32
        lib.ts_ngram_size.argtypes = [P, sz, P, P]
        _LIB = lib
    return _LIB


def library():
    """The loaded ctypes handle (raises if the library is not built)."""
    return _lib()


def _ptr(t):
    return None if t is None else t.data_ptr()


_Tensor, _BF16, _I32 = torch.Tensor, torch.bfloat16, torch.int32

# the current stream's handle without a Stream object around it (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None):
    """A stream's handle; without one, the current stream's of ``device`` (the
    current device where that is None)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device is None else device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _check_dev(name, t, dtype, device=None):
    # what every right call passes, in one test (checks are most of its host time)
    if (type(t) is _Tensor and t.dtype is dtype and t.is_contiguous() and
            (t.is_cuda if device is None else t.device == device and t.is_cuda)):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")


def _call_device(name, t):
    """The device a call runs on: that of its first tensor, which must be the
    current CUDA device (the kernels launch there, on its current stream)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{cur}")
    return t.device


def _ws_bytes(workspace, device):
    """Size in bytes of a workspace, after checking that it is a contiguous
    CUDA tensor on the call's device."""
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, the call's tensors on {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.nbytes


def _host_i32(a):
    import numpy as np
    arr = np.ascontiguousarray(a.cpu().numpy() if isinstance(a, torch.Tensor) else a,
                               dtype=np.int32)
    return arr, arr.ctypes.data_as(ctypes.c_void_p)


# one past the C ABI's integers (ctypes would cut what lies outside)
_C_INT, _C_INT64 = 1 << 31, 1 << 63


def _parent_arg(parent, n):
    """(keep-alive, address) of a host int32 parent array of n entries."""
    if type(parent) is list:
        try:   # a third of numpy's time for a list of integers
            ints = array.array("i", parent)
            if len(ints) != n:
                raise ValueError("parent must have one entry per tree node")
            return ints, ints.buffer_info()[0]
        except (TypeError, OverflowError):
            pass
    import numpy as np
    if isinstance(parent, torch.Tensor):
        parent = parent.cpu().numpy()
    arr = np.asarray(parent)
    if arr.shape != (n,):
        raise ValueError("parent must have one entry per tree node")
    if arr.dtype != np.int32:
        with np.errstate(invalid="ignore"):
            ints = arr.astype(np.int32)
        if not (ints == arr).all():
            raise ValueError("parent must hold 32-bit integers")
        arr = ints
    arr = np.ascontiguousarray(arr)
    return arr, arr.__array_interface__["data"][0]


def _raise(rc, where):
    if rc != 0:
        raise TsError(rc, where)


def _on(stream):
    """The context of a stream, which need not be torch's own kind: any object with
    its handle, as the calls take."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


# A call's own buffers are made on the stream that it runs on: a workspace's
# zeros are there before the kernel reads them, and memory that is freed when
# the call returns goes to what this stream runs next, not to another's work.
def new_workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """A zero-filled uint8 device buffer (torch allocations are 512-byte
    aligned), made on ``stream`` (None: the current one), behind which a call
    on another stream has to be ordered."""
    if stream is not None:
        with _on(stream):
            return new_workspace(nbytes, device)
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def _empty(shape, dtype, device, stream):
    if stream is not None:
        with _on(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


# ----------------------------------------------------------- attention
def tree_verify_attn_workspace_size(n_heads_q, n_heads_kv, head_dim, n_ctx, n_tree) -> int:
    return int(_lib().ts_tree_verify_attn_workspace_size(n_heads_q, n_heads_kv, head_dim, n_ctx,
                                                         n_tree))


def tree_verify_attn(q, k_cache, v_cache, n_ctx: int, parent, out=None, workspace=None,
                     softmax_scale: float | None = None, stream=None, root_scores_out=None):
    """Tree-masked attention (``ts_tree_verify_attn``).

    q: bf16 [T, Hq, D]; k_cache, v_cache: bf16 [Hkv, kv_cap, D]; parent: host
    int32 [T].  Returns fp32 [T, Hq, D].  With ``root_scores_out`` (fp32
    [Hq, n_ctx]) it also leaves the root node's base-2 scores over the
    context (``ts_tree_verify_attn_root_scores``), the input of
    :func:`kv_select_from_scores`.
    """
    _check_dev("q", q, torch.bfloat16)
    dev = _call_device("q", q)
    _check_dev("k_cache", k_cache, torch.bfloat16, dev)
    _check_dev("v_cache", v_cache, torch.bfloat16, dev)
    t, hq, d = q.shape
    hkv, cap, d2 = k_cache.shape
    if v_cache.shape != k_cache.shape or d2 != d:
        raise ValueError("k_cache / v_cache / q shapes disagree")
    if out is None:
        out = _empty((t, hq, d), torch.float32, dev, stream)
    _check_dev("out", out, torch.float32, dev)
    if workspace is None:
        workspace = new_workspace(tree_verify_attn_workspace_size(hq, hkv, d, n_ctx, t), dev, stream)
    par, par_p = _host_i32(parent)
    if len(par) != t:
        raise ValueError("parent must have one entry per tree node")
    scale = float(d) ** -0.5 if softmax_scale is None else float(softmax_scale)
    ws_bytes = _ws_bytes(workspace, dev)
    if root_scores_out is None:
        rc = _lib().ts_tree_verify_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), cap, hq, hkv, d,
                                        int(n_ctx), t, par_p, scale, _ptr(out), _ptr(workspace),
                                        ws_bytes, _stream(stream))
        _raise(rc, "ts_tree_verify_attn")
        return out
    _check_dev("root_scores_out", root_scores_out, torch.float32, dev)
    if tuple(root_scores_out.shape) != (hq, int(n_ctx)):
        raise ValueError("root_scores_out must be [Hq, n_ctx]")
    rc = _lib().ts_tree_verify_attn_root_scores(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), cap, hq, hkv, d, int(n_ctx), t, par_p, scale,
        _ptr(out), _ptr(root_scores_out), _ptr(workspace), ws_bytes, _stream(stream))
    _raise(rc, "ts_tree_verify_attn_root_scores")
    return out


# ------------------------------------------------------------ selection
def kv_importance_select_workspace_size(n_heads_q, n_heads_kv, head_dim, n_ctx) -> int:
    return int(_lib().ts_kv_importance_select_workspace_size(n_heads_q, n_heads_kv, head_dim,
                                                             n_ctx))


def kv_importance_select(q_last, k_cache, v_cache, n_ctx: int, n_sink: int, budget: int,
                         k_partial=None, v_partial=None, idx_out=None, scores_out=None,
                         workspace=None, softmax_scale: float | None = None, stream=None,
                         want_scores: bool = False):
    """Sink + top-budget partial-KV update (``ts_kv_importance_select``).

    Returns ``(idx [Hkv, n_keep] int32, k_partial, v_partial, scores or None)``.
    """
    _check_dev("q_last", q_last, torch.bfloat16)
    dev = _call_device("q_last", q_last)
    _check_dev("k_cache", k_cache, torch.bfloat16, dev)
    _check_dev("v_cache", v_cache, torch.bfloat16, dev)
    hq, d = q_last.shape
    hkv, cap, d2 = k_cache.shape
    n_keep = min(n_ctx, n_sink + budget)
    if k_partial is None:
        k_partial = _empty((hkv, n_keep, d), torch.bfloat16, dev, stream)
    if v_partial is None:
        v_partial = _empty(k_partial.shape, _BF16, dev, stream)
    if idx_out is None:
        idx_out = _empty((hkv, n_keep), torch.int32, dev, stream)
    if want_scores and scores_out is None:
        scores_out = _empty((hkv, n_ctx), torch.float32, dev, stream)
    for name, t, dt in (("k_partial", k_partial, torch.bfloat16),
                        ("v_partial", v_partial, torch.bfloat16),
                        ("idx_out", idx_out, torch.int32)):
        _check_dev(name, t, dt, dev)
    if scores_out is not None:
        _check_dev("scores_out", scores_out, torch.float32, dev)
    if workspace is None:
        workspace = new_workspace(kv_importance_select_workspace_size(hq, hkv, d, n_ctx), dev, stream)
    scale = float(d) ** -0.5 if softmax_scale is None else float(softmax_scale)
    rc = _lib().ts_kv_importance_select(
        _ptr(q_last), _ptr(k_cache), _ptr(v_cache), cap, hq, hkv, d, int(n_ctx), int(n_sink),
        int(budget), scale, _ptr(scores_out), _ptr(idx_out), _ptr(k_partial), _ptr(v_partial),
        k_partial.shape[1], _ptr(workspace), _ws_bytes(workspace, dev), _stream(stream))
    _raise(rc, "ts_kv_importance_select")
    return idx_out, k_partial, v_partial, scores_out


def kv_select_from_scores_workspace_size(n_heads_q, n_heads_kv, n_ctx) -> int:
    return int(_lib().ts_kv_select_from_scores_workspace_size(n_heads_q, n_heads_kv, n_ctx))


def kv_select_from_scores(root_scores, k_cache, v_cache, n_ctx: int, n_sink: int, budget: int,
                          k_partial=None, v_partial=None, idx_out=None, scores_out=None,
                          workspace=None, stream=None, want_scores: bool = False):
    """The partial-KV update from root scores left by the verify attention
    (``ts_kv_select_from_scores``).  root_scores: fp32 [Hq, n_ctx] (base 2).

    Returns ``(idx [Hkv, n_keep] int32, k_partial, v_partial, scores or None)``.
    """
    _check_dev("root_scores", root_scores, torch.float32)
    dev = _call_device("root_scores", root_scores)
    _check_dev("k_cache", k_cache, torch.bfloat16, dev)
    _check_dev("v_cache", v_cache, torch.bfloat16, dev)
    hq, n = root_scores.shape
    if n != int(n_ctx):
        raise ValueError("root_scores must be [Hq, n_ctx]")
    hkv, cap, d = k_cache.shape
    n_keep = min(n_ctx, n_sink + budget)
    if k_partial is None:
        k_partial = _empty((hkv, n_keep, d), torch.bfloat16, dev, stream)
    if v_partial is None:
        v_partial = _empty(k_partial.shape, _BF16, dev, stream)
    if idx_out is None:
        idx_out = _empty((hkv, n_keep), torch.int32, dev, stream)
    if want_scores and scores_out is None:
        scores_out = _empty((hkv, n_ctx), torch.float32, dev, stream)
    for name, t, dt in (("k_partial", k_partial, torch.bfloat16),
                        ("v_partial", v_partial, torch.bfloat16),
                        ("idx_out", idx_out, torch.int32)):
        _check_dev(name, t, dt, dev)
    if scores_out is not None:
        _check_dev("scores_out", scores_out, torch.float32, dev)
    if workspace is None:
        workspace = new_workspace(kv_select_from_scores_workspace_size(hq, hkv, int(n_ctx)), dev, stream)
    rc = _lib().ts_kv_select_from_scores(
        _ptr(root_scores), _ptr(k_cache), _ptr(v_cache), cap, hq, hkv, d, int(n_ctx),
        int(n_sink), int(budget), _ptr(scores_out), _ptr(idx_out), _ptr(k_partial),
        _ptr(v_partial), k_partial.shape[1], _ptr(workspace), _ws_bytes(workspace, dev),
        _stream(stream))
    _raise(rc, "ts_kv_select_from_scores")
    return idx_out, k_partial, v_partial, scores_out


# ------------------------------------------------------ penalty + accept
def penalize_accept_workspace_size(n_tree, vocab) -> int:
    return int(_lib().ts_penalize_accept_workspace_size(n_tree, vocab))


def penalize_accept(logits, window, penalty: float, parent, tree_tokens, argmax_out=None,
                    accept_out=None, workspace=None, stream=None, want_argmax: bool = True,
                    flags: int = 0, random: int = 0):
    """Contextual penalty + per-node argmax + longest accepted path
    (``ts_penalize_accept``; with ``flags`` -- TS_PENALIZE_PATH_TOKENS,
    TS_ACCEPT_RANDOM_TIE -- ``ts_penalize_accept_ex``, ``random`` the
    caller's random 64-bit integer for the choice among the deepest valid
    nodes).

    Returns ``(accept [2 + T] int32, argmax [T] int32 or None)``.
    """
    _check_dev("logits", logits, torch.float32)
    dev = _call_device("logits", logits)
    _check_dev("tree_tokens", tree_tokens, torch.int32, dev)
    t, vocab = logits.shape
    if window is not None and window.numel() > 0:
        _check_dev("window", window, torch.int32, dev)
        wlen, wptr = window.numel(), _ptr(window)
    else:
        wlen, wptr = 0, None
    if accept_out is None:
        accept_out = _empty(2 + t, torch.int32, dev, stream)
    if want_argmax and argmax_out is None:
        argmax_out = _empty(t, torch.int32, dev, stream)
    _check_dev("accept_out", accept_out, torch.int32, dev)
    if argmax_out is not None:
        _check_dev("argmax_out", argmax_out, torch.int32, dev)
    if workspace is None:
        workspace = new_workspace(penalize_accept_workspace_size(t, vocab), dev, stream)
    par, par_p = _host_i32(parent)
    if len(par) != t:
        raise ValueError("parent must have one entry per tree node")
    if flags == 0:
        rc = _lib().ts_penalize_accept(_ptr(logits), t, vocab, wptr, wlen, float(penalty), par_p,
                                       _ptr(tree_tokens), _ptr(argmax_out), _ptr(accept_out),
                                       _ptr(workspace), _ws_bytes(workspace, dev),
                                       _stream(stream))
        _raise(rc, "ts_penalize_accept")
    else:
        rc = _lib().ts_penalize_accept_ex(
            _ptr(logits), t, vocab, wptr, wlen, float(penalty), par_p, _ptr(tree_tokens),
            int(flags), int(random) & (2 ** 64 - 1), _ptr(argmax_out), _ptr(accept_out),
            _ptr(workspace), _ws_bytes(workspace, dev), _stream(stream))
        _raise(rc, "ts_penalize_accept_ex")
    return accept_out, argmax_out


def penalize_sample_accept(logits, gumbel, temperature: float, window, penalty: float, parent,
                           tree_tokens, target_out=None, accept_out=None, workspace=None,
                           stream=None, want_target: bool = True, flags: int = 0,
                           random: int = 0):
    """Contextual penalty + per-node temperature draw + longest accepted path
    (``ts_penalize_sample_accept``): node i's target token is the id
    maximising penalised / temperature + gumbel[i] (binary32), the
    Gumbel-max draw from softmax(penalised / temperature); ``gumbel`` is the
    caller's standard Gumbel noise, fp32 ``[T, V]`` on the device.  ``flags``
    and ``random`` as for :func:`penalize_accept`.

    Returns ``(accept [2 + T] int32, target [T] int32 or None)``.
    """
    _check_dev("logits", logits, torch.float32)
    dev = _call_device("logits", logits)
    _check_dev("gumbel", gumbel, torch.float32, dev)
    _check_dev("tree_tokens", tree_tokens, torch.int32, dev)
    t, vocab = logits.shape
    if tuple(gumbel.shape) != (t, vocab):
        raise ValueError("gumbel must have the logits' shape [T, V]")
    if window is not None and window.numel() > 0:
        _check_dev("window", window, torch.int32, dev)
        wlen, wptr = window.numel(), _ptr(window)
    else:
        wlen, wptr = 0, None
    if accept_out is None:
        accept_out = _empty(2 + t, torch.int32, dev, stream)
    if want_target and target_out is None:
        target_out = _empty(t, torch.int32, dev, stream)
    _check_dev("accept_out", accept_out, torch.int32, dev)
    if target_out is not None:
        _check_dev("target_out", target_out, torch.int32, dev)
    if workspace is None:
        workspace = new_workspace(penalize_accept_workspace_size(t, vocab), dev, stream)
    par, par_p = _host_i32(parent)
    if len(par) != t:
        raise ValueError("parent must have one entry per tree node")
    rc = _lib().ts_penalize_sample_accept(
        _ptr(logits), _ptr(gumbel), float(temperature), t, vocab, wptr, wlen, float(penalty),
        par_p, _ptr(tree_tokens), int(flags), int(random) & (2 ** 64 - 1), _ptr(target_out),
        _ptr(accept_out), _ptr(workspace), _ws_bytes(workspace, dev), _stream(stream))
    _raise(rc, "ts_penalize_sample_accept")
    return accept_out, target_out


def kv_commit_path(k_cache, v_cache, n_ctx: int, n_tree: int, accept, workspace=None,
                   stream=None):
    """Moves the accepted path's tree rows to n_ctx + 0 .. n_ctx + L in both
    caches, in place (``ts_kv_commit_path``); ``accept`` is the device
    result of :func:`penalize_accept`."""
    _check_dev("k_cache", k_cache, torch.bfloat16)
    dev = _call_device("k_cache", k_cache)
    _check_dev("v_cache", v_cache, torch.bfloat16, dev)
    _check_dev("accept", accept, torch.int32, dev)
    hkv, cap, d = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache / v_cache shapes disagree")
    if workspace is None:
        workspace = new_workspace(256, dev, stream)
    rc = _lib().ts_kv_commit_path(_ptr(k_cache), _ptr(v_cache), cap, hkv, d, int(n_ctx),
                                  int(n_tree), _ptr(accept), _ptr(workspace),
                                  _ws_bytes(workspace, dev), _stream(stream))
    _raise(rc, "ts_kv_commit_path")
    return k_cache, v_cache


# ------------------------------------------------- rotation and the 8-bit cache
def rope_inv_freq(rot_dim: int, base: float, kind: str = "plain", *params):
    """Frequency table of a rotary embedding (``ts_rope_inv_freq``): ``(host
    fp32 [rot_dim / 2], mscale)``.  kind and params: "plain"; "linear",
    factor; "wavelength", factor, low, high, ctx; "yarn", factor, ctx, fast,
    slow."""
    import numpy as np
    if kind not in ROPE_KINDS:
        raise ValueError(f"kind must be one of {sorted(ROPE_KINDS)}")
    want = (0, 1, 4, 4)[ROPE_KINDS[kind]]
    if len(params) != want:
        raise ValueError(f"{kind!r} takes {want} parameters")
    out = np.zeros(max(int(rot_dim) // 2, 1), dtype=np.float32)
    par = np.asarray(params + (1.0,), dtype=np.float64)
    m = ctypes.c_float(0.0)
    _raise(_lib().ts_rope_inv_freq(out.ctypes.data_as(ctypes.c_void_p), int(rot_dim), float(base),
                                   ROPE_KINDS[kind], par.ctypes.data_as(ctypes.c_void_p),
                                   ctypes.byref(m)), "ts_rope_inv_freq")
    return torch.from_numpy(out[:int(rot_dim) // 2]), float(m.value)


def _check_rows(name, t, heads, d, device):
    """A bf16 [tokens, heads, D] tensor whose tokens may lie apart: the
    elements from one token to the next."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != d:
        raise ValueError(f"{name} must be [tokens, heads, {d}]")
    st = t.stride()
    if (st[2] != 1 and d > 1) or (st[1] != d and shape[1] > 1):
        raise ValueError(f"{name}: the heads and elements of a token must be contiguous")
    return st[0] if shape[0] > 1 else shape[1] * d


def rope_append(q, k, v, k_cache, v_cache, row0: int, pos0: int, inv_freq, parent=None,
                interleaved: bool = False, mscale: float = 1.0, q_out=None, stream=None):
    """Rotary embedding of q and k and the append of k and v to a bf16 cache
    (``ts_rope_append``).

    q: bf16 [n, Hq, D] or None; k, v: bf16 [n, Hkv, D] (slices of one
    projection's output serve); k_cache, v_cache: bf16 [Hkv, kv_cap, D], rows
    ``row0 ..`` written; inv_freq: fp32 [rot / 2] on the device, or None;
    parent: the draft tree (host int32 [n]; position pos0 + depth) or None
    (positions pos0 + i).  Returns the turned queries, bf16 [n, Hq, D].
    """
    dev = _call_device("k", k)
    _check_dev("k_cache", k_cache, _BF16, dev)
    _check_dev("v_cache", v_cache, _BF16, dev)
    if k_cache.dim() != 3 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [Hkv, kv_cap, D]")
    hkv, cap, d = k_cache.shape
    ks, vs = _check_rows("k", k, hkv, d, dev), _check_rows("v", v, hkv, d, dev)
    n = k.shape[0]
    hq = qs = 0
    if q is not None:
        qs, hq = _check_rows("q", q, None, d, dev), q.shape[1]
        if q_out is None:
            q_out = _empty((n, hq, d), _BF16, dev, stream)
        _check_dev("q_out", q_out, _BF16, dev)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    if v.shape[0] != n or (q is not None and q.shape[0] != n):
        raise ValueError("q, k and v must have as many tokens")
    rot = 0
    if inv_freq is not None:
        _check_dev("inv_freq", inv_freq, torch.float32, dev)
        rot = 2 * inv_freq.numel()
    par, par_p = (None, None) if parent is None else _parent_arg(parent, n)
    row0, pos0 = int(row0), int(pos0)
    if not (-_C_INT64 <= row0 < _C_INT64 and -_C_INT64 <= pos0 < _C_INT64):
        raise ValueError("row0 and pos0 must be signed 64-bit integers")
    _raise(_lib().ts_rope_append(
        _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, hq, hkv, d, n, par_p, pos0,
        _ptr(inv_freq) if rot else None, rot, int(bool(interleaved)), float(mscale),
        _ptr(q_out) if hq else None, _ptr(k_cache), _ptr(v_cache), cap, row0,
        _stream(stream, dev)), "ts_rope_append")
    return q_out


def _check_q8(k8, v8, k_scale, v_scale, device):
    _check_dev("k8", k8, torch.float8_e4m3fn, device)
    _check_dev("v8", v8, torch.float8_e4m3fn, device)
    _check_dev("k_scale", k_scale, torch.uint8, device)
    _check_dev("v_scale", v_scale, torch.uint8, device)
    if k8.dim() != 3 or v8.shape != k8.shape or k8.shape[1] % TS_Q8_BLOCK:
        raise ValueError(f"k8 and v8 must be [Hkv, rows, D], rows a multiple of {TS_Q8_BLOCK}")
    want = (k8.shape[0], k8.shape[1] // TS_Q8_BLOCK)
    if tuple(k_scale.shape) != want or tuple(v_scale.shape) != want:
        raise ValueError(f"k_scale and v_scale must be {want}")


def kv_quantize_q8(k, v, row0: int, n_rows: int, k8, v8, k_scale, v_scale, dst_row: int,
                   stream=None):
    """Rows [row0, row0 + n_rows) of bf16 k and v [Hkv, cap, D] into 8-bit rows
    [dst_row, dst_row + n_rows) and their blocks' scales
    (``ts_kv_quantize_q8``); n_rows and dst_row multiples of 64."""
    _check_dev("k", k, _BF16)
    dev = _call_device("k", k)
    _check_dev("v", v, _BF16, dev)
    _check_q8(k8, v8, k_scale, v_scale, dev)
    if k.dim() != 3 or v.shape != k.shape or k.shape[0] != k8.shape[0] or k.shape[2] != k8.shape[2]:
        raise ValueError("k / v / k8 / v8 shapes disagree")
    hkv, cap, d = k.shape
    row0, n_rows, dst_row = int(row0), int(n_rows), int(dst_row)
    if not (-_C_INT64 <= row0 < _C_INT64 and -_C_INT <= n_rows < _C_INT and -_C_INT64 <= dst_row < _C_INT64):
        raise ValueError("row0 and dst_row must be signed 64-bit integers, n_rows a 32-bit integer")
    _raise(_lib().ts_kv_quantize_q8(
        _ptr(k), _ptr(v), cap, hkv, d, row0, n_rows, _ptr(k8), _ptr(v8), _ptr(k_scale), _ptr(v_scale),
        k8.shape[1], dst_row, _stream(stream, dev)), "ts_kv_quantize_q8")
    return k8, v8, k_scale, v_scale


class KvCacheQ8:
    """An 8-bit KV cache (``ts_q8_cache``): ``n_q8`` context rows as e4m3
    blocks of 64, then ``n_tail`` rows (and the draft tree's) as bf16 in a
    tail that starts at row ``tail_row0`` of its buffer.  The tensors are the
    caller's, or :meth:`empty`'s.

    A step: :meth:`append` the tree's rows, :func:`tree_verify_attn_q8`,
    :meth:`commit` the accepted path, :meth:`fold` the blocks that are full.
    A prompt: :meth:`append` without a tree, then :meth:`fold`.
    """

    def __init__(self, k8, v8, k_scale, v_scale, k_tail, v_tail, n_q8: int = 0, n_tail: int = 0,
                 tail_row0: int = 0):
        dev = _call_device("k_tail", k_tail)
        _check_q8(k8, v8, k_scale, v_scale, dev)
        _check_dev("k_tail", k_tail, _BF16, dev)
        _check_dev("v_tail", v_tail, _BF16, dev)
        if (k_tail.dim() != 3 or v_tail.shape != k_tail.shape or
                k_tail.shape[0] != k8.shape[0] or k_tail.shape[2] != k8.shape[2]):
            raise ValueError("k_tail and v_tail must be [Hkv, rows, D] as k8")
        if not 0 <= n_q8 <= k8.shape[1] or n_q8 % TS_Q8_BLOCK:
            raise ValueError("n_q8 must be a multiple of 64 within the 8-bit rows")
        if n_tail < 0 or tail_row0 < 0 or tail_row0 + n_tail > k_tail.shape[1]:
            raise ValueError("n_tail rows from tail_row0 must lie in the tail")
        self._tensors = (k8, v8, k_scale, v_scale, k_tail, v_tail)   # the struct's, for good
        self.device = dev
        self.n_q8, self.n_tail, self.tail_row0 = int(n_q8), int(n_tail), int(tail_row0)
        hkv, cap, d = k8.shape
        self._struct = _Q8Cache(k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(),
                                v_scale.data_ptr(), cap, k_tail.data_ptr(), v_tail.data_ptr(),
                                k_tail.shape[1], self.tail_row0, hkv, d, self.n_q8, self.n_tail)

    k8 = property(lambda self: self._tensors[0])
    v8 = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])
    k_tail = property(lambda self: self._tensors[4])
    v_tail = property(lambda self: self._tensors[5])

    @classmethod
    def empty(cls, n_heads_kv: int, head_dim: int, capacity: int, tail_rows: int = 256,
              device=None):
        """An empty cache for ``capacity`` 8-bit rows (rounded up to 64), made on
        the current stream.  The tail takes a step's tree, or a prompt's chunk,
        behind the up to 63 rows that :meth:`fold` leaves."""
        device = "cuda" if device is None else device
        cap = -(-int(capacity) // TS_Q8_BLOCK) * TS_Q8_BLOCK

        def new(rows, dtype):
            return torch.zeros((n_heads_kv, rows, head_dim), dtype=torch.uint8 if dtype is None
                               else dtype, device=device)

        scales = [torch.zeros((n_heads_kv, cap // TS_Q8_BLOCK), dtype=torch.uint8, device=device)
                  for _ in range(2)]
        return cls(new(cap, None).view(torch.float8_e4m3fn), new(cap, None).view(torch.float8_e4m3fn),
                   *scales, new(int(tail_rows), _BF16), new(int(tail_rows), _BF16))

    @property
    def n_ctx(self) -> int:
        return self.n_q8 + self.n_tail

    def struct(self):
        """The ``ts_q8_cache`` of the cache as it stands."""
        st = self._struct
        st.n_q8, st.n_tail, st.tail_row0 = self.n_q8, self.n_tail, self.tail_row0
        return st

    def append(self, q, k, v, inv_freq, parent=None, stream=None, **kw):
        """:func:`rope_append` behind the context, at its positions.  With
        ``parent`` the rows are a draft tree's and wait for :meth:`commit`;
        without, they are context at once.  Returns the turned queries."""
        out = rope_append(q, k, v, self.k_tail, self.v_tail, self.tail_row0 + self.n_tail,
                          self.n_ctx, inv_freq, parent=parent, stream=stream, **kw)
        if parent is None:
            self.n_tail += k.shape[0]
        return out

    def commit(self, accept, n_tree: int, n_accepted: int, workspace=None, stream=None) -> None:
        """Keeps the root's row and the accepted path's (``ts_kv_commit_path``
        on the tail).  ``accept``: the device result of
        :func:`penalize_accept`; ``n_accepted``: its path length, read by the
        caller."""
        if not 0 <= int(n_accepted) < int(n_tree):
            raise ValueError("n_accepted must lie in [0, n_tree)")
        _check_dev("accept", accept, _I32, self.device)
        if accept.numel() < 2 + int(n_tree):     # the kernel goes by the length it finds there
            raise ValueError("accept must hold 2 + n_tree entries")
        dev = _call_device("k_tail", self.k_tail)
        if workspace is None:
            workspace = new_workspace(256, dev, stream)
        hkv, cap, d = self.k_tail.shape
        if self.tail_row0 + self.n_tail + int(n_tree) > cap:
            raise ValueError("the tree's rows do not lie in the tail")
        off = 2 * d * self.tail_row0
        _raise(_lib().ts_kv_commit_path(
            ctypes.c_void_p(self.k_tail.data_ptr() + off),
            ctypes.c_void_p(self.v_tail.data_ptr() + off), cap, hkv, d, self.n_tail, int(n_tree),
            _ptr(accept), _ptr(workspace), _ws_bytes(workspace, dev), _stream(stream, dev)),
            "ts_kv_commit_path")
        self.n_tail += int(n_accepted) + 1

    def fold(self, stream=None) -> int:
        """Turns the tail's full blocks into 8 bits and moves the rows that are
        left (fewer than 64) to its start.  Returns the rows folded."""
        rows = self.n_tail // TS_Q8_BLOCK * TS_Q8_BLOCK
        if rows:
            kv_quantize_q8(self.k_tail, self.v_tail, self.tail_row0, rows, self.k8, self.v8,
                           self.k_scale, self.v_scale, self.n_q8, stream=stream)
            self.n_q8 += rows
            self.n_tail -= rows
            self.tail_row0 += rows
        if self.tail_row0:
            _call_device("k_tail", self.k_tail)
            n, at = self.n_tail, self.tail_row0
            with contextlib.nullcontext() if stream is None else _on(stream):
                for t in (self.k_tail, self.v_tail) if n else ():
                    left = t[:, at:at + n]
                    t[:, :n].copy_(left if at >= n else left.clone())
            self.tail_row0 = 0
        return rows


def _call_cache(cache):
    if not isinstance(cache, KvCacheQ8):
        raise ValueError("cache must be a KvCacheQ8")
    cur = torch.cuda.current_device()
    if cache.device.index != cur:
        raise ValueError(f"cache is on {cache.device} but the current device is cuda:{cur}")
    return cache.device, cache.struct()


def tree_verify_attn_q8_workspace_size(n_heads_q, n_heads_kv, head_dim, n_q8, n_tail,
                                       n_tree) -> int:
    return int(_lib().ts_tree_verify_attn_q8_workspace_size(n_heads_q, n_heads_kv, head_dim, n_q8,
                                                            n_tail, n_tree))


def tree_verify_attn_q8(q, cache: KvCacheQ8, parent, out=None, workspace=None,
                        softmax_scale: float | None = None, stream=None, root_scores_out=None):
    """Tree-masked attention over an 8-bit cache (``ts_tree_verify_attn_q8``);
    the tree's rows lie in the tail behind the context.  q: bf16 [T, Hq, D];
    returns bf16 [T, Hq, D].  ``root_scores_out``: fp32 [Hq, n_ctx], as for
    :func:`tree_verify_attn`.  A workspace that is kept serves this function
    alone: it has to come back as the last call of it left it."""
    _check_dev("q", q, _BF16)
    dev, st = _call_cache(cache)
    if q.device != dev:
        raise ValueError(f"q is on {q.device}, the call's other tensors on {dev}")
    t, hq, d = q.shape
    if d != st.head_dim:
        raise ValueError("q and the cache must have the same head_dim")
    if out is None:
        out = _empty((t, hq, d), _BF16, dev, stream)
    _check_dev("out", out, _BF16, dev)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if root_scores_out is not None:
        _check_dev("root_scores_out", root_scores_out, torch.float32, dev)
        if tuple(root_scores_out.shape) != (hq, cache.n_ctx):
            raise ValueError("root_scores_out must be [Hq, n_ctx]")
    if workspace is None:
        workspace = new_workspace(tree_verify_attn_q8_workspace_size(
            hq, st.n_heads_kv, d, st.n_q8, st.n_tail, t), dev, stream)
    par, par_p = _parent_arg(parent, t)
    scale = float(d) ** -0.5 if softmax_scale is None else float(softmax_scale)
    rc = _lib().ts_tree_verify_attn_q8(
        ctypes.byref(st), _ptr(q), hq, t, par_p, scale, _ptr(out), _ptr(root_scores_out),
        _ptr(workspace), _ws_bytes(workspace, dev), _stream(stream, dev))
    _raise(rc, "ts_tree_verify_attn_q8")
    return out


def _q8_partials(cache, n_keep, k_partial, v_partial, dev, stream):
    hkv, _, d = cache.k8.shape
    if k_partial is None:
        k_partial = _empty((hkv, n_keep, d), _BF16, dev, stream)
    if v_partial is None:
        v_partial = _empty(k_partial.shape, _BF16, dev, stream)
    _check_dev("k_partial", k_partial, _BF16, dev)
    _check_dev("v_partial", v_partial, _BF16, dev)
    if (k_partial.dim() != 3 or k_partial.shape[0] != hkv or k_partial.shape[2] != d or
            v_partial.shape != k_partial.shape):
        raise ValueError("k_partial and v_partial must be [Hkv, rows, D]")
    return k_partial, v_partial


def kv_gather_q8(cache: KvCacheQ8, idx, k_partial=None, v_partial=None, workspace=None,
                 stream=None):
    """Context rows ``idx`` (int32 [Hkv, n_keep]) of an 8-bit cache as bf16 rows
    (``ts_kv_gather_q8``).  Returns ``(k_partial, v_partial)``."""
    dev, st = _call_cache(cache)
    _check_dev("idx", idx, _I32, dev)
    if idx.dim() != 2 or idx.shape[0] != st.n_heads_kv:
        raise ValueError("idx must be [Hkv, n_keep]")
    k_partial, v_partial = _q8_partials(cache, idx.shape[1], k_partial, v_partial, dev, stream)
    if workspace is None:
        workspace = new_workspace(256, dev, stream)
    _raise(_lib().ts_kv_gather_q8(
        ctypes.byref(st), _ptr(idx), idx.shape[1], _ptr(k_partial), _ptr(v_partial),
        k_partial.shape[1], _ptr(workspace), _ws_bytes(workspace, dev), _stream(stream, dev)),
        "ts_kv_gather_q8")
    return k_partial, v_partial


def kv_select_from_scores_q8(root_scores, cache: KvCacheQ8, n_sink: int, budget: int,
                             k_partial=None, v_partial=None, idx_out=None, scores_out=None,
                             workspace=None, stream=None, want_scores: bool = False):
    """:func:`kv_select_from_scores` on an 8-bit cache
    (``ts_kv_select_from_scores_q8``).

    Returns ``(idx [Hkv, n_keep] int32, k_partial, v_partial, scores or None)``.
    """
    _check_dev("root_scores", root_scores, torch.float32)
    dev, st = _call_cache(cache)
    if root_scores.device != dev:
        raise ValueError(f"root_scores is on {root_scores.device}, the call's tensors on {dev}")
    hq, n_ctx, hkv = root_scores.shape[0], cache.n_ctx, st.n_heads_kv
    if root_scores.shape[1] != n_ctx:
        raise ValueError("root_scores must be [Hq, n_ctx]")
    n_sink, budget = int(n_sink), int(budget)
    if not (-_C_INT <= n_sink < _C_INT and -_C_INT <= budget < _C_INT):
        raise ValueError("n_sink and budget must be signed 32-bit integers")
    n_keep = min(n_ctx, n_sink + budget)
    k_partial, v_partial = _q8_partials(cache, n_keep, k_partial, v_partial, dev, stream)
    if idx_out is None:
        idx_out = _empty((hkv, n_keep), _I32, dev, stream)
    _check_dev("idx_out", idx_out, _I32, dev)
    if idx_out.numel() != hkv * n_keep:
        raise ValueError("idx_out must be [Hkv, n_keep]")
    if want_scores and scores_out is None:
        scores_out = _empty((hkv, n_ctx), torch.float32, dev, stream)
    if scores_out is not None:
        _check_dev("scores_out", scores_out, torch.float32, dev)
        if scores_out.numel() != hkv * n_ctx:
            raise ValueError("scores_out must be [Hkv, n_ctx]")
    if workspace is None:
        workspace = new_workspace(kv_select_from_scores_workspace_size(hq, hkv, n_ctx), dev, stream)
    _raise(_lib().ts_kv_select_from_scores_q8(
        _ptr(root_scores), ctypes.byref(st), hq, n_sink, budget, _ptr(scores_out),
        _ptr(idx_out), _ptr(k_partial), _ptr(v_partial), k_partial.shape[1], _ptr(workspace),
        _ws_bytes(workspace, dev), _stream(stream, dev)), "ts_kv_select_from_scores_q8")
    return idx_out, k_partial, v_partial, scores_out


def kernel_launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(_lib().ts_kernel_launch_count())


def selftest_bounded_wait(workspace=None, stream=None):
    """``ts_selftest_bounded_wait``: one CTA takes the kernels' bounded wait
    on a barrier nothing completes; about a second later TS_ERR_TIMEOUT is
    in the workspace's status word.  Returns the workspace."""
    if workspace is None:
        workspace = new_workspace(256, stream=stream)
    nbytes = _ws_bytes(workspace, _call_device("workspace", workspace))
    _raise(_lib().ts_selftest_bounded_wait(_ptr(workspace), nbytes, _stream(stream)),
           "ts_selftest_bounded_wait")
    return workspace


def workspace_status(workspace, clear: bool = True, stream=None) -> int:
    """Device-side status word of a workspace (synchronises the stream)."""
    _ws_bytes(workspace, _call_device("workspace", workspace))
    return int(_lib().ts_workspace_status(_ptr(workspace), _stream(stream), int(clear)))


# --------------------------------------------------------- n-gram reuse table
class NgramTable:
    """The n-gram reuse table (``ts_ngram_*``) in a host buffer this object
    owns.  ``update(text, n_new)`` counts the n-grams of ``text`` that end
    at its last ``n_new`` tokens; ``topk(first, k)`` returns the most
    frequent ones starting with ``first`` as ``(continuations [m, n-1],
    counts [m])``, count descending, ties by continuation ascending;
    ``topk_prefix(prefix, k)`` does the same for a prefix of 1 to n-1
    tokens (n-1 tokens: the next-token counts)."""

    def __init__(self, n: int, capacity: int):
        import numpy as np
        nbytes = int(_lib().ts_ngram_table_bytes(int(n), int(capacity)))
        if nbytes == 0:
            raise ValueError("n must be in [2, 8] and capacity a power of two >= 2")
        self.n, self.capacity, self.nbytes = int(n), int(capacity), nbytes
        self._buf = np.empty((nbytes + 7) // 8, dtype=np.uint64)   # 8-byte aligned
        self._p = self._buf.ctypes.data_as(ctypes.c_void_p)
        _raise(_lib().ts_ngram_init(self._p, nbytes, self.n, self.capacity), "ts_ngram_init")

    def update(self, text, n_new: int | None = None) -> None:
        arr, p = _host_i32(text)
        n_new = len(arr) if n_new is None else int(n_new)
        _raise(_lib().ts_ngram_update(self._p, self.nbytes, p, len(arr), n_new),
               "ts_ngram_update")

    def topk(self, first: int, k: int):
        import numpy as np
        cont = np.empty((int(k), self.n - 1), dtype=np.int32)
        cnt = np.empty(int(k), dtype=np.int64)
        found = ctypes.c_int(0)
        _raise(_lib().ts_ngram_topk(self._p, self.nbytes, int(first), int(k),
                                    cont.ctypes.data_as(ctypes.c_void_p),
                                    cnt.ctypes.data_as(ctypes.c_void_p), ctypes.byref(found)),
               "ts_ngram_topk")
        return cont[:found.value], cnt[:found.value]

    def topk_prefix(self, prefix, k: int):
        """The k most frequent n-grams that start with ``prefix`` (1 to n-1
        tokens): ``(continuations [m, n - len(prefix)], counts [m])``."""
        import numpy as np
        arr, p = _host_i32(prefix)
        cont = np.empty((int(k), max(self.n - len(arr), 0)), dtype=np.int32)
        cnt = np.empty(int(k), dtype=np.int64)
        found = ctypes.c_int(0)
        _raise(_lib().ts_ngram_topk_prefix(self._p, self.nbytes, p, len(arr), int(k),
                                           cont.ctypes.data_as(ctypes.c_void_p),
                                           cnt.ctypes.data_as(ctypes.c_void_p),
                                           ctypes.byref(found)),
               "ts_ngram_topk_prefix")
        return cont[:found.value], cnt[:found.value]

    def count(self, gram) -> int:
        arr, p = _host_i32(gram)
        if len(arr) != self.n:
            raise ValueError(f"an n-gram has {self.n} tokens")
        c = ctypes.c_int64(0)
        _raise(_lib().ts_ngram_count(self._p, self.nbytes, p, ctypes.byref(c)), "ts_ngram_count")
        return int(c.value)

    def size(self):
        """(distinct n-grams held, n-grams counted)."""
        d, t = ctypes.c_int64(0), ctypes.c_int64(0)
        _raise(_lib().ts_ngram_size(self._p, self.nbytes, ctypes.byref(d), ctypes.byref(t)),
               "ts_ngram_size")
        return int(d.value), int(t.value)
