"""Python binding of libkda's C ABI (include/kda.h).

Argument marshalling only (ctypes; csrc/kda_tree_py.cpp for the draft-tree,
linear-attention and rotary calls): every step of the recurrence runs in libkda's CUDA kernels.  torch
supplies device memory and streams.  There is no CPU or
PyTorch fallback: if libkda.so cannot be loaded, or a tensor is not on a CUDA
device, the call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os

import torch

from . import build as _build

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_BOUNDS = range(6)
KDA_F32, KDA_BF16 = 0, 1

SYMBOLS = ("kda_status_string", "kda_prefill_workspace_size", "kda_prefill_chunked", "kda_prefill_chunked_profiled",
           "kda_prefill_check", "kda_decode_step", "kda_prefill_chunked_noalloc", "kda_prefill_noalloc_check",
           "kda_decode_step_indexed", "kda_state_snapshot", "kda_state_restore", "kda_prefill_chunked_ex",
           "kda_decode_step_ex", "kda_short_conv_prefill", "kda_short_conv_decode", "kda_tree_step",
           "kda_tree_commit", "kda_tree_conv", "kda_tree_conv_commit", "kda_draft_verify", "kda_linear_workspace_size",
           "kda_linear_prefill", "kda_linear_decode_step", "kda_rope")
# include/kda_testing.h (test hooks)
TESTING_SYMBOLS = ("kda_testing_set_plan", "kda_testing_set_fault")
PLAN_AUTO, PLAN_THREE, PLAN_CHAIN, PLAN_PIPE = -1, 0, 2, 3
FAULT_NONE, FAULT_NO_PUBLISH, FAULT_CHUNK_TABLE = 0, 1, 2
PREFILL_MAX_KERNELS = 4
TREE_MAX_NODES = 64
ROPE_MAX_D = 1024

_lib = None


class FusionOpts(ctypes.Structure):
    """kda_fusion_opts (include/kda.h): the fused q/k normalisation and gated output normalisation."""
    _fields_ = [("qk_l2norm", ctypes.c_int32), ("qk_eps", ctypes.c_float), ("out_gate", ctypes.c_void_p),
                ("out_weight", ctypes.c_void_p), ("out_eps", ctypes.c_float)]


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s" % (where, status_string(status)))


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Loads libkda.so (building it first when it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing:
        _build.build()
    if not os.path.exists(_build.LIB):
        raise RuntimeError("libkda.so is not built (%s); run gated_delta_rule_27_gb300.build" % _build.LIB)
    _lib = _declare(ctypes.CDLL(_build.LIB))
    return _lib


def load_debug() -> ctypes.CDLL:
    """Loads the bounds-checking build, libkda_debug.so (built on first use): the same C ABI, for tests."""
    _build.build(debug=True)
    return _declare(ctypes.CDLL(_build.DEBUG_LIB))


def _declare(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Sets the argument and result types of libkda's entry points on a loaded library."""
    vp, i32, fp = ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_prefill_workspace_size.restype = ctypes.c_size_t
    lib.kda_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.c_int, i32]
    lib.kda_prefill_chunked.restype = ctypes.c_int
    lib.kda_prefill_chunked.argtypes = [vp, vp, vp, fp, fp, vp, i32, i32, i32, i32, i32, ctypes.c_int, i32,
                                        fp, vp, fp, vp, ctypes.c_size_t, vp]
    lib.kda_prefill_chunked_profiled.restype = ctypes.c_int
    lib.kda_prefill_chunked_profiled.argtypes = lib.kda_prefill_chunked.argtypes + [
        ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_char_p)]
    lib.kda_prefill_check.restype = ctypes.c_int
    lib.kda_prefill_check.argtypes = [vp, vp]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [vp, vp, vp, fp, fp, i32, i32, i32, i32, ctypes.c_int, fp, vp, vp]
    lib.kda_prefill_chunked_noalloc.restype = ctypes.c_int
    lib.kda_prefill_chunked_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_int,
                                                i32, vp, vp, vp, vp]
    lib.kda_prefill_noalloc_check.restype = ctypes.c_int
    lib.kda_prefill_noalloc_check.argtypes = [vp]
    lib.kda_prefill_chunked_ex.restype = ctypes.c_int
    lib.kda_prefill_chunked_ex.argtypes = lib.kda_prefill_chunked.argtypes + [ctypes.POINTER(FusionOpts)]
    lib.kda_decode_step_ex.restype = ctypes.c_int
    lib.kda_decode_step_ex.argtypes = lib.kda_decode_step.argtypes + [ctypes.POINTER(FusionOpts)]
    lib.kda_short_conv_prefill.restype = ctypes.c_int
    lib.kda_short_conv_prefill.argtypes = [vp, fp, vp, i32, i32, i32, i32, ctypes.c_int, fp, vp, fp, vp]
    lib.kda_short_conv_decode.restype = ctypes.c_int
    lib.kda_short_conv_decode.argtypes = [vp, fp, i32, i32, i32, ctypes.c_int, fp, vp, vp]
    lib.kda_decode_step_indexed.restype = ctypes.c_int
    lib.kda_decode_step_indexed.argtypes = [vp, vp, vp, fp, fp, vp, i32, i32, i32, i32, i32, ctypes.c_int, fp, vp,
                                            vp, vp]
    for name in ("kda_state_snapshot", "kda_state_restore"):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = [fp, vp, i32, i32, i32, i32, i32, fp, vp, vp]
    dt, fusion = ctypes.c_int, ctypes.POINTER(FusionOpts)
    for name, types in (("kda_tree_step", [vp] * 8 + [i32] * 7 + [dt] + [vp] * 5 + [fusion]),
                        ("kda_tree_commit", [vp] * 7 + [i32] * 7 + [dt] + [vp] * 3 + [fusion]),
                        ("kda_tree_conv", [vp] * 5 + [i32] * 6 + [dt] + [vp] * 4),
                        ("kda_tree_conv_commit", [vp] * 5 + [i32] * 6 + [dt] + [vp] * 3),
                        ("kda_draft_verify", [vp] * 8 + [i32] * 3 + [dt, i32] + [vp] * 5),
                        ("kda_linear_prefill", [vp] * 4 + [i32, vp] + [i32] * 6 + [dt] + [vp] * 4 + [ctypes.c_size_t, vp, fusion]),
                        ("kda_linear_decode_step", [vp] * 4 + [i32, vp] + [i32] * 6 + [dt] + [vp] * 4 + [fusion]),
                        ("kda_rope", [vp] * 4 + [i32] * 6 + [ctypes.c_float, dt] + [vp] * 3)):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = types
    lib.kda_linear_workspace_size.restype = ctypes.c_size_t
    lib.kda_linear_workspace_size.argtypes = [i32, i32, i32, i32, i32, dt]
    lib.kda_testing_set_plan.restype = ctypes.c_int
    lib.kda_testing_set_plan.argtypes = [i32]
    lib.kda_testing_set_fault.restype = ctypes.c_int
    lib.kda_testing_set_fault.argtypes = [i32, ctypes.c_int64]
    return lib


def status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError("libkda takes bf16 or fp32 q/k/v, got %s" % t.dtype)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libkda takes device tensors; got a %s tensor" % t.device)
    if not t.is_contiguous():
        raise ValueError("libkda takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream, allocate, *args):
    """allocate(*args) as the given stream's memory (None: the current stream's).  The allocator hands out what is free in
    a stream's own order: a block of another stream may still be in use there when the call starts, and one that is given
    back right behind the call may be in use by the call when it is handed out again."""
    if stream is None:
        return allocate(*args)
    with torch.cuda.stream(stream):
        return allocate(*args)


def _output_on(stream, allocate, *args):
    """_on, for a tensor that the caller gets: one that the current stream's work may use too before its memory is given
    out again."""
    out = _on(stream, allocate, *args)
    if stream is not None:
        out.record_stream(torch.cuda.current_stream(out.device))
    return out


def kda_prefill_workspace_size(total_tokens: int, num_seqs: int, H: int, d_k: int, d_v: int, in_dtype: int,
                               chunk_size: int = 64) -> int:
    return int(load().kda_prefill_workspace_size(total_tokens, num_seqs, H, d_k, d_v, in_dtype, chunk_size))


def kda_prefill_chunked(q, k, v, g, beta, cu_seqlens, o, S0=None, S_final=None, workspace=None, chunk_size=64,
                        stream=None) -> None:
    """Calls kda_prefill_chunked on caller-owned device tensors (see include/kda.h)."""
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    dt = _dtype_code(q)
    if workspace is None:
        workspace = _on(stream, new_workspace, T, N, H, d_k, d_v, dt, chunk_size, q.device)
    rc = load().kda_prefill_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), N, T, H,
                                    d_k, d_v, dt, chunk_size, _ptr(S0), _ptr(o), _ptr(S_final), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_prefill_chunked")


def kda_prefill_chunked_profiled(q, k, v, g, beta, cu_seqlens, o, events, S0=None, S_final=None, workspace=None,
                                 chunk_size=64, stream=None):
    """kda_prefill_chunked plus CUDA events around its kernels.

    `events` is a list of torch.cuda.Event (len >= PREFILL_MAX_KERNELS + 1,
    created with enable_timing=True and already initialised by a record).
    Returns the names of the launched kernels; events[i] precedes kernel i and
    events[len(names)] follows the last one.
    """
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    dt = _dtype_code(q)
    if workspace is None:
        workspace = _on(stream, new_workspace, T, N, H, d_k, d_v, dt, chunk_size, q.device)
    n_ev = PREFILL_MAX_KERNELS + 1
    ev_arr = (ctypes.c_void_p * n_ev)(*[ctypes.c_void_p(e.cuda_event) for e in events[:n_ev]])
    n_k = ctypes.c_int32(0)
    names = (ctypes.c_char_p * PREFILL_MAX_KERNELS)()
    rc = load().kda_prefill_chunked_profiled(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), N, T,
                                             H, d_k, d_v, dt, chunk_size, _ptr(S0), _ptr(o), _ptr(S_final),
                                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                                             _stream(stream), ev_arr, ctypes.byref(n_k), names)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_prefill_chunked_profiled")
    return [names[i].decode() for i in range(n_k.value)]


def kda_prefill_check(workspace, stream=None) -> int:
    return int(load().kda_prefill_check(_ptr(workspace), _stream(stream)))


def kda_prefill_noalloc_check(stream=None) -> int:
    return int(load().kda_prefill_noalloc_check(_stream(stream)))


def testing_set_plan(plan: int) -> None:
    """Test hook (include/kda_testing.h): force a launch plan of the tensor-core prefill (PLAN_AUTO restores)."""
    rc = load().kda_testing_set_plan(int(plan))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_testing_set_plan")


def testing_set_fault(fault: int, wait_limit_ns: int = 0) -> None:
    """Test hook (include/kda_testing.h): inject a fault and bound the flag waits (FAULT_NONE, 0 restores)."""
    rc = load().kda_testing_set_fault(int(fault), int(wait_limit_ns))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_testing_set_fault")


def kda_decode_step(q, k, v, g, beta, S_inout, o, stream=None) -> None:
    """Calls kda_decode_step on caller-owned device tensors (see include/kda.h)."""
    N, H, d_k = q.shape
    d_v = v.shape[2]
    rc = load().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), N, H, d_k, d_v, _dtype_code(q),
                                _ptr(S_inout), _ptr(o), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_decode_step")


def fusion_opts(qk_l2norm=False, qk_eps=1e-6, out_gate=None, out_weight=None, out_eps=1e-6):
    """A kda_fusion_opts for the _ex entry points (None when nothing is fused)."""
    if not qk_l2norm and out_gate is None:
        return None
    return FusionOpts(1 if qk_l2norm else 0, float(qk_eps), _ptr(out_gate), _ptr(out_weight), float(out_eps))


def kda_prefill_chunked_ex(q, k, v, g, beta, cu_seqlens, o, S0=None, S_final=None, workspace=None, chunk_size=64,
                           stream=None, **fusion) -> None:
    """kda_prefill_chunked with the fused prologue / epilogue (keywords of fusion_opts)."""
    T, H, d_k = q.shape
    d_v = v.shape[2]
    N = cu_seqlens.numel() - 1
    dt = _dtype_code(q)
    if workspace is None:
        workspace = _on(stream, new_workspace, T, N, H, d_k, d_v, dt, chunk_size, q.device)
    opts = fusion_opts(**fusion)
    rc = load().kda_prefill_chunked_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), N, T, H,
                                       d_k, d_v, dt, chunk_size, _ptr(S0), _ptr(o), _ptr(S_final), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream),
                                       None if opts is None else ctypes.byref(opts))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_prefill_chunked_ex")


def kda_decode_step_ex(q, k, v, g, beta, S_inout, o, stream=None, **fusion) -> None:
    """kda_decode_step with the fused prologue / epilogue (keywords of fusion_opts)."""
    N, H, d_k = q.shape
    opts = fusion_opts(**fusion)
    rc = load().kda_decode_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), N, H, d_k, v.shape[2],
                                   _dtype_code(q), _ptr(S_inout), _ptr(o), _stream(stream),
                                   None if opts is None else ctypes.byref(opts))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_decode_step_ex")


def kda_short_conv_prefill(x, w, cu_seqlens, y, conv_state=None, conv_state_out=None, stream=None) -> None:
    """kda_short_conv_prefill on x [T, C] (or [T, H, d], flattened), w [C, W]."""
    T = x.shape[0]
    C, W = w.shape
    rc = load().kda_short_conv_prefill(_ptr(x), _ptr(w), _ptr(cu_seqlens), cu_seqlens.numel() - 1, T, C, W,
                                       _dtype_code(x), _ptr(conv_state), _ptr(y), _ptr(conv_state_out),
                                       _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_short_conv_prefill")


def kda_short_conv_decode(x, w, conv_state, y, stream=None) -> None:
    """kda_short_conv_decode on x [N, C]: one token per sequence, conv_state [N, W - 1, C] rolled in place."""
    N = x.shape[0]
    C, W = w.shape
    rc = load().kda_short_conv_decode(_ptr(x), _ptr(w), N, C, W, _dtype_code(x), _ptr(conv_state), _ptr(y),
                                      _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_short_conv_decode")


def kda_decode_step_indexed(q, k, v, g, beta, seq_idx, S_pool, o, status=None, stream=None) -> None:
    """Calls kda_decode_step_indexed: one token for each listed pool slot (see include/kda.h)."""
    A, H, d_k = q.shape
    d_v = v.shape[2]
    rc = load().kda_decode_step_indexed(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(seq_idx), A,
                                        S_pool.shape[0], H, d_k, d_v, _dtype_code(q), _ptr(S_pool), _ptr(o),
                                        _ptr(status), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_decode_step_indexed")


def kda_state_snapshot(S_pool, seq_idx, S_saved, status=None, stream=None) -> None:
    """S_saved[i] = S_pool[seq_idx[i]] (kda_state_snapshot)."""
    num_slots, H, d_k, d_v = S_pool.shape
    rc = load().kda_state_snapshot(_ptr(S_pool), _ptr(seq_idx), seq_idx.numel(), num_slots, H, d_k, d_v,
                                   _ptr(S_saved), _ptr(status), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_state_snapshot")


def kda_state_restore(S_saved, seq_idx, S_pool, status=None, stream=None) -> None:
    """S_pool[seq_idx[i]] = S_saved[i] (kda_state_restore)."""
    num_slots, H, d_k, d_v = S_pool.shape
    rc = load().kda_state_restore(_ptr(S_saved), _ptr(seq_idx), seq_idx.numel(), num_slots, H, d_k, d_v,
                                  _ptr(S_pool), _ptr(status), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_state_restore")


# the draft-tree, linear-attention and rotary calls: marshalled and checked by csrc/kda_tree_py.cpp, which calls
# libkda.so's entry points
_tree_calls = None


def _tree():
    """The marshalling module, built and loaded on first use and given the addresses of the loaded library."""
    global _tree_calls
    if _tree_calls is None:
        lib = load()
        spec = importlib.util.spec_from_file_location("_kda_tree", _build.build_tree_py())
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.init(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                      for name in ("kda_tree_step", "kda_tree_commit", "kda_tree_conv", "kda_tree_conv_commit",
                                   "kda_draft_verify", "kda_linear_prefill", "kda_linear_decode_step", "kda_rope")))
        _tree_calls = module
    return _tree_calls


def kda_tree_step(q, k, v, g, beta, parent, cu_nodes, seq_idx, S_pool, o, u, max_nodes, status=None, stream=None,
                  qk_l2norm=False, qk_eps=1e-6, out_gate=None, out_weight=None, out_eps=1e-6) -> None:
    """KDA attention of every draft-tree node over the state pool (kda_tree_step): q, k, v, g [T, H, d] and beta
    [T, H] packed as include/kda.h says, o and u (or None) written; the fused normalisations as for fusion_opts."""
    rc = (_tree_calls or _tree()).tree_step(q, k, v, g, beta, parent, cu_nodes, seq_idx, S_pool, o, u, max_nodes, status,
                                            stream, qk_l2norm, qk_eps, out_gate, out_weight, out_eps)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_tree_step")


def kda_tree_commit(k, g, u, cu_nodes, path, path_len, seq_idx, S_pool, status=None, stream=None, qk_l2norm=False,
                    qk_eps=1e-6) -> None:
    """Moves the pool's states along the accepted paths (kda_tree_commit), in place."""
    rc = (_tree_calls or _tree()).tree_commit(k, g, u, cu_nodes, path, path_len, seq_idx, S_pool, status, stream, qk_l2norm,
                                              qk_eps)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_tree_commit")


def kda_tree_conv(x, w, parent, cu_nodes, seq_idx, conv_pool, y, max_nodes, status=None, stream=None) -> None:
    """The short convolution along every node's path (kda_tree_conv): x, y [T, C], w [C, W], conv_pool
    [slots, W - 1, C] (read only)."""
    rc = (_tree_calls or _tree()).tree_conv(x, w, parent, cu_nodes, seq_idx, conv_pool, y, max_nodes, status, stream)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_tree_conv")


def kda_tree_conv_commit(x, cu_nodes, path, path_len, seq_idx, conv_pool, status=None, stream=None) -> None:
    """Moves the carried convolution inputs along the accepted paths (kda_tree_conv_commit), in place."""
    rc = (_tree_calls or _tree()).tree_conv_commit(x, cu_nodes, path, path_len, seq_idx, conv_pool, status, stream)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_tree_conv_commit")


def kda_draft_verify(logits, tokens, parent, cu_nodes, u_accept, u_next, path, path_len, next_token, draft_probs=None,
                     temperature=None, status=None, stream=None) -> None:
    """Verifies drafted tokens against the target's logits [T, V] (kda_draft_verify): writes the kept paths
    [N, max nodes], their lengths and the next tokens."""
    rc = (_tree_calls or _tree()).draft_verify(logits, tokens, parent, cu_nodes, u_accept, u_next, path, path_len, next_token,
                                               draft_probs, temperature, status, stream)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_draft_verify")


def kda_linear_workspace_size(total_tokens: int, num_seqs: int, H: int, d_k: int, d_v: int, in_dtype: int) -> int:
    return int(load().kda_linear_workspace_size(total_tokens, num_seqs, H, d_k, d_v, in_dtype))


def new_linear_workspace(q, v, cu_seqlens) -> torch.Tensor:
    """The device scratch of kda_linear_prefill for tensors of these shapes."""
    T, H, d = v.shape
    n = kda_linear_workspace_size(T, cu_seqlens.numel() - 1, H, d, d, _dtype_code(q))
    if n == 0:
        raise KdaError(KDA_ERR_UNSUPPORTED, "kda_linear_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def kda_linear_prefill(q, k, v, g, cu_seqlens, o, S0=None, S_final=None, workspace=None, stream=None, qk_l2norm=False,
                       qk_eps=1e-6, out_gate=None, out_weight=None, out_eps=1e-6) -> None:
    """Linear attention with one decay per head over packed documents (kda_linear_prefill): q, k [T, H_qk, d], v, o
    [T, H, d], g [T, H] or [H]; the fused normalisations as for fusion_opts."""
    if workspace is None and torch.is_tensor(q) and torch.is_tensor(v) and v.dim() == 3 and torch.is_tensor(cu_seqlens):
        workspace = _on(stream, new_linear_workspace, q, v, cu_seqlens)
    rc = (_tree_calls or _tree()).linear_prefill(q, k, v, g, cu_seqlens, o, S0, S_final, workspace, stream, qk_l2norm, qk_eps,
                                                 out_gate, out_weight, out_eps)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_linear_prefill")


def kda_linear_decode_step(q, k, v, g, S_pool, o, seq_idx=None, status=None, stream=None, qk_l2norm=False, qk_eps=1e-6,
                           out_gate=None, out_weight=None, out_eps=1e-6) -> None:
    """One token for each listed slot of a pool of linear-attention states (kda_linear_decode_step): q, k [N, H_qk, d],
    v, o [N, H, d], g [N, H] or [H], S_pool [slots, H, d, d] updated in place."""
    rc = (_tree_calls or _tree()).linear_decode_step(q, k, v, g, S_pool, o, seq_idx, status, stream, qk_l2norm, qk_eps,
                                                     out_gate, out_weight, out_eps)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_linear_decode_step")


def kda_rope(q, k, positions, steps, q_out, k_out, interleaved=False, scale=1.0, stream=None) -> None:
    """Rotary positions of q [T, H_q, d] and k [T, H_k, d] (or None) (kda_rope): positions [T] int32, steps from
    rope_steps; q_out and k_out may be q and k."""
    rc = (_tree_calls or _tree()).rope(q, k, positions, steps, q_out, k_out, interleaved, scale, stream)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_rope")


def rope_steps(inv_freq) -> torch.Tensor:
    """kda_rope's table for frequencies in radians a position (fp64, [rot / 2]): int64 with the bits of the part of a
    turn that a position adds, in steps of 2^-64 turn.  Negative frequencies turn back."""
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise TypeError("rope_steps takes a one-dimensional tensor of float64")
    turn = torch.remainder(inv_freq / (2 * math.pi), 1.0) * 2.0 ** 32
    upper = torch.floor(turn)
    lower = torch.floor((turn - upper) * 2.0 ** 32)
    return (upper.to(torch.int64) << 32) + lower.to(torch.int64)


def rope_frequencies(rot: int, base: float = 10000.0, scaling=None):
    """(inv_freq [rot / 2] fp64, scale) of rotary positions, pair i turning base^(-2i / rot) radians a position.

    scaling stretches them for contexts longer than the original one:
      {"type": "linear", "factor": s}  every pair s times slower
      {"type": "ntk", "factor": s}     the base grown so that the slowest pair is s times slower and the fastest kept
      {"type": "yarn", "factor": s, "original_max_position": n, "beta_fast": 32, "beta_slow": 1}
          pairs that turn more than beta_fast times in n positions kept, those that turn less than beta_slow times s
          times slower, a linear blend between; scale is 0.1 ln s + 1
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot is even and at least 2, got %r" % (rot,))
    pair = torch.arange(rot // 2, dtype=torch.float64)
    kind = None if scaling is None else scaling["type"]
    factor = 1.0 if scaling is None else float(scaling["factor"])
    if factor < 1.0:
        raise ValueError("a scaling's factor is at least 1, got %r" % (factor,))
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    plain = base ** (-2.0 * pair / rot)
    if kind in (None, "ntk"):
        return plain, 1.0
    if kind == "linear":
        return plain / factor, 1.0
    if kind != "yarn":
        raise ValueError("unknown scaling %r" % (kind,))
    original = scaling["original_max_position"]
    at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo = max(0.0, math.floor(at(scaling.get("beta_fast", 32.0))))
    hi = min(rot - 1.0, math.ceil(at(scaling.get("beta_slow", 1.0))))
    slow = ((pair - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return plain * (1 - slow) + plain / factor * slow, 0.1 * math.log(factor) + 1.0


def new_workspace(T, N, H, d_k, d_v, in_dtype, chunk_size, device) -> torch.Tensor:
    n = kda_prefill_workspace_size(T, N, H, d_k, d_v, in_dtype, chunk_size)
    if n == 0:
        raise KdaError(KDA_ERR_UNSUPPORTED, "kda_prefill_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def prefill(q, k, v, g, beta, cu_seqlens, S0=None, chunk_size=64, want_state=True, workspace=None, stream=None):
    """Allocates o (and S_final) with torch, as the stream's memory, and runs kda_prefill_chunked; returns (o, S_final)."""
    T, H, d_k = q.shape
    N = cu_seqlens.numel() - 1
    fresh = lambda shape, dtype: _output_on(stream, lambda: torch.empty(shape, dtype=dtype, device=q.device))  # noqa: E731
    o = fresh((T, H, v.shape[2]), v.dtype)
    S_final = fresh((N, H, d_k, v.shape[2]), torch.float32) if want_state else None
    kda_prefill_chunked(q, k, v, g, beta, cu_seqlens, o, S0=S0, S_final=S_final, workspace=workspace,
                        chunk_size=chunk_size, stream=stream)
    return o, S_final


def decode_step(q, k, v, g, beta, S_inout, stream=None):
    """Allocates o with torch, as the stream's memory, runs kda_decode_step (S_inout updated in place); returns o."""
    o = _output_on(stream, torch.empty_like, v)
    kda_decode_step(q, k, v, g, beta, S_inout, o, stream=stream)
    return o


NOALLOC_SCRATCH_BYTES = 64 << 20


def kda_prefill_chunked_noalloc(q, k, v, g, beta, cu_seqlens, o, S0=None, S_final=None, chunk_size=64,
                                stream=None) -> None:
    """Calls kda_prefill_chunked_noalloc: the prefill with the library's static scratch, no workspace argument.

    For callers that must not allocate device memory; see include/kda.h for
    the scratch limit and the rule that overlapping calls on one GPU race.
    """
    lib = load()
    T, H, d_k = q.shape
    N = cu_seqlens.numel() - 1
    rc = lib.kda_prefill_chunked_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), N, T, H,
                                         d_k, v.shape[2], _dtype_code(q), chunk_size, _ptr(S0), _ptr(o),
                                         _ptr(S_final), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_prefill_chunked_noalloc")
