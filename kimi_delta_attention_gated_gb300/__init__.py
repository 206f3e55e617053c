"""Kimi Delta Attention core on GB300: Python binding of libkda.

Thin ctypes marshalling over the C ABI declared in include/kda.h: every step of
the computation runs in libkda's CUDA kernels; torch only allocates device memory
and supplies the current stream.  There is no CPU fallback: calling any function
without a built libkda (or without a GPU) raises.

Entry points (same names as the C ABI, minus the ``kda_`` prefix):
  chunk_fwd       chunked prefill  (q, k, v, g, beta, initial_state) -> (o, final_state[, y])
  recurrent_fwd   token-by-token form over T tokens, optional per-token states
  recurrent_step  one decode token per sequence with the fused gated norm
  gated_rmsnorm   y = RMSNorm_v(o) * w * sigmoid(gate) per (token, head)
The full-attention layers beside the KDA layers:
  rotary          rotary positions (rotary_inv_freq: the angles, scaled for long contexts)
  kv_append       keys and values into a paged 8-bit cache (kv_cache), rotated on the way
  attn_decode     one query token per sequence over that cache
  attn_prompt     causal attention over whole (packed) prompts

Inputs may live on the host: they are copied to the current CUDA device, and the
results are copied back to the host, which makes the call end-to-end.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import NamedTuple

import torch

__all__ = ["chunk_fwd", "chunk_fwd_logits", "recurrent_fwd", "recurrent_step", "recurrent_step_logits",
           "gated_rmsnorm", "short_conv", "o_proj", "launch_count", "device_status", "set_wait_limit",
           "workspace_size", "release_workspaces", "prepass_hits",
           "KVCache", "kv_cache", "rotary_inv_freq", "rotary", "kv_append", "attn_decode", "attn_decode_workspace_size",
           "attn_prompt", "attn_prompt_workspace_size",
           "library_path", "KDAError", "MODE_AUTO", "MODE_TENSOR", "MODE_FP32", "MODE_SPLIT"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libkda.so")
_lib = None
_lock = threading.Lock()

BF16, F32 = 0, 1
MODE_AUTO, MODE_TENSOR, MODE_FP32, MODE_SPLIT = 0, 1, 2, 3
_MODES = {"auto": MODE_AUTO, "tensor": MODE_TENSOR, "fp32": MODE_FP32, "split": MODE_SPLIT}
_STATUS = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED", 3: "KDA_ERR_CUDA",
           4: "KDA_ERR_TIMEOUT"}


class KDAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libkda.so is not built ({_LIB_PATH}); run __graft_entry__.build() "
                               "or python kimi_delta_attention_gated_gb300/build.py")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        Z = ctypes.c_size_t
        lib.kda_chunk_fwd.argtypes = [P, P, P, I, P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, F, I,
                                      P, I, P, F, P, P, Z, I, P]
        lib.kda_chunk_fwd_noalloc.argtypes = [P, P, P, I, P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, F, I,
                                              P, I, P, F, P, I, P]
        lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.kda_chunk_workspace_size.argtypes = [I, I, I, I]
        lib.kda_chunk_workspace_size.restype = Z
        lib.kda_chunk_fwd_host_workspace_size.argtypes = [I, I, I, I, I]
        lib.kda_chunk_fwd_host_workspace_size.restype = Z
        lib.kda_chunk_fwd_host.argtypes = [P, P, P, I, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, I, P, F, P, I,
                                           P, Z, I, P]
        lib.kda_chunk_fwd_logits_host.argtypes = [P, P, P, I, P, I, P, P, F, P, I, P, P, P, I, I, I, I, I, I, I,
                                                  F, I, P, I, P, F, P, I, P, Z, I, P]
        lib.kda_recurrent_fwd.argtypes = [P, P, P, I, P, P, P, P, P, I, P, P, P, I, I, I, I, I, I, F, I,
                                          P, I, P, F, P, P]
        lib.kda_recurrent_step.argtypes = [P, P, P, I, P, P, P, P, P, I, I, I, I, I, F, I, P, I, P, F,
                                           P, P]
        lib.kda_gated_rmsnorm.argtypes = [P, I, P, I, P, F, P, I, ctypes.c_int64, I, I, P]
        lib.kda_short_conv_fwd.argtypes = [P, I, P, P, P, P, P, I, P, P, I, I, I, I, I, I, P]
        lib.kda_chunk_fwd_logits.argtypes = [P, P, P, I, P, I, P, P, F, P, I, P, P, P, I, P, P, I, I, I, I, I, I,
                                             I, F, I, P, I, P, F, P, P, Z, I, P]
        lib.kda_recurrent_step_logits.argtypes = [P, P, P, I, P, I, P, P, F, P, I, P, P, P, I, I, I, I, I, F, I,
                                                  P, I, P, F, P, P]
        lib.kda_o_proj.argtypes = [P, P, P, I, ctypes.c_int64, I, I, P]
        P3 = ctypes.POINTER(ctypes.c_void_p)  # a host array of three device pointers, or NULL
        lib.kda_recurrent_step_conv.argtypes = [P, P, P, I, P3, I, P3, P3, P, P, P, I, P, P, F, P, I, P, P, P, I,
                                                I, I, I, I, F, I, P, I, P, F, P, P]
        for fn in ("kda_chunk_fwd", "kda_recurrent_fwd", "kda_recurrent_step", "kda_gated_rmsnorm",
                   "kda_short_conv_fwd", "kda_chunk_fwd_logits", "kda_recurrent_step_logits", "kda_o_proj",
                   "kda_recurrent_step_conv", "kda_chunk_fwd_host", "kda_chunk_fwd_logits_host"):
            getattr(lib, fn).restype = ctypes.c_int
        L = ctypes.c_int64
        lib.kda_rotary.argtypes = [P, I, L, P, P, F, I, I, I, P, L, L, I, I, P]
        lib.kda_kv_append.argtypes = [P, L, P, L, L, I, I, P, P, P, P, I, I, P, I, P, P, I, P, F, I, I, P, L, I, P, P, P]
        lib.kda_attn_decode.argtypes = [P, L, P, P, P, P, I, I, P, I, P, I, I, I, I, F, P, I, P, P, Z, P]
        lib.kda_attn_decode_workspace_size.argtypes = [I, I, I, I, L]
        lib.kda_attn_decode_workspace_size.restype = Z
        lib.kda_attn_prompt.argtypes = [P, L, P, L, P, L, L, L, I, I, I, I, P, P, I, F, P, I, P, P, Z, P]
        lib.kda_attn_prompt_workspace_size.argtypes = [L, L, I, I, I, I]
        lib.kda_attn_prompt_workspace_size.restype = Z
        for fn in ("kda_rotary", "kda_kv_append", "kda_attn_decode", "kda_attn_prompt"):
            getattr(lib, fn).restype = ctypes.c_int
        lib.kda_device_status.argtypes = [P]
        lib.kda_device_status.restype = ctypes.c_int
        lib.kda_chunk_prepass_hits.argtypes = [P, ctypes.POINTER(ctypes.c_uint64)]
        lib.kda_chunk_prepass_hits.restype = ctypes.c_int
        lib.kda_set_wait_limit.argtypes = [ctypes.c_int64]
        lib.kda_set_wait_limit.restype = ctypes.c_int
        lib.kda_last_error.restype = ctypes.c_char_p
        lib.kda_launch_count.restype = ctypes.c_uint64
        lib.kda_version.restype = ctypes.c_int
        _lib = lib
    return _lib


def _check(status: int):
    if status != 0:
        raise KDAError(status, _load().kda_last_error().decode())


def launch_count() -> int:
    """Kernels libkda has launched in this process."""
    return int(_load().kda_launch_count())


def device_status(stream=None):
    """Synchronise the stream (default: the current one) and raise KDAError with
    KDA_ERR_TIMEOUT if a bounded wait inside a kernel gave up since the last check
    (those outputs hold NaN).  Clears the device's counters."""
    st = ctypes.c_void_p((stream or torch.cuda.current_stream()).cuda_stream)
    _check(_load().kda_device_status(st))


def prepass_hits(stream=None) -> int:
    """Chunks of the concurrent prefill form that took their grams and UT transform from the
    pre-pass since the last call (synchronises the stream; clears the device's counter)."""
    st = ctypes.c_void_p((stream or torch.cuda.current_stream()).cuda_stream)
    n = ctypes.c_uint64(0)
    _check(_load().kda_chunk_prepass_hits(st, ctypes.byref(n)))
    return int(n.value)


def set_wait_limit(polls):
    """Bound on the streaming kernels' first-line waits (None or a negative value: the
    default; 0: every such wait gives up at once, for tests of the failure handling)."""
    _check(_load().kda_set_wait_limit(-1 if polls is None else int(polls)))


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _prep(t, device, dtype=None):
    """Contiguous device tensor (host tensors are copied; pinned ones asynchronously)."""
    if t is None:
        return None
    if dtype is not None and t.dtype != dtype:
        t = t.to(dtype)
    if t.device.type != "cuda":
        t = t.to(device, non_blocking=t.is_pinned())
    return t.contiguous()


def _device_of(*ts):
    for t in ts:
        if t is not None and t.device.type == "cuda":
            return t.device
    return torch.device("cuda", torch.cuda.current_device())


def _cu(cu_seqlens, device):
    if cu_seqlens is None:
        return None, None, 0
    host = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
    dev = cu_seqlens.to(device=device, dtype=torch.int32).contiguous()
    return dev, host, host.numel() - 1


def _to_host(ts, host, dests=None):
    """Copy results back to the host: into the caller's host tensors when given
    (asynchronously when they are pinned, then the stream is synchronised)."""
    if not host:
        return ts
    out = []
    for i, t in enumerate(ts):
        dst = dests[i] if dests is not None else None
        if t is None:
            out.append(None)
        elif dst is not None:
            dst.copy_(t, non_blocking=dst.is_pinned())
            out.append(dst)
        else:
            out.append(t.to("cpu"))
    torch.cuda.current_stream().synchronize()
    return tuple(out)


def _dev_out(t):
    """A caller-provided output on the host is computed on the device first."""
    return None if (t is None or t.device.type != "cuda") else t


def chunk_fwd(q, k, v, g, beta, initial_state=None, *, scale=None, chunk=64, use_qk_l2norm=True,
              cu_seqlens=None, output_final_state=True, gate=None, norm_w=None, eps=1e-5,
              out_dtype=torch.float32, mode="auto", return_o=True, o=None, y=None, final_state=None,
              workspace=None):
    """Chunked prefill.  q, k [B,T,H,K]; v [B,T,H,V]; g [B,T,H,K] fp32; beta [B,T,H] fp32;
    initial_state [N,H,K,V] fp32 or None.  With ``cu_seqlens`` (int, n_seqs + 1) B must be 1.
    Returns (o, final_state) or, with ``gate``/``norm_w``, (o, final_state, y) where
    y [B,T,H*V] is the sigmoid-gated RMSNorm of o (o is None when return_o=False).
    Preallocated outputs may be passed as o / y / final_state (final_state may be
    initial_state itself for an in-place update).  ``workspace``: None (the fused one-kernel
    tensor-core form), a uint8 device tensor of at least workspace_size(...) bytes, or
    "auto" (a per-device buffer this binding keeps).  With a workspace the fused kernel is
    joined by a pre-pass on the SMs it leaves idle (fewer (sequence, head) units than SMs),
    which forms chunks' grams and UT transform ahead of it (the concurrent form); with
    ``mode="split"`` the pre-pass instead forms every chunk's first and a per-head chain
    kernel follows (the split form).  Every form gives the same bits.  The kept buffer is
    shared by every "auto" call on a device: calls on streams that may run at the same time
    need workspaces of their own."""
    return _chunk(q, k, v, (g, beta), None, initial_state, scale, chunk, use_qk_l2norm, cu_seqlens,
                  output_final_state, gate, norm_w, eps, out_dtype, mode, return_o, o, y, final_state, workspace)


def chunk_fwd_logits(q, k, v, g_logits, beta_logits, A_log, initial_state=None, *, dt_bias=None,
                     g_lower_bound=-5.0, scale=None, chunk=64, use_qk_l2norm=True, cu_seqlens=None,
                     output_final_state=True, gate=None, norm_w=None, eps=1e-5, out_dtype=torch.float32,
                     mode="auto", return_o=True, o=None, y=None, final_state=None, workspace=None):
    """chunk_fwd with g = max(g_lower_bound, -exp(A_log[h]) * softplus(g_logits + dt_bias)) and
    beta = sigmoid(beta_logits) computed inside the kernels.  g_logits [B,T,H,K] and
    beta_logits [B,T,H] in bf16 or fp32; A_log [H]; dt_bias [H,K] (or [H*K]) or None;
    g_lower_bound None for no floor."""
    lb = float("-inf") if g_lower_bound is None else float(g_lower_bound)
    return _chunk(q, k, v, None, (g_logits, beta_logits, A_log, dt_bias, lb), initial_state, scale, chunk,
                  use_qk_l2norm, cu_seqlens, output_final_state, gate, norm_w, eps, out_dtype, mode, return_o, o, y,
                  final_state, workspace)


def workspace_size(B, T, H, n_seqs=0) -> int:
    """Bytes of workspace the split tensor-core prefill needs (kda_chunk_workspace_size)."""
    return int(_load().kda_chunk_workspace_size(int(B), int(T), int(H), int(n_seqs)))


_CHUNK_WS = {}


def _chunk_workspace(spec, dev, B, T, H, n_seqs):
    """(pointer, bytes) of the workspace for one call: None -> the fused form."""
    if spec is None:
        return None, 0
    need = workspace_size(B, T, H, n_seqs)
    if isinstance(spec, str):
        if spec != "auto":
            raise ValueError('workspace must be "auto", None or a device tensor')
        key = dev.index if dev.index is not None else torch.cuda.current_device()
        ws = _CHUNK_WS.get(key)
        if ws is None or ws.numel() < need:
            _CHUNK_WS.pop(key, None)
            ws = _CHUNK_WS[key] = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        return ctypes.c_void_p(ws.data_ptr()), ws.numel()
    return ctypes.c_void_p(spec.data_ptr()), spec.numel() * spec.element_size()


def release_workspaces():
    """Drop the workspaces this binding keeps (the next call allocates again)."""
    _CHUNK_WS.clear()


def _pinned(t):
    return t if t.is_pinned() else t.pin_memory()


def _chunk_host_streamed(q, k, v, gb, lg, initial_state, scale, chunk, use_qk_l2norm, output_final_state, gate,
                         norm_w, eps, out_dtype, mode, return_o, o, y, final_state):
    """A host-resident dense prompt through kda_chunk_fwd_host (_logits_host): the library
    streams it through the device in HOST_SEGMENT-token segments, copies in and out on two
    streams of its own while the kernels run on the current stream.  Inputs are made
    page-locked (copied once if they are not); outputs are page-locked host tensors (or the
    caller's).  The fused kernel runs each segment; the result equals one device call."""
    lib = _load()
    dev = torch.device("cuda", torch.cuda.current_device())
    B, T, H, K = q.shape
    V = v.shape[-1]
    if scale is None:
        scale = K ** -0.5
    pin = lambda t: None if t is None else _pinned(t.detach().contiguous())
    host32 = lambda t: None if t is None else t.detach().to("cpu", torch.float32).contiguous()
    q, k, v = pin(q), pin(k), pin(v)
    want_o = return_o or gate is None or o is not None
    o_h = (o if o is not None else torch.empty((B, T, H, V), dtype=out_dtype).pin_memory()) if want_o else None
    y_h = norm_h = None
    if gate is not None:
        gate = pin(gate)
        norm_h = host32(norm_w)
        y_h = y if y is not None else torch.empty((B, T, H * V), dtype=out_dtype).pin_memory()
    fs_h = final_state if final_state is not None else (
        torch.empty((B, H, K, V), dtype=torch.float32).pin_memory() if output_final_state else None)
    s0 = host32(initial_state)
    need = int(lib.kda_chunk_fwd_host_workspace_size(B, H, K, V, HOST_SEGMENT))
    key = ("host", dev.index)
    ws = _CHUNK_WS.get(key)
    if ws is None or ws.numel() < need:
        _CHUNK_WS.pop(key, None)
        ws = _CHUNK_WS[key] = torch.empty(need, dtype=torch.uint8, device=dev)
    mode_i = _MODES[mode] if isinstance(mode, str) else int(mode)
    tail = (_ptr(s0), _ptr(fs_h), _ptr(o_h), _dt(o_h if o_h is not None else y_h), B, T, H, K, V, int(chunk),
            float(scale), int(bool(use_qk_l2norm)), _ptr(gate), _dt(gate) if gate is not None else BF16, _ptr(norm_h),
            float(eps), _ptr(y_h), HOST_SEGMENT, ctypes.c_void_p(ws.data_ptr()), ws.numel(), mode_i, _stream())
    if lg is None:
        g, beta = pin(gb[0].to(torch.float32)), pin(gb[1].to(torch.float32))
        _check(lib.kda_chunk_fwd_host(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), *tail))
    else:
        z, b, A_log, dt_bias, lb = lg
        z, b, A_log, dt_bias = pin(z), pin(b), host32(A_log), host32(dt_bias)
        _check(lib.kda_chunk_fwd_logits_host(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(z), _dt(z), _ptr(A_log),
                                             _ptr(dt_bias), lb, _ptr(b), _dt(b), *tail))
    torch.cuda.current_stream().synchronize()  # the outputs are in host memory once the stream is done
    o_ret = o_h if return_o or gate is None else None
    if gate is not None:
        return o_ret, fs_h, y_h
    return o_ret, fs_h


def _logit_args(lg, dev):
    z, b, A_log, dt_bias, lb = lg
    z, b = _prep(z, dev), _prep(b, dev)
    A_log = _prep(A_log, dev, torch.float32)
    dt_bias = _prep(dt_bias, dev, torch.float32)
    return z, b, A_log, dt_bias, lb


# Host-resident prompts at least this long are streamed through the device in segments
# of HOST_SEGMENT tokens (a multiple of the 64-token chunk).
HOST_SEGMENT = 1024


def _chunk(q, k, v, gb, lg, initial_state, scale, chunk, use_qk_l2norm, cu_seqlens, output_final_state, gate,
           norm_w, eps, out_dtype, mode, return_o, o, y, final_state, workspace=None):
    lib = _load()
    host = q.device.type != "cuda"
    on_host = lambda t: t is None or t.device.type == "cpu"
    if (host and cu_seqlens is None and q.shape[1] >= 2 * HOST_SEGMENT and workspace is None
            and on_host(o) and on_host(y) and on_host(final_state) and torch.cuda.is_available()):
        return _chunk_host_streamed(q, k, v, gb, lg, initial_state, scale, chunk, use_qk_l2norm,
                                    output_final_state, gate, norm_w, eps, out_dtype, mode, return_o, o, y,
                                    final_state)
    dev = _device_of(q, k, v)
    dests = (o, final_state, y) if host else None
    if host:
        o, final_state, y = _dev_out(o), _dev_out(final_state), _dev_out(y)
    q, k, v = _prep(q, dev), _prep(k, dev), _prep(v, dev)
    initial_state = _prep(initial_state, dev, torch.float32)
    B, T, H, K = q.shape
    V = v.shape[-1]
    cu_d, cu_h, n_seqs = _cu(cu_seqlens, dev)
    N = n_seqs if cu_d is not None else B
    if gate is not None:
        gate, norm_w = _prep(gate, dev), _prep(norm_w, dev, torch.float32)
        if y is None:
            y = torch.empty((B, T, H * V), device=dev, dtype=out_dtype)
    if o is None and (return_o or (dests is not None and dests[0] is not None) or gate is None):
        o = torch.empty((B, T, H, V), device=dev, dtype=out_dtype)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, K, V), device=dev, dtype=torch.float32)
    if scale is None:
        scale = K ** -0.5
    mode_i = _MODES[mode] if isinstance(mode, str) else int(mode)
    ws_ptr, ws_bytes = _chunk_workspace(workspace if mode_i != MODE_FP32 else None, dev, B, T, H, n_seqs)
    tail = (_ptr(initial_state), _ptr(final_state), _ptr(o), _dt(o if o is not None else y), _ptr(cu_d), _ptr(cu_h),
            n_seqs, B, T, H, K, V, int(chunk), float(scale), int(bool(use_qk_l2norm)), _ptr(gate),
            _dt(gate) if gate is not None else BF16, _ptr(norm_w), float(eps), _ptr(y), ws_ptr, ws_bytes,
            mode_i, _stream())
    if lg is None:
        g, beta = _prep(gb[0], dev, torch.float32), _prep(gb[1], dev, torch.float32)
        _check(lib.kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), *tail))
    else:
        z, b, A_log, dt_bias, lb = _logit_args(lg, dev)
        _check(lib.kda_chunk_fwd_logits(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(z), _dt(z), _ptr(A_log),
                                        _ptr(dt_bias), lb, _ptr(b), _dt(b), *tail))
    if gate is not None:
        return _to_host((o, final_state, y), host, dests)
    return _to_host((o, final_state), host, dests)


def recurrent_fwd(q, k, v, g, beta, initial_state=None, *, scale=None, use_qk_l2norm=True,
                  cu_seqlens=None, output_final_state=True, output_states=False, gate=None,
                  norm_w=None, eps=1e-5, out_dtype=torch.float32):
    """Token-by-token form over T tokens (fp32).  Returns (o, final_state[, states][, y])."""
    lib = _load()
    host = q.device.type != "cuda"
    dev = _device_of(q, k, v)
    q, k, v = _prep(q, dev), _prep(k, dev), _prep(v, dev)
    g, beta = _prep(g, dev, torch.float32), _prep(beta, dev, torch.float32)
    initial_state = _prep(initial_state, dev, torch.float32)
    B, T, H, K = q.shape
    V = v.shape[-1]
    cu_d, cu_h, n_seqs = _cu(cu_seqlens, dev)
    N = n_seqs if cu_d is not None else B
    o = torch.empty((B, T, H, V), device=dev, dtype=out_dtype)
    final_state = torch.empty((N, H, K, V), device=dev, dtype=torch.float32) if output_final_state else None
    states = torch.empty((B, T, H, K, V), device=dev, dtype=torch.float32) if output_states else None
    y = None
    if gate is not None:
        gate, norm_w = _prep(gate, dev), _prep(norm_w, dev, torch.float32)
        y = torch.empty((B, T, H * V), device=dev, dtype=out_dtype)
    if scale is None:
        scale = K ** -0.5
    _check(lib.kda_recurrent_fwd(
        _ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(final_state),
        _ptr(o), _dt(o), _ptr(states), _ptr(cu_d), _ptr(cu_h), n_seqs, B, T, H, K, V, float(scale),
        int(bool(use_qk_l2norm)), _ptr(gate), _dt(gate) if gate is not None else BF16, _ptr(norm_w),
        float(eps), _ptr(y), _stream()))
    out = [o, final_state]
    if output_states:
        out.append(states)
    if gate is not None:
        out.append(y)
    return _to_host(tuple(out), host)


def recurrent_step(q, k, v, g, beta, state, *, scale=None, use_qk_l2norm=True, gate=None, norm_w=None,
                   eps=1e-5, out_dtype=torch.float32, state_out=None, return_o=True, o=None, y=None, conv=None):
    """One decode token per sequence.  q, k [B,H,K]; v [B,H,V]; g [B,H,K]; beta [B,H];
    state [B,H,K,V] fp32 (or None).  ``state_out=state`` updates the state in place.

    ``conv=(weights, states_in[, states_out])`` fuses the q, k, v short convolutions
    (+ SiLU) ahead of the step (K = V = 128): q, k, v are then the raw projections,
    weights three [H*128, W] (or [H*128, 1, W]) filters, states_in three [B, W-1, H*128]
    fp32 histories (or None: zero history), states_out three buffers for the new ones
    (default: fresh; ``states_in`` itself updates them in place).
    Returns (o, state_out[, y][, conv_states_out])."""
    return _step(q, k, v, (g, beta), None, state, scale, use_qk_l2norm, gate, norm_w, eps, out_dtype, state_out,
                 return_o, o, y, conv)


def recurrent_step_logits(q, k, v, g_logits, beta_logits, A_log, state, *, dt_bias=None, g_lower_bound=-5.0,
                          scale=None, use_qk_l2norm=True, gate=None, norm_w=None, eps=1e-5, out_dtype=torch.float32,
                          state_out=None, return_o=True, o=None, y=None, conv=None):
    """recurrent_step with g and beta computed from their logits (see chunk_fwd_logits):
    g_logits [B,H,K], beta_logits [B,H]."""
    lb = float("-inf") if g_lower_bound is None else float(g_lower_bound)
    return _step(q, k, v, None, (g_logits, beta_logits, A_log, dt_bias, lb), state, scale, use_qk_l2norm, gate,
                 norm_w, eps, out_dtype, state_out, return_o, o, y, conv)


def _conv_args(conv, dev, B, H):
    """Marshal the fused convolutions' (weights, states_in[, states_out]) for the C call."""
    weights, s_in = conv[0], conv[1]
    s_out = conv[2] if len(conv) > 2 else None
    if len(weights) != 3 or (s_in is not None and len(s_in) != 3) or (s_out is not None and len(s_out) != 3):
        raise ValueError("conv takes three filters (q, k, v), three histories and three outputs")
    ws = [_prep(w[:, 0, :] if w.dim() == 3 else w, dev, torch.float32) for w in weights]
    W = ws[0].shape[1]
    sin = None if s_in is None else [_prep(x, dev, torch.float32) for x in s_in]
    if s_out is None:
        s_out = [torch.empty((B, W - 1, H * 128), device=dev, dtype=torch.float32) for _ in range(3)]
    P3 = ctypes.c_void_p * 3
    ptr3 = lambda ts: P3(*[t.data_ptr() for t in ts])
    keep = (ws, sin, s_out)  # the tensors stay alive through the call
    return ptr3(ws), W, (ptr3(sin) if sin is not None else None), ptr3(s_out), tuple(s_out), keep


def _step(q, k, v, gb, lg, state, scale, use_qk_l2norm, gate, norm_w, eps, out_dtype, state_out, return_o, o, y,
          conv=None):
    lib = _load()
    host = q.device.type != "cuda"
    dev = _device_of(q, k, v, state)
    q, k, v = _prep(q, dev), _prep(k, dev), _prep(v, dev)
    state = _prep(state, dev, torch.float32)
    B, H, K = q.shape
    V = v.shape[-1]
    if state_out is None:
        state_out = torch.empty((B, H, K, V), device=dev, dtype=torch.float32)
    if gate is not None:
        gate, norm_w = _prep(gate, dev), _prep(norm_w, dev, torch.float32)
        if y is None:
            y = torch.empty((B, H * V), device=dev, dtype=out_dtype)
    if o is None and (return_o or gate is None):
        o = torch.empty((B, H, V), device=dev, dtype=out_dtype)
    if scale is None:
        scale = K ** -0.5
    tail = (_ptr(state), _ptr(state_out), _ptr(o), _dt(o if o is not None else y), B, H, K, V, float(scale),
            int(bool(use_qk_l2norm)), _ptr(gate), _dt(gate) if gate is not None else BF16, _ptr(norm_w), float(eps),
            _ptr(y), _stream())
    if conv is not None:
        cw, W, cin, cout_p, cout, _keep = _conv_args(conv, dev, B, H)
        if lg is None:
            g, beta = _prep(gb[0], dev, torch.float32), _prep(gb[1], dev, torch.float32)
            gates = (_ptr(g), _ptr(beta), None, BF16, None, None, 0.0, None, BF16)
        else:
            z, b, A_log, dt_bias, lb = _logit_args(lg, dev)
            gates = (None, None, _ptr(z), _dt(z), _ptr(A_log), _ptr(dt_bias), lb, _ptr(b), _dt(b))
        _check(lib.kda_recurrent_step_conv(_ptr(q), _ptr(k), _ptr(v), _dt(q), cw, W, cin, cout_p, *gates, *tail))
        res = (o, state_out, y) if gate is not None else (o, state_out)
        if host:
            res = _to_host(res + cout, True)
            return res[:-3] + (res[-3:],)
        return res + (cout,)
    if lg is None:
        g, beta = _prep(gb[0], dev, torch.float32), _prep(gb[1], dev, torch.float32)
        _check(lib.kda_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), *tail))
    else:
        z, b, A_log, dt_bias, lb = _logit_args(lg, dev)
        _check(lib.kda_recurrent_step_logits(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(z), _dt(z), _ptr(A_log),
                                             _ptr(dt_bias), lb, _ptr(b), _dt(b), *tail))
    if gate is not None:
        return _to_host((o, state_out, y), host)
    return _to_host((o, state_out), host)


def gated_rmsnorm(o, gate, w, eps=1e-5, *, out_dtype=torch.float32, y=None):
    """y [.., H*V] = o / sqrt(mean_v(o^2) + eps) * w * sigmoid(gate) over each (token, head)."""
    lib = _load()
    host = o.device.type != "cuda"
    dev = _device_of(o, gate)
    o, gate, w = _prep(o, dev), _prep(gate, dev), _prep(w, dev, torch.float32)
    H, V = o.shape[-2], o.shape[-1]
    rows = o.numel() // (H * V)
    if y is None:
        y = torch.empty(o.shape[:-2] + (H * V,), device=dev, dtype=out_dtype)
    _check(lib.kda_gated_rmsnorm(_ptr(o), _dt(o), _ptr(gate), _dt(gate), _ptr(w), float(eps), _ptr(y), _dt(y),
                                 rows, H, V, _stream()))
    return _to_host((y,), host)[0]


def short_conv(x, weight, bias=None, conv_state=None, *, cu_seqlens=None, activation="silu",
               output_final_state=True, out_dtype=None, y=None, final_state=None):
    """Causal depthwise short convolution (+ SiLU) along the sequence.

    x [B,T,D] (bf16 or fp32); weight [D,W] (or the Conv1d weight [D,1,W]); bias [D] or
    None; conv_state [N,W-1,D] fp32 or None (the W-1 inputs before each sequence,
    oldest first).  With ``cu_seqlens`` B must be 1.  A decode step is T = 1;
    ``final_state=conv_state`` then updates the state in place.
    Returns (y [B,T,D], final_state [N,W-1,D] or None)."""
    lib = _load()
    host = x.device.type != "cuda"
    dev = _device_of(x, conv_state)
    dests = (y, final_state) if host else None
    if host:
        y, final_state = _dev_out(y), _dev_out(final_state)
    x = _prep(x, dev)
    if weight.dim() == 3:
        weight = weight[:, 0, :]
    weight = _prep(weight, dev, torch.float32)
    bias = _prep(bias, dev, torch.float32)
    conv_state = _prep(conv_state, dev, torch.float32)
    B, T, D = x.shape
    W = weight.shape[1]
    cu_d, cu_h, n_seqs = _cu(cu_seqlens, dev)
    N = n_seqs if cu_d is not None else B
    if y is None:
        y = torch.empty((B, T, D), device=dev, dtype=out_dtype or x.dtype)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, W - 1, D), device=dev, dtype=torch.float32)
    act = {"silu": 1, "swish": 1, None: 0, "none": 0, "identity": 0}[activation]
    _check(lib.kda_short_conv_fwd(
        _ptr(x), _dt(x), _ptr(weight), _ptr(bias), _ptr(conv_state), _ptr(final_state), _ptr(y), _dt(y),
        _ptr(cu_d), _ptr(cu_h), n_seqs, B, T, D, W, act, _stream()))
    return _to_host((y, final_state), host, dests)


def o_proj(y, w_o, *, out_dtype=torch.bfloat16, out=None):
    """out [rows, out_features] = y [rows, in_features] @ w_o[out_features, in_features]^T
    (bf16 operands, fp32 accumulation, on the library's tcgen05 GEMM).  y may carry extra
    leading dimensions."""
    lib = _load()
    host = y.device.type != "cuda"
    dev = _device_of(y, w_o)
    y2 = _prep(y, dev, torch.bfloat16).reshape(-1, y.shape[-1])
    w = _prep(w_o, dev, torch.bfloat16)
    rows, K = y2.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("w_o must be [out_features, in_features]")
    dest = out if host else None
    if out is None or host:
        out = torch.empty((rows, N), device=dev, dtype=out_dtype)
    _check(lib.kda_o_proj(_ptr(y2), _ptr(w), _ptr(out), _dt(out), rows, K, N, _stream()))
    res = out.reshape(*y.shape[:-1], N)
    if host:
        return _to_host((res,), True, (dest,))[0]
    return res


# ---------------------------------------------------------------------------
# full attention: rotary positions, the paged 8-bit cache, attention

class KVCache(NamedTuple):
    """A paged 8-bit key/value cache: codes float8_e4m3fn [pages, kv_heads, page_size, dim], one
    power-of-two fp32 scale for each (page, head); a value is code * scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv_cache(num_pages, kv_heads, dim, page_size=64, device=None) -> KVCache:
    """An empty cache on the device (default: the current CUDA device)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    shape = (num_pages, kv_heads, page_size, dim)
    codes = lambda: torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    scale = lambda: torch.ones(shape[:2], dtype=torch.float32, device=device)
    return KVCache(codes(), codes(), scale(), scale())


def rotary_inv_freq(rotary_dim, base=10000.0, *, scaling=None, factor=1.0, original_max_position=4096, beta_fast=32.0,
                    beta_slow=1.0, device=None):
    """(inv_freq, magnitude) for ``rotary`` and ``kv_append``: radians per position of each of the
    rotary_dim / 2 pairs (float64) and the factor on the rotated channels.

    scaling: None; "linear" (positions divided by ``factor``); "ntk" (the base raised to
    base * factor^(R / (R - 2)), R = rotary_dim, so that the slowest pair turns ``factor``
    times slower); "yarn" (a pair that makes at least ``beta_fast`` turns within
    ``original_max_position`` positions is kept, one that makes at most ``beta_slow`` is divided
    by ``factor``, those between are blended linearly in their number of turns; magnitude
    0.1 ln(factor) + 1)."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not 1.0 <= factor < math.inf:
        raise ValueError("factor must be finite and at least 1")
    if not 0.0 < base < math.inf:
        raise ValueError("base must be finite and positive")
    pair = torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** -pair
    magnitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not beta_fast > beta_slow:
            raise ValueError("yarn needs beta_fast > beta_slow")
        turns = original_max_position * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        magnitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return f.to(device), magnitude


_LAYOUTS = {"half": 0, "interleaved": 1}


def _layout(layout):
    if layout not in _LAYOUTS:
        raise ValueError(f'layout must be "half" or "interleaved", not {layout!r}')
    return _LAYOUTS[layout]


# The current device and a device's current stream without torch.cuda's lazy-initialisation
# and type checks, which cost more than a small kernel runs.  (A torch built without CUDA has
# neither, nor any tensor with which a call gets this far.)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(fn, index, *args):
    """One library call on device `index` and its current stream."""
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        _check(status)


def _refuse(t, name, dtype, dim, index):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (index is not None and t.get_device() != index):
        raise ValueError(f"{name} must be a tensor on {'a CUDA device' if index is None else f'cuda:{index}'}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, not {t.dim()}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, name, dtype, dim, index):
    """A small or in-place argument on device `index`: used as it lies, so it has to be
    contiguous -> its address."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.dim() == dim and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, dim, index)


def _rows(t, name, dtype, index):
    """[tokens, heads, dim] on device `index` with dense rows a 16-byte multiple apart (slices of a
    fused projection are used as they lie, anything else is copied) -> (tensor, address, stride)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index or t.dim() != 3 or index < 0:
        _refuse(t, name, dtype, 3, index if index >= 0 else None)
    n, h, d = t.shape
    row, at = h * d, t.data_ptr()
    if at % 16 == 0:
        if t.is_contiguous():
            return t, at, row
        s0, s1, s2 = t.stride()
        if s2 == 1 and (s1 == d or h == 1) and (s0 >= row or n == 1) and s0 * t.element_size() % 16 == 0:
            return t, at, max(s0, row)
    t = t.clone(memory_format=torch.contiguous_format)
    return t, t.data_ptr(), row


def _cache_args(cache):
    """(device index, kv_heads, page_size, dim, (k, v, k_scale, v_scale, pages, page_size))."""
    k, v, ks, vs = cache
    index = k.get_device()
    if index < 0:
        raise ValueError("the cache must lie on a CUDA device")
    ptrs = (_dense(k, "cache.k", torch.float8_e4m3fn, 4, index), _dense(v, "cache.v", torch.float8_e4m3fn, 4, index),
            _dense(ks, "cache.k_scale", torch.float32, 2, index), _dense(vs, "cache.v_scale", torch.float32, 2, index))
    shape = k.shape
    pages, Hk, P, D = shape
    if v.shape != shape or ks.shape != (pages, Hk) or vs.shape != (pages, Hk):
        raise ValueError("the cache's tensors do not fit together: codes [pages, kv_heads, page_size, dim], "
                         "scales [pages, kv_heads]")
    return index, Hk, P, D, (*ptrs, pages, P)


def rotary(x, positions, inv_freq, *, magnitude=1.0, layout="half", inverse=False, out=None):
    """Rotary positions: x [T, H, D] (bf16 or fp32) with the first 2 * len(inv_freq) channels of
    each head turned in pairs by positions[t] * inv_freq[i] and multiplied by ``magnitude``; the
    others are copied.  positions int32 [T] (angles are reduced exactly, however far);
    inv_freq float64 (``rotary_inv_freq``).  layout "half": pairs (i, i + R/2), "interleaved":
    (2i, 2i + 1).  ``inverse`` turns back (the gradient of the call without it).  ``out``:
    a tensor like x, or x itself.  A host x is copied to the device and the result back."""
    lib = _lib or _load()
    lay = _layout(layout)
    if not x.is_cuda:
        dev = _device_of(positions, inv_freq)
        y = rotary(_prep(x, dev), _prep(positions, dev), _prep(inv_freq, dev), magnitude=magnitude, layout=layout,
                   inverse=inverse)
        return _to_host((y,), True, (out,))[0]
    index = x.get_device()
    x, xp, xs = _rows(x, "x", torch.bfloat16 if x.dtype is torch.bfloat16 else torch.float32, index)
    T, H, D = x.shape
    pos = _dense(positions, "positions", torch.int32, 1, index)
    freq = _dense(inv_freq, "inv_freq", torch.float64, 1, index)
    if positions.shape[0] != T:
        raise ValueError("positions must have one entry per token")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        op, os_ = out.data_ptr(), H * D
    else:
        o, op, os_ = _rows(out, "out", x.dtype, index)
        if o is not out or out.shape != x.shape:
            raise ValueError("out must be like x, with dense rows, 16-byte aligned")
    _call(lib.kda_rotary, index, xp, _dt(x), xs, pos, freq, magnitude, 2 * inv_freq.shape[0], lay, 1 if inverse else 0,
          op, os_, T, H, D)
    return out


def kv_append(k, v, cache, block_table, context_lens, *, cu_seqlens=None, inv_freq=None, magnitude=1.0, layout="half",
              q=None, return_k=False, q_out=None, k_out=None):
    """Appends new tokens to a paged 8-bit cache (in place) and rotates their keys and queries.

    k, v [T, kv_heads, dim] bf16 and q [T, q_heads, dim] bf16 (optional) may be slices of a fused
    projection; context_lens int32 [N]: tokens already in the cache; cu_seqlens int32 [N + 1] on
    the device: which rows belong to which sequence, None for one token per sequence (T = N);
    block_table int32 [N, max_blocks].  inv_freq None: no rotation; else the position is the
    token's place in its sequence.  Tokens whose page is negative or out of range are not
    stored.  Returns (rotated q or None, rotated keys if return_k or k_out is given else None).
    Every tensor lies on the cache's device."""
    lib = _lib or _load()
    lay = _layout(layout)
    index, Hk, P, D, cache_args = _cache_args(cache)
    k, kp, k_stride = _rows(k, "k", torch.bfloat16, index)
    v, vp, v_stride = _rows(v, "v", torch.bfloat16, index)
    T, kh, kd = shape = k.shape
    if kh != Hk or kd != D or v.shape != shape:
        raise ValueError("k and v must be [tokens, kv_heads, dim] as the cache is")
    table = _dense(block_table, "block_table", torch.int32, 2, index)
    ctx = _dense(context_lens, "context_lens", torch.int32, 1, index)
    N, max_blocks = block_table.shape
    if context_lens.shape[0] != N:
        raise ValueError("context_lens must have one entry per row of block_table")
    cu = freq = qp = qo = ko = None
    R = Hq = q_stride = 0
    if cu_seqlens is not None:
        cu = _dense(cu_seqlens, "cu_seqlens", torch.int32, 1, index)
        if cu_seqlens.shape[0] != N + 1:
            raise ValueError("cu_seqlens must have one entry more than block_table has rows")
    if inv_freq is not None:
        freq, R = _dense(inv_freq, "inv_freq", torch.float64, 1, index), 2 * inv_freq.shape[0]
    if q is not None:
        q, qp, q_stride = _rows(q, "q", torch.bfloat16, index)
        tq, Hq, dq = q.shape
        if tq != T or dq != D:
            raise ValueError("q must be [tokens, q_heads, dim]")
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        qo = _dense(q_out, "q_out", torch.bfloat16, 3, index)
        if q_out.shape != q.shape:
            raise ValueError("q_out must be like q")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k_out is None and return_k:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    if k_out is not None:
        ko = _dense(k_out, "k_out", torch.bfloat16, 3, index)
        if k_out.shape != shape:
            raise ValueError("k_out must be like k")
    cp = cache_args
    _call(lib.kda_kv_append, index, kp, k_stride, vp, v_stride, T, Hk, D, cp[0], cp[1], cp[2], cp[3], cp[4], P, table,
          max_blocks, ctx, cu, N, freq, magnitude, R, lay, qp, q_stride, Hq, qo, ko)
    return q_out, k_out


def attn_decode_workspace_size(n_seqs, q_heads, kv_heads, dim, max_tokens) -> int:
    """Bytes of workspace one attn_decode call needs; max_tokens: what the block table can hold,
    max_blocks * page_size."""
    return int(_load().kda_attn_decode_workspace_size(int(n_seqs), int(q_heads), int(kv_heads), int(dim), int(max_tokens)))


def attn_decode(q, cache, block_table, seq_lens, *, scale=None, out_dtype=torch.bfloat16, return_lse=False, o=None,
                workspace=None):
    """One query token per sequence over the paged 8-bit cache: q [N, q_heads, dim] bf16 (rows may
    be strided), seq_lens int32 [N] tokens to attend to (the new one included), block_table
    int32 [N, max_blocks].  scale: default dim^-0.5.  Returns o [N, q_heads, dim] (zero for an
    empty sequence, NaN where a needed page number is out of range) or, with return_lse,
    (o, lse [N, q_heads] fp32).  A block_table no wider than the sequences need serves short ones
    faster (they are then not cut into pieces).  workspace: a uint8 tensor of attn_decode_workspace_size(...)
    bytes for this call alone, or None: taken from torch's allocator for the call."""
    lib = _lib or _load()
    index, Hk, P, D, cache_args = _cache_args(cache)
    q, qp, q_stride = _rows(q, "q", torch.bfloat16, index)
    N, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q must be [sequences, q_heads, dim] as the cache is")
    table = _dense(block_table, "block_table", torch.int32, 2, index)
    lens = _dense(seq_lens, "seq_lens", torch.int32, 1, index)
    rows, max_blocks = block_table.shape
    if rows != N or seq_lens.shape[0] != N:
        raise ValueError("block_table and seq_lens must have one row per query")
    device = q.device
    if o is None:
        o = torch.empty((N, Hq, D), dtype=out_dtype, device=device)
    elif o.shape != q.shape:
        raise ValueError("o must be like q")
    lse = torch.empty((N, Hq), dtype=torch.float32, device=device) if return_lse else None
    if workspace is None:
        need, ws = lib.kda_attn_decode_workspace_size(N, Hq, Hk, D, max_blocks * P), None
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
            ws = workspace.data_ptr()
    else:
        need, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
    _call(lib.kda_attn_decode, index, qp, q_stride, *cache_args, table, max_blocks, lens, N, Hq, Hk, D,
          D ** -0.5 if scale is None else float(scale), _dense(o, "o", o.dtype, 3, index), _dt(o),
          None if lse is None else lse.data_ptr(), ws, need)
    return (o, lse) if return_lse else o


def attn_prompt_workspace_size(q_rows, k_rows, q_heads, kv_heads, dim_v, n_seqs=1) -> int:
    """Bytes of workspace with which one attn_prompt call divides its keys among more CTAs; 0
    where it would not."""
    return int(_load().kda_attn_prompt_workspace_size(int(q_rows), int(k_rows), int(q_heads), int(kv_heads), int(dim_v),
                                                      int(n_seqs)))


def attn_prompt(q, k, v, *, cu_seqlens=None, cu_seqlens_k=None, scale=None, out_dtype=torch.bfloat16, return_lse=False,
                o=None, workspace="auto"):
    """Causal attention over whole prompts: q [T, q_heads, D], k [S, kv_heads, D],
    v [S, kv_heads, DV] bf16 (rows may be strided), (D, DV) one of (64, 64), (128, 128),
    (192, 128); query head h reads key/value head h // (q_heads // kv_heads).

    Packed sequences: cu_seqlens int32 [N + 1] on the device gives the queries' rows,
    cu_seqlens_k the keys' (None: the same); without both there is one sequence, or, with
    q [B, T, ..], k and v [B, S, ..], B of equal lengths.  Query i of a sequence sees its first
    i + 1 + (keys - queries) keys: more keys than queries continue a context, and a row that
    sees nothing is zero.  scale: default D^-0.5.  Returns o like q with DV channels or, with
    return_lse, (o, lse) with lse the fp32 log-sum-exp of each row's scores.  Host tensors are
    copied to the device and the results back.

    With few rows and heads the keys are divided among CTAs, whose sums go through a workspace:
    "auto" takes it from torch's allocator for the call; a uint8 tensor of
    attn_prompt_workspace_size(...) bytes is used for this call alone; None goes through every
    row's keys in one go."""
    lib = _lib or _load()
    if not q.is_cuda:
        dev = _device_of(k, v, cu_seqlens, cu_seqlens_k)
        r = attn_prompt(*(_prep(t, dev) for t in (q, k, v)), cu_seqlens=_prep(cu_seqlens, dev),
                        cu_seqlens_k=_prep(cu_seqlens_k, dev), scale=scale, out_dtype=out_dtype, return_lse=return_lse,
                        workspace=workspace)
        r = _to_host(r if return_lse else (r,), True, (o, None))
        return r if return_lse else r[0]
    index, lead, N = q.get_device(), None, 1
    if q.dim() == 4:
        if cu_seqlens is not None or cu_seqlens_k is not None:
            raise ValueError("packed sequences take q, k and v of three dimensions")
        if k.dim() != 4 or v.dim() != 4 or k.shape[0] != q.shape[0] or v.shape[0] != q.shape[0]:
            raise ValueError("q, k and v must have the same batch")
        lead, N = q.shape[:2], q.shape[0]
        q, k, v = q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1)
    q, qp, qs = _rows(q, "q", torch.bfloat16, index)
    k, kp, ks = _rows(k, "k", torch.bfloat16, index)
    v, vp, vs = _rows(v, "v", torch.bfloat16, index)
    T, Hq, D = q.shape
    S, Hk, Dk = k.shape
    Sv, Hv, DV = v.shape
    if Dk != D or Hv != Hk or Sv != S:
        raise ValueError("k must be [keys, kv_heads, D] with q's D, v [keys, kv_heads, DV]")
    cu = cuk = None
    if cu_seqlens is not None:
        cu = _dense(cu_seqlens, "cu_seqlens", torch.int32, 1, index)
        N = cu_seqlens.shape[0] - 1
    if cu_seqlens_k is not None:
        cuk = _dense(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1, index)
        if cu is None or cu_seqlens_k.shape[0] != N + 1:
            raise ValueError("cu_seqlens_k must come with a cu_seqlens of the same length")
    shape = (T, Hq, DV) if lead is None else (*lead, Hq, DV)
    if o is None:
        o = torch.empty(shape, dtype=out_dtype, device=q.device)
    elif o.shape != shape:
        raise ValueError("o must be like q with v's channels")
    lse = torch.empty(shape[:-1], dtype=torch.float32, device=q.device) if return_lse else None
    ws, need = None, 0
    if workspace is not None:
        if S > 128 * N:  # (one block of keys a sequence is never divided)
            need = lib.kda_attn_prompt_workspace_size(T, S, Hq, Hk, DV, N)
        if isinstance(workspace, torch.Tensor):
            if workspace.get_device() != index or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on q's device")
            ws, need = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        elif workspace != "auto":
            raise ValueError('workspace must be "auto", None or a device tensor')
        elif need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    _call(lib.kda_attn_prompt, index, qp, qs, kp, ks, vp, vs, T, S, Hq, Hk, D, DV, cu, cuk, N,
          D ** -0.5 if scale is None else float(scale), _dense(o, "o", o.dtype, len(shape), index), _dt(o),
          None if lse is None else lse.data_ptr(), ws, need)
    return (o, lse) if return_lse else o
