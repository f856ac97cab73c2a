"""Python binding of libkda (ctypes).  Argument marshalling only: every step
of the computation runs in the HIP kernels behind the C ABI of
``include/kda.h``.  PyTorch provides device memory and the stream.

There is no fallback: if libkda.so is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARGUMENT, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_ERR_HIP = range(5)
KDA_DTYPE_F32, KDA_DTYPE_BF16 = 0, 1
KDA_FLAG_L2NORM_QK, KDA_FLAG_BETA_SIGMOID = 1, 2
KDA_ROTARY_INTERLEAVED, KDA_ROTARY_INVERSE = 1, 2
CHUNK = 64  # tokens per chunk of the chunkwise prefill (rows of chunk_states)

# name -> (restype, argtypes) for every entry point of include/kda.h
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_f32, _f64, _u32 = ctypes.c_float, ctypes.c_double, ctypes.c_uint32
SIGNATURES = {
    "kda_prefill_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "kda_prefill": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
                                   _i32, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
    "kda_prefill_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32,
                                      _i32, _i32, ctypes.c_int, ctypes.c_uint32, _vp, _vp, _vp,
                                      _vp, _sz, _vp]),
    "kda_prefill_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32,
                                           _i32, _i32, ctypes.c_int, _vp, _vp, _vp]),
    "kda_decode_step": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                       ctypes.c_int, _vp, _vp]),
    "kda_decode_tokens": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                         _i32, _i32, _i32, _i32, ctypes.c_int, ctypes.c_uint32,
                                         _vp, _vp]),
    "kda_backward_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "kda_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
                                    _i32, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _sz, _vp]),
    "kda_latent_attention": (ctypes.c_int, [_vp, _vp, _vp, _vp]),
    "kda_latent_attention_backward_workspace_bytes": (_sz, [_i64, _i64, _i32, _i32]),
    "kda_latent_attention_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _i64,
                                                     _i64, _vp, _vp, _sz, _vp]),
    "kda_latent_decode_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "kda_latent_decode": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _i64, _i32,
                                         _i32, _i32, _i32, ctypes.c_int, _f32, _vp, _vp, _vp, _sz, _vp]),
    "kda_latent_append": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _vp, _vp, _i64, _i32, _i32, _i32,
                                         ctypes.c_int, _vp, _i64, _vp, _i64, _vp, _f32, _vp, _f32, _u32, _vp,
                                         _vp, _vp]),
    "kda_rotary": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i32, _i32, _i32, _i32,
                                  ctypes.c_int, _f32, _u32, _vp]),
    "kda_rotary_frequencies": (ctypes.c_int, [_i32, _f64, _f64, _i64, ctypes.POINTER(_f32),
                                              ctypes.POINTER(_f32)]),
    "kda_window_attention": (ctypes.c_int, [_vp, _vp, _vp, _vp]),
    "kda_window_attention_backward_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32, _i32, _i32]),
    "kda_window_attention_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp,
                                                     _sz, _vp]),
    "kda_window_decode_workspace_bytes": (_sz, [_i32]),
    "kda_window_decode": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i64, _i32, _i32, _i32, _i32, ctypes.c_int, _i32,
                                         _i32, _f32, _vp, _vp, _vp, _sz, _vp]),
    "kda_kv_append": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i32, _i32, _i32, ctypes.c_int,
                                     _vp, _f32, _vp, _i32, _i32, _f32, _u32, _vp, _vp]),
    "kda_qk_norm_rotary": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, ctypes.c_int, _f32, _f32, _u32,
                                          _vp]),
    "kda_qk_norm_rotary_backward_workspace_bytes": (_sz, [_i32]),
    "kda_qk_norm_rotary_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, ctypes.c_int, _f32,
                                                   _f32, _u32, _vp, _sz, _vp]),
    "kda_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kda_last_error_message": (ctypes.c_char_p, []),
    "kda_version": (_i32, []),
    "kda_set_kernel_timing": (ctypes.c_int, [_i32]),
    "kda_prefill_kernel_times": (_i32, [ctypes.POINTER(ctypes.c_float),
                                        ctypes.POINTER(ctypes.c_char_p), _i32]),
}


class KDAError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {status_string(status)} ({detail})")
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libkda.so (built in-tree by ``gated_delta_rule_prefill_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run "
                              "`python -m gated_delta_rule_prefill_amd.build` (needs hipcc)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def last_error() -> str:
    return lib().kda_last_error_message().decode()


def _check(status: int, where: str) -> None:
    if status != KDA_OK:
        raise KDAError(status, where, last_error())


def workspace_bytes(total_tokens: int, num_seqs: int, H: int, dk: int, dv: int,
                    bf16: bool) -> int:
    return int(lib().kda_prefill_workspace_bytes(int(total_tokens), int(num_seqs), int(H),
                                                 int(dk), int(dv),
                                                 KDA_DTYPE_BF16 if bf16 else KDA_DTYPE_F32))


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDA_DTYPE_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device, stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _flags(l2norm_qk: bool, beta_sigmoid: bool) -> int:
    return (KDA_FLAG_L2NORM_QK if l2norm_qk else 0) | (KDA_FLAG_BETA_SIGMOID if beta_sigmoid else 0)


def num_chunk_states(T: int, N: int, cu_seqlens=None) -> int:
    """Rows of ``chunk_states``: sum over sequences of ceil(len / 64)."""
    if cu_seqlens is None:
        return N * ((T // N + CHUNK - 1) // CHUNK)
    cu = [int(x) for x in cu_seqlens.tolist()]
    return sum((b - a + CHUNK - 1) // CHUNK for a, b in zip(cu[:-1], cu[1:]))


def prefill(q, k, v, log_alpha, beta, initial_state=None, cu_seqlens=None,
            num_seqs: Optional[int] = None, output_final_state: bool = True,
            final_state=None, out=None, workspace=None, stream=None,
            l2norm_qk: bool = False, beta_sigmoid: bool = False, chunk_states=None):
    """Chunkwise KDA prefill of a packed batch (``kda_prefill_ex``).

    q, k: [T, H, dk]; v: [T, H, dv] (bf16 or fp32, same dtype, CUDA/HIP device);
    log_alpha: [T, H, dk] fp32; beta: [T, H] fp32 (logits with beta_sigmoid);
    initial_state: [N, H, dk, dv] fp32 or None; cu_seqlens: [N+1] int32 or None
    (then ``num_seqs`` equal rows, default 1).  ``final_state`` may be the
    same tensor as ``initial_state``.  l2norm_qk / beta_sigmoid: in-kernel
    preprocessing (KDA_FLAG_*).  chunk_states: None, True (allocate) or an fp32
    [NC, H, dk, dv] tensor for the state entering every 64-token chunk.
    Returns (o [T, H, dv], final_state or None), plus chunk_states if asked.
    """
    import torch
    T, H, dk = q.shape
    dv = v.shape[2]
    if cu_seqlens is not None:
        _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1, "cu_seqlens: int32 [N+1]")
        N = cu_seqlens.shape[0] - 1
    else:
        N = int(num_seqs or 1)
    dev = q.device
    for name, t, shape, dt in (("k", k, (T, H, dk), q.dtype), ("v", v, (T, H, dv), q.dtype),
                               ("log_alpha", log_alpha, (T, H, dk), torch.float32),
                               ("beta", beta, (T, H), torch.float32)):
        _require(tuple(t.shape) == shape, f"{name}: expected shape {shape}, got {tuple(t.shape)}")
        _require(t.dtype == dt, f"{name}: expected dtype {dt}, got {t.dtype}")
    tensors = [q, k, v, log_alpha, beta]
    if initial_state is not None:
        _require(tuple(initial_state.shape) == (N, H, dk, dv) and
                 initial_state.dtype == torch.float32, "initial_state: fp32 [N, H, dk, dv]")
        tensors.append(initial_state)
    if cu_seqlens is not None:
        tensors.append(cu_seqlens)
    for t in tensors:
        _require(t.device == dev and t.is_contiguous(), "all inputs: contiguous, on one device")
    if out is None:
        out = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    want_cs = chunk_states is not None and chunk_states is not False
    if chunk_states is True:
        nc = num_chunk_states(T, N, cu_seqlens)
        chunk_states = torch.empty((nc, H, dk, dv), dtype=torch.float32, device=dev)
    elif want_cs:
        nc = num_chunk_states(T, N, cu_seqlens)
        _require(chunk_states.dtype == torch.float32 and chunk_states.is_contiguous() and
                 chunk_states.device == dev and chunk_states.numel() >= nc * H * dk * dv,
                 "chunk_states: contiguous fp32 with room for [NC, H, dk, dv]")
    else:
        chunk_states = None
    need = workspace_bytes(T, N, H, dk, dv, q.dtype == torch.bfloat16)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _require(workspace.numel() * workspace.element_size() >= need, "workspace too small")
    st = lib().kda_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                              _ptr(initial_state), _ptr(cu_seqlens), T, N, H, dk, dv,
                              _dtype_code(q), _flags(l2norm_qk, beta_sigmoid), _ptr(out),
                              _ptr(final_state), _ptr(chunk_states), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(dev, stream))
    _check(st, "kda_prefill_ex")
    return (out, final_state, chunk_states) if want_cs else (out, final_state)


def decode_step(state, q, k, v, log_alpha, beta, out=None, stream=None):
    """One recurrent KDA token per sequence (``kda_decode_step``); ``state``
    (fp32 [N, H, dk, dv]) is updated in place.  Returns o [N, H, dv]."""
    import torch
    N, H, dk, dv = state.shape
    _require(state.dtype == torch.float32 and state.is_contiguous(), "state: contiguous fp32")
    for name, t, shape, dt in (("q", q, (N, H, dk), q.dtype), ("k", k, (N, H, dk), q.dtype),
                               ("v", v, (N, H, dv), q.dtype),
                               ("log_alpha", log_alpha, (N, H, dk), torch.float32),
                               ("beta", beta, (N, H), torch.float32)):
        _require(tuple(t.shape) == shape, f"{name}: expected shape {shape}, got {tuple(t.shape)}")
        _require(t.dtype == dt, f"{name}: expected dtype {dt}")
        _require(t.device == state.device and t.is_contiguous(), f"{name}: contiguous, same device")
    if out is None:
        out = torch.empty((N, H, dv), dtype=q.dtype, device=state.device)
    st = lib().kda_decode_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                               _ptr(beta), N, H, dk, dv, _dtype_code(q), _ptr(out),
                               _stream(state.device, stream))
    _check(st, "kda_decode_step")
    return out


def decode_tokens(state_pool, q, k, v, log_alpha, beta, state_indices=None, cu_seqlens=None,
                  num_seqs: Optional[int] = None, l2norm_qk: bool = False,
                  beta_sigmoid: bool = False, out=None, stream=None):
    """Recurrent KDA over the tokens of a packed batch on pooled states
    (``kda_decode_tokens``).  state_pool: fp32 [P, H, dk, dv], updated in
    place; state_indices: int32 [N] slot per sequence (None = slot s for
    sequence s; a slot outside [0, P) marks padding); tokens as for
    ``prefill``.  Returns o [T, H, dv]."""
    import torch
    P, H, dk, dv = state_pool.shape
    T = q.shape[0]
    dev = state_pool.device
    _require(state_pool.dtype == torch.float32 and state_pool.is_contiguous(),
             "state_pool: contiguous fp32")
    if cu_seqlens is not None:
        _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1, "cu_seqlens: int32 [N+1]")
        N = cu_seqlens.shape[0] - 1
    else:
        N = int(num_seqs or 1)
    for name, t, shape, dt in (("q", q, (T, H, dk), q.dtype), ("k", k, (T, H, dk), q.dtype),
                               ("v", v, (T, H, dv), q.dtype),
                               ("log_alpha", log_alpha, (T, H, dk), torch.float32),
                               ("beta", beta, (T, H), torch.float32)):
        _require(tuple(t.shape) == shape, f"{name}: expected shape {shape}, got {tuple(t.shape)}")
        _require(t.dtype == dt, f"{name}: expected dtype {dt}")
        _require(t.device == dev and t.is_contiguous(), f"{name}: contiguous, same device")
    if state_indices is not None:
        _require(state_indices.dtype == torch.int32 and tuple(state_indices.shape) == (N,) and
                 state_indices.device == dev and state_indices.is_contiguous(),
                 "state_indices: int32 [N] on the same device")
    if cu_seqlens is not None:
        _require(cu_seqlens.device == dev and cu_seqlens.is_contiguous(), "cu_seqlens: same device")
    if out is None:
        out = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    st = lib().kda_decode_tokens(_ptr(state_pool), P, _ptr(state_indices), _ptr(q), _ptr(k),
                                 _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(cu_seqlens), T, N,
                                 H, dk, dv, _dtype_code(q), _flags(l2norm_qk, beta_sigmoid),
                                 _ptr(out), _stream(dev, stream))
    _check(st, "kda_decode_tokens")
    return out


def backward_workspace_bytes(total_tokens: int, num_seqs: int, H: int, dk: int, dv: int,
                             bf16: bool) -> int:
    return int(lib().kda_backward_workspace_bytes(int(total_tokens), int(num_seqs), int(H),
                                                  int(dk), int(dv),
                                                  KDA_DTYPE_BF16 if bf16 else KDA_DTYPE_F32))


def backward(q, k, v, log_alpha, beta, d_o, initial_state=None, cu_seqlens=None,
             num_seqs: Optional[int] = None, d_final_state=None, chunk_states=None,
             need_initial_state_grad: bool = True, workspace=None, stream=None) -> dict:
    """Gradients of ``prefill`` (``kda_backward``): for dL/do = d_o and
    dL/dfinal_state = d_final_state (or zero) returns dq, dk, dv (q/k/v dtype),
    dlog_alpha, dbeta and dinitial_state (fp32).  chunk_states: the forward's
    exported chunk states, or None to recompute them."""
    import torch
    T, H, dk = q.shape
    dv = v.shape[2]
    if cu_seqlens is not None:
        _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1, "cu_seqlens: int32 [N+1]")
        N = cu_seqlens.shape[0] - 1
    else:
        N = int(num_seqs or 1)
    dev = q.device
    for name, t, shape, dt in (("k", k, (T, H, dk), q.dtype), ("v", v, (T, H, dv), q.dtype),
                               ("log_alpha", log_alpha, (T, H, dk), torch.float32),
                               ("beta", beta, (T, H), torch.float32),
                               ("d_o", d_o, (T, H, dv), q.dtype)):
        _require(tuple(t.shape) == shape, f"{name}: expected shape {shape}, got {tuple(t.shape)}")
        _require(t.dtype == dt, f"{name}: expected dtype {dt}, got {t.dtype}")
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            _require(tuple(t.shape) == (N, H, dk, dv) and t.dtype == torch.float32,
                     f"{name}: fp32 [N, H, dk, dv]")
    if chunk_states is not None:
        _require(chunk_states.dtype == torch.float32 and
                 chunk_states.numel() >= num_chunk_states(T, N, cu_seqlens) * H * dk * dv,
                 "chunk_states: fp32 [NC, H, dk, dv]")
    for t in (q, k, v, log_alpha, beta, d_o, initial_state, cu_seqlens, d_final_state, chunk_states):
        if t is not None:
            _require(t.device == dev and t.is_contiguous(), "all inputs: contiguous, on one device")
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dlog_alpha=torch.empty_like(log_alpha), dbeta=torch.empty_like(beta),
               dinitial_state=torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
               if need_initial_state_grad else None)
    need = backward_workspace_bytes(T, N, H, dk, dv, q.dtype == torch.bfloat16)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _require(workspace.numel() * workspace.element_size() >= need, "workspace too small")
    st = lib().kda_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                            _ptr(initial_state), _ptr(cu_seqlens), T, N, H, dk, dv,
                            _dtype_code(q), _ptr(d_o), _ptr(d_final_state), _ptr(chunk_states),
                            _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                            _ptr(out["dlog_alpha"]), _ptr(out["dbeta"]),
                            _ptr(out["dinitial_state"]), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(dev, stream))
    _check(st, "kda_backward")
    return out


def set_kernel_timing(enabled: bool) -> None:
    _check(lib().kda_set_kernel_timing(1 if enabled else 0), "kda_set_kernel_timing")


def prefill_kernel_times():
    """[(kernel name, ms)] of the last prefill recorded with timing enabled on
    this thread, in launch order (a long batch runs its kernels once per segment)."""
    ms = (ctypes.c_float * 256)()
    names = (ctypes.c_char_p * 256)()
    n = min(lib().kda_prefill_kernel_times(ms, names, 256), 256)
    if n < 0:
        raise RuntimeError("no timed prefill recorded")
    return [(names[i].decode(), float(ms[i])) for i in range(n)]


# -- latent attention ------------------------------------------------------------

# A decode step makes several of these calls per layer, so they look torch up
# once, compare before they word a message, and enter a context only where one
# is needed.

_torch = None


def _lib_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


_CODES = {}   # torch dtype -> KDA_DTYPE_*, filled on first use


def _code(t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        code = _CODES[t.dtype] = _dtype_code(t)
    return code


def _elsewhere(device, stream):
    """Context that a call must enter: its stream argument's, or its tensors'
    device's; None where they are on the current device and stream.  Outputs and
    workspaces the binding allocates belong to the stream the call runs on."""
    torch = _torch or _lib_torch()
    index = device.index   # None on the CPU
    if stream is None and index is not None and index == torch._C._cuda_getDevice():
        return None
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream: it belongs to {stream.device}, the tensors are on {device}")
        return torch.cuda.stream(stream)
    return torch.cuda.device(device)


def _raw_stream(device) -> int:
    return _torch._C._cuda_getCurrentRawStream(device.index)


def _rows3(t, name, shape, dtype, device) -> None:
    """A tensor whose last axis is dense."""
    if (t.shape == shape and t.dtype is dtype and t.device == device and
            (t.stride(-1) == 1 or shape[-1] == 1 or t.numel() == 0)):
        return
    raise ValueError(f"{name}: expected {dtype} {shape} on {device} with a dense last axis, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _stride(t, axis: int) -> int:
    """Elements from one index of an axis to the next (0 for an axis of one)."""
    return t.stride(axis) if t.shape[axis] > 1 else 0


def _dense(t, name, shape, dtype, device) -> None:
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {shape} on {device}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _offsets(cu, name, device) -> int:
    if (cu.dtype is (_torch or _lib_torch()).int32 and cu.dim() == 1 and cu.shape[0] >= 2 and cu.device == device and
            cu.is_contiguous()):
        return cu.shape[0] - 1
    raise ValueError(f"{name}: expected contiguous int32 [N+1] on {device}, got {cu.dtype} {tuple(cu.shape)} "
                     f"on {cu.device}")


_INPUTS = struct.Struct("@4P7q2P2q7if")   # kda_latent_inputs of include/kda.h


def _latent_inputs(q, k, v, k_pe, cu_seqlens, cu_seqlens_k, num_seqs, causal, scale):
    """The packed kda_latent_inputs, and (T, Tk, H, dn, dr, dv)."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v: [tokens, heads, channels]")
    T, H, dqk = q.shape
    Tk, _, dn = k.shape
    dv = v.shape[2]
    dev, dt = q.device, q.dtype
    dr = dqk - dn
    if dr < 0:
        raise ValueError("q must have at least k's channels")
    _rows3(q, "q", (T, H, dqk), dt, dev)
    _rows3(k, "k", (Tk, H, dn), dt, dev)
    _rows3(v, "v", (Tk, H, dv), dt, dev)
    pe = pes = 0
    if dr:
        if k_pe is None:
            raise ValueError("q has channels beyond k's: k_pe is needed")
        _rows3(k_pe, "k_pe", (Tk, dr), dt, dev)
        pe, pes = k_pe.data_ptr(), _stride(k_pe, 0)
    elif k_pe is not None:
        raise ValueError("k_pe: q has no channels for it")
    cu = cuk = 0
    if cu_seqlens is not None:
        N = _offsets(cu_seqlens, "cu_seqlens", dev)
        cu = cu_seqlens.data_ptr()
        if cu_seqlens_k is not None:
            if cu_seqlens_k is not cu_seqlens and _offsets(cu_seqlens_k, "cu_seqlens_k", dev) != N:
                raise ValueError("cu_seqlens_k: as many sequences as cu_seqlens")
            cuk = cu_seqlens_k.data_ptr()
    else:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        N = 1 if num_seqs is None else int(num_seqs)
    if scale is None:
        scale = dqk ** -0.5
    packed = _INPUTS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), pe, _stride(q, 0), _stride(q, 1),
                          _stride(k, 0), _stride(k, 1), _stride(v, 0), _stride(v, 1), pes, cu, cuk, T, Tk, N, H, dn,
                          dr, dv, _code(q), 1 if causal else 0, scale)
    return packed, (T, Tk, H, dn, dr, dv)


def latent_attention(q, k, v, k_pe=None, cu_seqlens=None, cu_seqlens_k=None, num_seqs: Optional[int] = None,
                     causal: bool = True, scale: Optional[float] = None, out=None, lse=None, stream=None):
    """Expanded latent attention over packed sequences (``kda_latent_attention``).

    q: [T, H, dn + dr]; k: [Tk, H, dn]; v: [Tk, H, dn] (bf16 or fp32; strided
    views, e.g. the halves of one expansion product); k_pe: [Tk, dr], the rotary
    key part shared by the heads, or None with dr = 0.  cu_seqlens (and
    cu_seqlens_k where the keys are more than the queries): int32 [N+1], or
    ``num_seqs`` equal rows.  scale: default (dn + dr)^-0.5.
    Returns (o [T, H, dn], lse [T, H] fp32).  Rows behind the last sequence are
    left as they were."""
    packed, (T, _, H, _, _, dv) = _latent_inputs(q, k, v, k_pe, cu_seqlens, cu_seqlens_k, num_seqs, causal, scale)
    dev = q.device
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return latent_attention(q, k, v, k_pe, cu_seqlens, cu_seqlens_k, num_seqs, causal, scale, out, lse)
    torch = _torch
    if out is None:
        out = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    else:
        _dense(out, "out", (T, H, dv), q.dtype, dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    else:
        _dense(lse, "lse", (T, H), torch.float32, dev)
    st = lib().kda_latent_attention(packed, out.data_ptr(), lse.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "kda_latent_attention")
    return out, lse


def latent_attention_backward(q, k, v, o, lse, d_o, k_pe=None, cu_seqlens=None, cu_seqlens_k=None,
                              num_seqs: Optional[int] = None, causal: bool = True, scale: Optional[float] = None,
                              dk=None, dv=None, workspace=None, stream=None) -> dict:
    """Gradients of ``latent_attention`` (``kda_latent_attention_backward``) for
    dL/do = d_o, from the forward's o and lse: returns dq [T, H, dn + dr], dk and
    dv [Tk, H, dn] and dk_pe [Tk, dr] or None, in the inputs' type.  dk, dv:
    tensors to write (strided, e.g. the halves of one [Tk, H, 2 dn] gradient),
    or None to allocate both halves of one such tensor."""
    packed, (T, Tk, H, dn, dr, dvw) = _latent_inputs(q, k, v, k_pe, cu_seqlens, cu_seqlens_k, num_seqs, causal, scale)
    dev, dt = q.device, q.dtype
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return latent_attention_backward(q, k, v, o, lse, d_o, k_pe, cu_seqlens, cu_seqlens_k, num_seqs, causal,
                                             scale, dk, dv, workspace)
    torch = _torch
    _dense(o, "o", (T, H, dvw), dt, dev)
    _dense(d_o, "d_o", (T, H, dvw), dt, dev)
    _dense(lse, "lse", (T, H), torch.float32, dev)
    if dk is None and dv is None:
        dkv = torch.empty((Tk, H, dn + dvw), dtype=dt, device=dev)
        dk, dv = dkv[..., :dn], dkv[..., dn:]
    else:
        _require(dk is not None and dv is not None, "dk and dv: both or neither")
        _rows3(dk, "dk", (Tk, H, dn), dt, dev)
        _rows3(dv, "dv", (Tk, H, dvw), dt, dev)
    dq = torch.empty((T, H, dn + dr), dtype=dt, device=dev)
    dk_pe = torch.empty((Tk, dr), dtype=dt, device=dev) if dr else None
    if workspace is None:
        workspace = torch.empty(lib().kda_latent_attention_backward_workspace_bytes(T, Tk, H, dr), dtype=torch.uint8,
                                device=dev)
    else:
        _require(workspace.device == dev and workspace.is_contiguous(), "workspace: contiguous, same device")
    st = lib().kda_latent_attention_backward(
        packed, o.data_ptr(), lse.data_ptr(), d_o.data_ptr(), dq.data_ptr(), dk.data_ptr(), _stride(dk, 0),
        _stride(dk, 1), dv.data_ptr(), _stride(dv, 0), _stride(dv, 1), _ptr(dk_pe), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(dev))
    if st:
        _check(st, "kda_latent_attention_backward")
    return dict(dq=dq, dk=dk, dv=dv, dk_pe=dk_pe)


def _paged(cache, block_table, seq_lens, cu_seqlens, num_seqs) -> int:
    """Number of sequences of a paged call, with its shared arguments checked."""
    int32, dev = _lib_torch().int32, cache.device
    if cache.dim() != 3 or not cache.is_contiguous():
        raise ValueError("cache: contiguous [pages, page_size, channels]")
    if cu_seqlens is not None:
        N = _offsets(cu_seqlens, "cu_seqlens", dev)
    else:
        N = int(num_seqs) if num_seqs is not None else seq_lens.shape[0]
    if not (block_table.dtype is int32 and block_table.dim() == 2 and block_table.shape[0] == N and
            block_table.device == dev and block_table.is_contiguous()):
        raise ValueError("block_table: contiguous int32 [N, max_pages], on the cache's device")
    _dense(seq_lens, "seq_lens", (N,), int32, dev)
    return N


def latent_decode_workspace_bytes(total_tokens: int, num_seqs: int, H: int, dl: int, dr: int, bf16: bool) -> int:
    return int(lib().kda_latent_decode_workspace_bytes(int(total_tokens), int(num_seqs), int(H), int(dl), int(dr),
                                                       KDA_DTYPE_BF16 if bf16 else KDA_DTYPE_F32))


def latent_decode(q, cache, block_table, seq_lens, latent_dim: int, scale: float, cu_seqlens=None,
                  num_seqs: Optional[int] = None, out=None, lse=None, workspace=None, stream=None):
    """Absorbed latent attention over a paged cache (``kda_latent_decode``).

    q: [T, H, dl + dr], the queries multiplied into the latent space and their
    rotated part (strided); cache: [pages, page_size, dl + dr], rows as
    ``latent_append`` writes them; block_table: int32 [N, max_pages]; seq_lens:
    int32 [N] cached tokens, the new ones included; cu_seqlens: int32 [N+1]
    offsets of the new tokens, or None for T / N each.  latent_dim = dl; scale:
    of the heads before absorption, e.g. (dn + dr)^-0.5.
    Returns (o [T, H, dl], lse [T, H] fp32)."""
    if q.dim() != 3:
        raise ValueError("q: [T, H, dl + dr]")
    T, H, width = q.shape
    N = _paged(cache, block_table, seq_lens, cu_seqlens, num_seqs)
    dev, dt = cache.device, cache.dtype
    P, page, cw = cache.shape
    _rows3(q, "q", (T, H, cw), dt, dev)
    dl = int(latent_dim)
    dr, code = width - dl, _code(q)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return latent_decode(q, cache, block_table, seq_lens, latent_dim, scale, cu_seqlens, num_seqs, out, lse,
                                 workspace)
    torch = _torch
    if out is None:
        out = torch.empty((T, H, dl), dtype=dt, device=dev)
    else:
        _dense(out, "out", (T, H, dl), dt, dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    else:
        _dense(lse, "lse", (T, H), torch.float32, dev)
    handle = lib()
    if workspace is None:
        need = handle.kda_latent_decode_workspace_bytes(T, N, H, dl, dr, code)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _require(workspace.device == dev and workspace.is_contiguous(), "workspace: contiguous, same device")
        need = workspace.numel() * workspace.element_size()
    st = handle.kda_latent_decode(
        q.data_ptr(), _stride(q, 0), _stride(q, 1), cache.data_ptr(), P, page, block_table.data_ptr(),
        block_table.shape[1], seq_lens.data_ptr(), _ptr(cu_seqlens), T, N, H, dl, dr, code, scale, out.data_ptr(),
        lse.data_ptr(), workspace.data_ptr() or None, need, _raw_stream(dev))
    if st:
        _check(st, "kda_latent_decode")
    return out, lse


def latent_append(cache, c, block_table, seq_lens, k_pe=None, cu_seqlens=None, num_seqs: Optional[int] = None,
                  norm_weight=None, eps: float = 1e-6, inv_freq=None, interleaved: bool = False,
                  mscale: float = 1.0, c_out=None, k_pe_out=None, stream=None):
    """Write the new tokens' rows of a paged latent cache (``kda_latent_append``).

    cache, block_table, seq_lens, cu_seqlens: as for ``latent_decode`` (seq_lens
    counts the new tokens).  c: [T, dl] latents and k_pe: [T, dr] rotary key
    parts (strided rows, e.g. parts of one down projection; k_pe None with
    dr = 0).  norm_weight: fp32 [dl] of the RMS norm, or None for no norm;
    inv_freq: fp32 [dr / 2], or None for no rotation; mscale multiplies the
    rotated part.  c_out, k_pe_out: True (allocate) or a dense tensor for the
    normalised latents and rotated key parts.  Returns (c_out, k_pe_out)."""
    if c.dim() != 2:
        raise ValueError("c: [T, dl]")
    T, dl = c.shape
    N = _paged(cache, block_table, seq_lens, cu_seqlens, num_seqs)
    dev, dt, float32 = cache.device, cache.dtype, _torch.float32
    P, page, width = cache.shape
    dr = width - dl
    _rows3(c, "c", (T, dl), dt, dev)
    pe = pes = None
    if dr:
        if k_pe is None:
            raise ValueError("the cache has channels beyond c's: k_pe is needed")
        _rows3(k_pe, "k_pe", (T, dr), dt, dev)
        pe, pes = k_pe.data_ptr(), _stride(k_pe, 0)
    elif k_pe is not None:
        raise ValueError("k_pe: the cache has no channels for it")
    if norm_weight is not None:
        _dense(norm_weight, "norm_weight", (dl,), float32, dev)
    if inv_freq is not None:
        _dense(inv_freq, "inv_freq", (dr // 2,), float32, dev)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return latent_append(cache, c, block_table, seq_lens, k_pe, cu_seqlens, num_seqs, norm_weight, eps,
                                 inv_freq, interleaved, mscale, c_out, k_pe_out)
    if c_out is True:
        c_out = _torch.empty((T, dl), dtype=dt, device=dev)
    elif c_out is None or c_out is False:
        c_out = None
    else:
        _dense(c_out, "c_out", (T, dl), dt, dev)
    if k_pe_out is True:
        k_pe_out = _torch.empty((T, dr), dtype=dt, device=dev)
    elif k_pe_out is None or k_pe_out is False:
        k_pe_out = None
    else:
        _dense(k_pe_out, "k_pe_out", (T, dr), dt, dev)
    st = lib().kda_latent_append(
        cache.data_ptr(), P, page, block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
        _ptr(cu_seqlens), T, N, dl, dr, _code(cache), c.data_ptr(), _stride(c, 0), pe, pes or 0, _ptr(norm_weight), eps,
        _ptr(inv_freq), mscale, KDA_ROTARY_INTERLEAVED if interleaved else 0, _ptr(c_out), _ptr(k_pe_out),
        _raw_stream(dev))
    if st:
        _check(st, "kda_latent_append")
    return c_out, k_pe_out


def rotary(x, positions, inv_freq, start: int = 0, interleaved: bool = False, mscale: float = 1.0,
           inverse: bool = False, out=None, stream=None):
    """Rotary positions on channels [start, start + 2 len(inv_freq)) of every
    head (``kda_rotary``).  x: [T, H, d] (last axis dense, otherwise strided);
    positions: int32 [T]; inv_freq: fp32 [dr / 2]; inverse: the gradient of the
    rotation.  out: None (allocate), x itself (in place), or a [T, H, d] tensor
    that does not overlap x.  Returns the rotated tensor."""
    if x.dim() != 3 or inv_freq.dim() != 1:
        raise ValueError("x: [T, H, d]; inv_freq: [dr / 2]")
    torch = _lib_torch()
    T, H, d = x.shape
    dev, dt = x.device, x.dtype
    _rows3(x, "x", (T, H, d), dt, dev)
    _dense(positions, "positions", (T,), torch.int32, dev)
    half = inv_freq.shape[0]
    _dense(inv_freq, "inv_freq", (half,), torch.float32, dev)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return rotary(x, positions, inv_freq, start, interleaved, mscale, inverse, out)
    if out is None:
        out = torch.empty((T, H, d), dtype=dt, device=dev)
    else:
        _rows3(out, "out", (T, H, d), dt, dev)
    st = lib().kda_rotary(x.data_ptr(), _stride(x, 0), _stride(x, 1), out.data_ptr(), _stride(out, 0), _stride(out, 1),
                          positions.data_ptr(), inv_freq.data_ptr(), T, H, d, start, 2 * half, _code(x), mscale,
                          (KDA_ROTARY_INTERLEAVED if interleaved else 0) | (KDA_ROTARY_INVERSE if inverse else 0),
                          _raw_stream(dev))
    if st:
        _check(st, "kda_rotary")
    return out


def rotary_frequencies(dr: int, base: float = 10000.0, factor: float = 1.0, original_context: int = 0,
                       device=None):
    """(inv_freq fp32 [dr / 2], amplitude) for ``rotary`` and ``latent_append``
    (``kda_rotary_frequencies``): plain frequencies, or a context stretched by
    ``factor`` -- linearly, or by parts with ``original_context``."""
    import torch
    f = (_f32 * max(1, dr // 2))()
    a = _f32()
    _check(lib().kda_rotary_frequencies(dr, base, factor, original_context, f, ctypes.byref(a)),
           "kda_rotary_frequencies")
    return torch.tensor(list(f), dtype=torch.float32, device=device), float(a.value)


# -- window attention --------------------------------------------------------------

_WINDOW = struct.Struct("@3P6q2P2q7if")            # kda_window_inputs of include/kda.h
_KV_CACHE = struct.Struct("@2P3q2P3i4x")           # kda_kv_cache
_NORM_HEADS = struct.Struct("@P2qP2q2P2qP2qPi4x")  # kda_norm_heads


def _int32(x, name) -> int:
    if type(x) is not int:
        x = int(x)
    if not -2147483648 <= x <= 2147483647:
        raise ValueError(f"{name}: {x} does not fit in 32 bits")
    return x


def _strides3(t, name, T, H, d, dtype, device):
    """Token and head strides of a [T, H, d] tensor whose last axis is dense (0 for
    an axis of one)."""
    s = t.stride()
    if (t.shape == (T, H, d) and t.dtype is dtype and t.device == device and
            (s[2] == 1 or d == 1 or T == 0 or H == 0 or d == 0)):
        return (s[0] if T > 1 else 0), (s[1] if H > 1 else 0)
    raise ValueError(f"{name}: expected {dtype} {(T, H, d)} on {device} with a dense last axis, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}, strides {s}")


def _window_inputs(q, k, v, window, sinks, cu_seqlens, cu_seqlens_k, num_seqs, scale):
    """The packed kda_window_inputs, and (T, Tk, N, H, Hk, d)."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k, v: [tokens, heads, channels]")
    T, H, d = q.shape
    Tk, Hk, _ = k.shape
    dev, dt = q.device, q.dtype
    qt, qh = _strides3(q, "q", T, H, d, dt, dev)
    kt, kh = _strides3(k, "k", Tk, Hk, d, dt, dev)
    vt, vh = _strides3(v, "v", Tk, Hk, d, dt, dev)
    cu = cuk = 0
    if cu_seqlens is not None:
        N = _offsets(cu_seqlens, "cu_seqlens", dev)
        cu = cu_seqlens.data_ptr()
        if cu_seqlens_k is not None:
            if cu_seqlens_k is not cu_seqlens and _offsets(cu_seqlens_k, "cu_seqlens_k", dev) != N:
                raise ValueError("cu_seqlens_k: as many sequences as cu_seqlens")
            cuk = cu_seqlens_k.data_ptr()
    else:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        N = 1 if num_seqs is None else _int32(num_seqs, "num_seqs")
    if scale is None:
        scale = d ** -0.5
    packed = _WINDOW.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), qt, qh, kt, kh, vt, vh, cu, cuk, T, Tk, N, H, Hk, d,
                          _code(q), _int32(window, "window"), _int32(sinks, "sinks"), scale)
    return packed, (T, Tk, N, H, Hk, d)


def window_attention(q, k, v, window: int, sinks: int = 0, cu_seqlens=None, cu_seqlens_k=None,
                     num_seqs: Optional[int] = None, scale: Optional[float] = None, out=None, lse=None, stream=None):
    """Attention over a window of the last ``window`` tokens, the row's own
    included, and the first ``sinks`` of its sequence, packed sequences
    (``kda_window_attention``).

    q: [T, H, d]; k, v: [Tk, Hk, d], H a multiple of Hk (bf16 or fp32; strided
    views, e.g. parts of one projection).  cu_seqlens (and cu_seqlens_k where the
    keys are more than the queries): int32 [N+1], or ``num_seqs`` equal rows.
    scale: default d^-0.5.  Returns (o [T, H, d], lse [T, H] fp32).  Rows behind
    the last sequence are left as they were."""
    packed, (T, _, _, H, _, d) = _window_inputs(q, k, v, window, sinks, cu_seqlens, cu_seqlens_k, num_seqs, scale)
    dev = q.device
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return window_attention(q, k, v, window, sinks, cu_seqlens, cu_seqlens_k, num_seqs, scale, out, lse)
    torch = _torch
    if out is None:
        out = q.new_empty(T, H, d)
    else:
        _dense(out, "out", (T, H, d), q.dtype, dev)
    if lse is None:
        lse = q.new_empty((T, H), dtype=torch.float32)
    else:
        _dense(lse, "lse", (T, H), torch.float32, dev)
    st = lib().kda_window_attention(packed, out.data_ptr(), lse.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "kda_window_attention")
    return out, lse


def window_attention_backward_workspace_bytes(total_q: int, num_seqs: int, H: int, Hk: int, d: int, sinks: int) -> int:
    return int(lib().kda_window_attention_backward_workspace_bytes(int(total_q), int(num_seqs), int(H), int(Hk),
                                                                   int(d), int(sinks)))


def window_attention_backward(q, k, v, o, lse, d_o, window: int, sinks: int = 0, cu_seqlens=None, cu_seqlens_k=None,
                              num_seqs: Optional[int] = None, scale: Optional[float] = None, dk=None, dv=None,
                              workspace=None, stream=None) -> dict:
    """Gradients of ``window_attention`` (``kda_window_attention_backward``) for
    dL/do = d_o, from the forward's o and lse: returns dq [T, H, d], dk and dv
    [Tk, Hk, d], in the inputs' type.  dk, dv: tensors to write (strided, e.g. parts
    of one gradient), or None to allocate both as the halves of one [Tk, 2 Hk, d]
    tensor."""
    packed, (T, Tk, N, H, Hk, d) = _window_inputs(q, k, v, window, sinks, cu_seqlens, cu_seqlens_k, num_seqs, scale)
    dev, dt = q.device, q.dtype
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return window_attention_backward(q, k, v, o, lse, d_o, window, sinks, cu_seqlens, cu_seqlens_k, num_seqs,
                                             scale, dk, dv, workspace)
    torch = _torch
    _dense(o, "o", (T, H, d), dt, dev)
    _dense(d_o, "d_o", (T, H, d), dt, dev)
    _dense(lse, "lse", (T, H), torch.float32, dev)
    if dk is None and dv is None:
        dkv = q.new_empty(Tk, 2 * Hk, d)
        dk, dv = dkv[:, :Hk], dkv[:, Hk:]
    else:
        _require(dk is not None and dv is not None, "dk and dv: both or neither")
        _rows3(dk, "dk", (Tk, Hk, d), dt, dev)
        _rows3(dv, "dv", (Tk, Hk, d), dt, dev)
    dq = q.new_empty(T, H, d)
    handle = lib()
    if workspace is None:
        need = handle.kda_window_attention_backward_workspace_bytes(T, N, H, Hk, d, sinks)
        workspace = q.new_empty(need, dtype=torch.uint8)
    else:
        _require(workspace.device == dev and workspace.is_contiguous(), "workspace: contiguous, same device")
        need = workspace.numel() * workspace.element_size()
    st = handle.kda_window_attention_backward(
        packed, o.data_ptr(), lse.data_ptr(), d_o.data_ptr(), dq.data_ptr(), dk.data_ptr(), _stride(dk, 0),
        _stride(dk, 1), dv.data_ptr(), _stride(dv, 0), _stride(dv, 1), workspace.data_ptr() or None, need,
        _raw_stream(dev))
    if st:
        _check(st, "kda_window_attention_backward")
    return dict(dq=dq, dk=dk, dv=dv)


def _kv_cache(k_cache, v_cache, block_table, seq_lens, cu_seqlens, num_seqs):
    """The packed kda_kv_cache, the number of sequences, and the cache's heads and
    channels, type and device."""
    int32, dev, dt, shape, s = _lib_torch().int32, k_cache.device, k_cache.dtype, k_cache.shape, k_cache.stride()
    if len(shape) != 4 or not (s[3] == 1 or shape[3] == 1):
        raise ValueError("k_cache: [pages, page_size, heads, channels] with a dense last axis")
    if not (v_cache.shape == shape and v_cache.stride() == s and v_cache.dtype is dt and v_cache.device == dev):
        raise ValueError("v_cache: shape, strides, type and device of k_cache")
    if cu_seqlens is not None:
        N = _offsets(cu_seqlens, "cu_seqlens", dev)
    else:
        N = _int32(num_seqs, "num_seqs") if num_seqs is not None else seq_lens.shape[0]
    rows = block_table.shape
    if not (len(rows) == 2 and rows[0] == N and block_table.dtype is int32 and block_table.device == dev and
            block_table.is_contiguous()):
        raise ValueError("block_table: contiguous int32 [N, max_pages], on the cache's device")
    _dense(seq_lens, "seq_lens", (N,), int32, dev)
    P, page, H, d = shape
    packed = _KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), s[0] if P > 1 else 0, s[1] if page > 1 else 0,
                            s[2] if H > 1 else 0, block_table.data_ptr(), seq_lens.data_ptr(), P, page, rows[1])
    return packed, N, H, d, dt, dev


def window_decode_workspace_bytes(d: int) -> int:
    return int(lib().kda_window_decode_workspace_bytes(int(d)))


def window_decode(q, k_cache, v_cache, block_table, seq_lens, window: int, sinks: int = 0,
                  scale: Optional[float] = None, cu_seqlens=None, num_seqs: Optional[int] = None, out=None, lse=None,
                  workspace=None, stream=None):
    """``window_attention`` of new tokens over a paged cache that already holds
    them (``kda_window_decode``).

    q: [T, H, d] (strided); k_cache, v_cache: [pages, page_size, Hk, d], two views
    of the same strides (e.g. a [pages, Hk, page_size, d] tensor with two axes
    swapped, or halves of one tensor); block_table: int32 [N, max_pages], a page
    outside the pool marks absent tokens; seq_lens: int32 [N] cached tokens, the new
    ones included; cu_seqlens: int32 [N+1] offsets of the new tokens, or None for
    T / N each.  Returns (o [T, H, d], lse [T, H] fp32)."""
    if q.dim() != 3:
        raise ValueError("q: [T, H, d]")
    T, H, _ = q.shape
    cache, N, Hk, d, dt, dev = _kv_cache(k_cache, v_cache, block_table, seq_lens, cu_seqlens, num_seqs)
    qt, qh = _strides3(q, "q", T, H, d, dt, dev)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return window_decode(q, k_cache, v_cache, block_table, seq_lens, window, sinks, scale, cu_seqlens, num_seqs,
                                 out, lse, workspace)
    torch = _torch
    if out is None:
        out = q.new_empty(T, H, d)
    else:
        _dense(out, "out", (T, H, d), dt, dev)
    if lse is None:
        lse = q.new_empty((T, H), dtype=torch.float32)
    else:
        _dense(lse, "lse", (T, H), torch.float32, dev)
    handle = lib()
    if workspace is None:
        need = handle.kda_window_decode_workspace_bytes(d)
        workspace = q.new_empty(need, dtype=torch.uint8)
    else:
        _require(workspace.device == dev and workspace.is_contiguous(), "workspace: contiguous, same device")
        need = workspace.numel() * workspace.element_size()
    st = handle.kda_window_decode(
        cache, q.data_ptr(), qt, qh, None if cu_seqlens is None else cu_seqlens.data_ptr(), T, N, H, Hk, d, _code(q),
        _int32(window, "window"), _int32(sinks, "sinks"), d ** -0.5 if scale is None else scale, out.data_ptr(),
        lse.data_ptr(), workspace.data_ptr() or None, need, _raw_stream(dev))
    if st:
        _check(st, "kda_window_decode")
    return out, lse


def kv_append(k_cache, v_cache, k, v, block_table, seq_lens, cu_seqlens=None, num_seqs: Optional[int] = None,
              norm_weight=None, eps: float = 1e-6, inv_freq=None, start: int = 0, interleaved: bool = False,
              mscale: float = 1.0, k_out=None, stream=None):
    """Write the new tokens' keys and values to a paged cache (``kda_kv_append``).

    k_cache, v_cache, block_table, seq_lens, cu_seqlens: as for ``window_decode``
    (seq_lens counts the new tokens).  k, v: [T, Hk, d] (strided, e.g. parts of one
    projection).  norm_weight: fp32 [d] of the keys' RMS norm per head, or None for
    no norm; inv_freq: fp32 [dr / 2], or None for no rotation, of channels [start,
    start + dr); mscale multiplies the rotated part.  k_out: True (allocate) or a
    dense [T, Hk, d] tensor for the keys as they are cached.  Returns k_out."""
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k, v: [T, Hk, d]")
    T = k.shape[0]
    cache, N, Hk, d, dt, dev = _kv_cache(k_cache, v_cache, block_table, seq_lens, cu_seqlens, num_seqs)
    float32 = _torch.float32
    kt, kh = _strides3(k, "k", T, Hk, d, dt, dev)
    vt, vh = _strides3(v, "v", T, Hk, d, dt, dev)
    if norm_weight is not None:
        _dense(norm_weight, "norm_weight", (d,), float32, dev)
    dr = 0
    if inv_freq is not None:
        dr = 2 * inv_freq.numel()
        _dense(inv_freq, "inv_freq", (dr // 2,), float32, dev)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return kv_append(k_cache, v_cache, k, v, block_table, seq_lens, cu_seqlens, num_seqs, norm_weight, eps,
                             inv_freq, start, interleaved, mscale, k_out)
    if k_out is True:
        k_out = k.new_empty(T, Hk, d)
    elif k_out is None or k_out is False:
        k_out = None
    else:
        _dense(k_out, "k_out", (T, Hk, d), dt, dev)
    st = lib().kda_kv_append(
        cache, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, None if cu_seqlens is None else cu_seqlens.data_ptr(), T, N,
        Hk, d, _code(k), _ptr(norm_weight), eps, _ptr(inv_freq) if dr else None, _int32(start, "start"), dr, mscale,
        KDA_ROTARY_INTERLEAVED if interleaved else 0, _ptr(k_out), _raw_stream(dev))
    if st:
        _check(st, "kda_kv_append")
    return k_out


def _norm_weight(weight, name, d, device) -> int:
    if weight is None:
        return 0
    _dense(weight, name, (d,), _torch.float32, device)
    return weight.data_ptr()


def _norm_rotation(positions, inv_freq, T, dev):
    """Rotated channels, with the rotation's arguments checked."""
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq: both or neither")
    if inv_freq is None:
        return 0
    half = inv_freq.numel()
    _dense(inv_freq, "inv_freq", (half,), _torch.float32, dev)
    _dense(positions, "positions", (T,), _torch.int32, dev)
    return 2 * half


def qk_norm_rotary(q, k=None, q_weight=None, k_weight=None, positions=None, inv_freq=None, start: int = 0,
                   interleaved: bool = False, mscale: float = 1.0, eps: float = 1e-6, q_out=None, k_out=None,
                   stream=None):
    """RMS norm of every query and key head and rotary positions in one pass
    (``kda_qk_norm_rotary``).

    q: [T, H, d]; k: [T, Hk, d] or None (strided, e.g. parts of one projection);
    q_weight, k_weight: fp32 [d], or None for ones; positions: int32 [T] and
    inv_freq: fp32 [dr / 2], or both None for no rotation, of channels [start,
    start + dr); mscale multiplies the rotated part.  q_out, k_out: None (allocate),
    the input itself (in place), or a tensor that overlaps no other.  Returns
    (q_out, k_out)."""
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q, k: [T, heads, channels]")
    torch = _lib_torch()
    T, H, d = q.shape
    dev, dt = q.device, q.dtype
    qt, qh = _strides3(q, "q", T, H, d, dt, dev)
    qw = _norm_weight(q_weight, "q_weight", d, dev)
    if k is not None:
        Hk = k.shape[1]
        kt, kh = _strides3(k, "k", T, Hk, d, dt, dev)
        kw = _norm_weight(k_weight, "k_weight", d, dev)
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    dr = _norm_rotation(positions, inv_freq, T, dev)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return qk_norm_rotary(q, k, q_weight, k_weight, positions, inv_freq, start, interleaved, mscale, eps, q_out,
                                  k_out)
    if q_out is None:
        q_out = q.new_empty(T, H, d)
        ot, oh = H * d, d
    else:
        ot, oh = _strides3(q_out, "q_out", T, H, d, dt, dev)
    a = _NORM_HEADS.pack(q.data_ptr(), qt, qh, q_out.data_ptr(), ot, oh, qw, 0, 0, 0, 0, 0, 0, 0, H)
    b = None
    if k is not None:
        if k_out is None:
            k_out = k.new_empty(T, Hk, d)
            ot, oh = Hk * d, d
        else:
            ot, oh = _strides3(k_out, "k_out", T, Hk, d, dt, dev)
        b = _NORM_HEADS.pack(k.data_ptr(), kt, kh, k_out.data_ptr(), ot, oh, kw, 0, 0, 0, 0, 0, 0, 0, Hk)
    st = lib().kda_qk_norm_rotary(a, b, _ptr(positions) if dr else None, _ptr(inv_freq) if dr else None, T, d,
                                  _int32(start, "start"), dr, _code(q), eps, mscale,
                                  KDA_ROTARY_INTERLEAVED if interleaved else 0, _raw_stream(dev))
    if st:
        _check(st, "kda_qk_norm_rotary")
    return q_out, k_out


def qk_norm_rotary_backward_workspace_bytes(d: int) -> int:
    return int(lib().kda_qk_norm_rotary_backward_workspace_bytes(int(d)))


def qk_norm_rotary_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, positions=None, inv_freq=None,
                            start: int = 0, interleaved: bool = False, mscale: float = 1.0, eps: float = 1e-6, dq=None,
                            dk=None, workspace=None, stream=None) -> dict:
    """Gradients of ``qk_norm_rotary`` (``kda_qk_norm_rotary_backward``) from its
    inputs q and k (k and dk_out may be None) and dL/dq_out, dL/dk_out (strided):
    returns dq, dk in the inputs' type, and dq_weight, dk_weight (fp32 [d], None
    without that weight).  dq, dk: None (allocate), or tensors to write: dq_out or q
    itself (in place), or one that overlaps no other, e.g. part of the projection's
    gradient."""
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q, k: [T, heads, channels]")
    torch = _lib_torch()
    T, H, d = q.shape
    dev, dt = q.device, q.dtype
    if k is None:
        if k_weight is not None or dk_out is not None or dk is not None:
            raise ValueError("k_weight, dk_out and dk need k")
    elif dk_out is None:
        raise ValueError("dk_out: it goes with k")
    dr = _norm_rotation(positions, inv_freq, T, dev)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return qk_norm_rotary_backward(q, k, dq_out, dk_out, q_weight, k_weight, positions, inv_freq, start,
                                           interleaved, mscale, eps, dq, dk, workspace)

    def heads(x, name, dy, dx, weight):
        H = x.shape[1]
        xt, xh = _strides3(x, name, T, H, d, dt, dev)
        yt, yh = _strides3(dy, f"d{name}_out", T, H, d, dt, dev)
        w = _norm_weight(weight, f"{name}_weight", d, dev)
        if dx is None:
            dx = x.new_empty(T, H, d)
        dt_, dh = _strides3(dx, f"d{name}", T, H, d, dt, dev)
        dw = x.new_empty(d, dtype=torch.float32) if weight is not None else None
        packed = _NORM_HEADS.pack(x.data_ptr(), xt, xh, 0, 0, 0, w, dy.data_ptr(), yt, yh, dx.data_ptr(), dt_, dh,
                                  0 if dw is None else dw.data_ptr(), H)
        return packed, dx, dw

    a, dq, dqw = heads(q, "q", dq_out, dq, q_weight)
    b, dk, dkw = heads(k, "k", dk_out, dk, k_weight) if k is not None else (None, None, None)
    handle = lib()
    if workspace is None:
        need = handle.kda_qk_norm_rotary_backward_workspace_bytes(d)
        workspace = q.new_empty(need, dtype=torch.uint8)
    else:
        _require(workspace.device == dev and workspace.is_contiguous(), "workspace: contiguous, same device")
        need = workspace.numel() * workspace.element_size()
    st = handle.kda_qk_norm_rotary_backward(
        a, b, _ptr(positions) if dr else None, _ptr(inv_freq) if dr else None, T, d, _int32(start, "start"), dr, _code(q),
        eps, mscale, KDA_ROTARY_INTERLEAVED if interleaved else 0, workspace.data_ptr() or None, need, _raw_stream(dev))
    if st:
        _check(st, "kda_qk_norm_rotary_backward")
    return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)
