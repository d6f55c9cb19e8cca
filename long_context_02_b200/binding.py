"""Thin ctypes binding of liblightning.so (argument marshalling only).

Each ``la_*`` function mirrors the C entry point of the same name in
include/lightning.h: it takes torch tensors that already live on the GPU,
derives the sizes from their shapes, passes raw device pointers and the
current CUDA stream, and raises ``LightningError`` on a non-zero status.
Every step of the computation runs in the library's CUDA kernels; there is no
other implementation to fall back to. If the library has not been built,
``lib()`` raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblightning.so")

LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_CUDA, LA_ERR_TIMEOUT, LA_ERR_WORKSPACE = (
    0, -1, -2, -3, -4, -5)
LA_BF16, LA_F32 = 0, 1
LA_OP_PREFILL, LA_OP_PREFILL_VARLEN, LA_OP_DECODE, LA_OP_BACKWARD = 0, 1, 2, 3
LA_OP_SCAN, LA_OP_SCAN_BACKWARD, LA_OP_CONV_BACKWARD, LA_OP_NORM_BACKWARD = 4, 5, 6, 7

EXPORTED = ["la_workspace_bytes", "la_prefill", "la_prefill_varlen", "la_decode", "la_backward",
            "la_status_string", "la_read_device_status", "la_set_tuning", "la_get_tuning",
            "la_last_launch_count", "la_prefill_noalloc", "la_set_fault_injection",
            "la_prefill_with_state", "la_prefill_varlen_with_state", "la_mixed_step",
            "la_output_norm_gate", "la_state_prefix", "la_prefill_state", "la_noalloc_device_status",
            "la_selective_scan", "la_selective_scan_step", "la_selective_scan_backward",
            "la_short_conv", "la_short_conv_step", "la_short_conv_backward", "la_layer_norm",
            "la_layer_norm_backward"]

_lib = None


# la_scan_inputs and la_scan_grads of include/lightning.h.
SCAN_INPUTS = struct.Struct("@5P5q3Pi4x")  # u delta z B C, their strides, A D delta_bias, softplus
SCAN_GRADS = struct.Struct("@9P")  # du ddelta dz dB dC dA dD ddelta_bias dstate_in


class LightningError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = lib().la_status_string(status).decode()
        super().__init__(f"{fn} failed: {msg} ({status})")


def lib():
    """Load liblightning.so (built in-tree by long_context_02_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m long_context_02_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, LL, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
        L.la_workspace_bytes.argtypes = [I, I, I, LL, I, I, I]
        L.la_workspace_bytes.restype = SZ
        L.la_prefill.argtypes = [P, P, P, P, P, P, I, I, LL, I, I, I, P, SZ, P]
        L.la_prefill_varlen.argtypes = [P, I, P, P, P, P, P, P, I, LL, I, I, I, P, SZ, P]
        L.la_prefill_with_state.argtypes = [P, P, P, P, P, P, P, I, I, LL, I, I, I, P, SZ, P]
        L.la_prefill_varlen_with_state.argtypes = [P, I, P, P, P, P, P, P, P, I, LL, I, I, I, P,
                                                   SZ, P]
        L.la_mixed_step.argtypes = [P, I, P, P, P, P, P, P, I, LL, I, I, I, P, SZ, P, P]
        L.la_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P]
        L.la_prefill_state.argtypes = [P, P, P, P, P, I, I, LL, I, I, P, SZ, P]
        L.la_state_prefix.argtypes = [P, P, ctypes.POINTER(LL), I, I, I, I, I, P, P]
        L.la_output_norm_gate.argtypes = [P, P, P, ctypes.c_float, P, I, I, LL, I, I, I, P]
        L.la_backward.argtypes = [P, P, P, P, P, P, P, P, I, I, LL, I, I, I, P, SZ, P]
        SI, SG = P, P  # packed structures
        L.la_selective_scan.argtypes = [P, I, SI, P, P, P, LL, I, I, I, I, I, P, SZ, P]
        L.la_selective_scan_step.argtypes = [SI, P, P, I, I, I, I, I, I, P]
        L.la_selective_scan_backward.argtypes = [P, I, SI, P, P, LL, P, SG, LL, I, I, I, I, I, P,
                                                 SZ, P]
        L.la_short_conv.argtypes = [P, I, P, LL, P, P, P, P, P, LL, I, I, I, I, I, P]
        L.la_short_conv_step.argtypes = [P, LL, P, P, P, P, I, I, I, I, I, I, P]
        L.la_short_conv_backward.argtypes = [P, I, P, LL, P, LL, P, P, P, P, P, P, P, P, LL, I, I,
                                             I, I, I, P, SZ, P]
        L.la_layer_norm.argtypes = [P, P, P, ctypes.c_float, P, P, P, LL, I, I, I, P]
        L.la_layer_norm_backward.argtypes = [P, P, P, P, P, P, P, P, LL, I, I, I, P, SZ, P]
        L.la_status_string.argtypes = [I]
        L.la_status_string.restype = ctypes.c_char_p
        L.la_read_device_status.argtypes = [P, P]
        L.la_set_tuning.argtypes = [I, I]
        L.la_get_tuning.argtypes = [ctypes.POINTER(I), ctypes.POINTER(I)]
        L.la_last_launch_count.argtypes = []
        L.la_prefill_noalloc.argtypes = [P, P, P, P, P, P, I, I, LL, I, I, I, P]
        L.la_set_fault_injection.argtypes = [I, I]
        L.la_noalloc_device_status.argtypes = [P]
        for f in ("la_prefill", "la_prefill_varlen", "la_prefill_with_state",
                  "la_prefill_varlen_with_state", "la_mixed_step", "la_output_norm_gate",
                  "la_state_prefix", "la_prefill_state",
                  "la_decode", "la_backward",
                  "la_read_device_status", "la_set_tuning", "la_get_tuning",
                  "la_last_launch_count", "la_prefill_noalloc", "la_set_fault_injection",
                  "la_noalloc_device_status", "la_selective_scan", "la_selective_scan_step",
                  "la_selective_scan_backward", "la_short_conv", "la_short_conv_step",
                  "la_short_conv_backward", "la_layer_norm", "la_layer_norm_backward"):
            getattr(L, f).restype = I
        _lib = L
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LA_BF16
    if t.dtype == torch.float32:
        return LA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None or t.numel() == 0:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, status):
    if status != LA_OK:
        raise LightningError(fn, status)


def la_workspace_bytes(op, B, H, N_or_total, d, num_seqs=0, in_dtype=torch.bfloat16) -> int:
    in_t = LA_BF16 if in_dtype == torch.bfloat16 else LA_F32
    return int(lib().la_workspace_bytes(op, B, H, N_or_total, d, num_seqs, in_t))


def workspace(op, B, H, N_or_total, d, num_seqs=0, in_dtype=torch.bfloat16, device="cuda"):
    n = la_workspace_bytes(op, B, H, N_or_total, d, num_seqs, in_dtype)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def la_prefill(q, k, v, slopes, o, state_out, ws, stream=None):
    B, H, N, d = q.shape
    _check("la_prefill", lib().la_prefill(
        _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(o), _ptr(state_out), B, H, N, d,
        _dt(q), _dt(o), _ptr(ws), ws.numel(), _stream(stream)))


def la_prefill_varlen(cu_seqlens, q, k, v, slopes, o, state_out, ws, stream=None):
    H, T, d = q.shape
    num_seqs = cu_seqlens.numel() - 1
    _check("la_prefill_varlen", lib().la_prefill_varlen(
        _ptr(cu_seqlens), num_seqs, _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(o),
        _ptr(state_out), H, T, d, _dt(q), _dt(o), _ptr(ws), ws.numel(), _stream(stream)))


def la_prefill_with_state(q, k, v, slopes, state_in, o, state_out, ws, stream=None):
    B, H, N, d = q.shape
    _check("la_prefill_with_state", lib().la_prefill_with_state(
        _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(state_in), _ptr(o), _ptr(state_out),
        B, H, N, d, _dt(q), _dt(o), _ptr(ws), ws.numel(), _stream(stream)))


def la_prefill_varlen_with_state(cu_seqlens, q, k, v, slopes, state_in, o, state_out, ws,
                                 stream=None):
    H, T, d = q.shape
    num_seqs = cu_seqlens.numel() - 1
    _check("la_prefill_varlen_with_state", lib().la_prefill_varlen_with_state(
        _ptr(cu_seqlens), num_seqs, _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(state_in),
        _ptr(o), _ptr(state_out), H, T, d, _dt(q), _dt(o), _ptr(ws), ws.numel(),
        _stream(stream)))


def la_mixed_step(cu_seqlens, q, k, v, slopes, states, o, ws, prefill_stream=None,
                  decode_stream=None):
    H, T, d = q.shape
    num_seqs = cu_seqlens.numel() - 1
    _check("la_mixed_step", lib().la_mixed_step(
        _ptr(cu_seqlens), num_seqs, _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(states),
        _ptr(o), H, T, d, _dt(q), _dt(o), _ptr(ws), ws.numel(), _stream(prefill_stream),
        _stream(decode_stream)))


def la_output_norm_gate(o, gate, weight, eps, y, stream=None):
    B, H, N, d = o.shape
    _check("la_output_norm_gate", lib().la_output_norm_gate(
        _ptr(o), _ptr(gate), _ptr(weight), float(eps), _ptr(y), B, H, N, d, _dt(o), _dt(y),
        _stream(stream)))


def la_state_prefix(states, slopes, lens, r, out, stream=None):
    R, B, H, d, _ = states.shape
    arr = (ctypes.c_longlong * R)(*[int(x) for x in lens])
    _check("la_state_prefix", lib().la_state_prefix(
        _ptr(states), _ptr(slopes), arr, R, int(r), B, H, d, _ptr(out), _stream(stream)))


def la_prefill_state(k, v, slopes, state_in, state_out, ws, stream=None):
    B, H, N, d = k.shape
    _check("la_prefill_state", lib().la_prefill_state(
        _ptr(k), _ptr(v), _ptr(slopes), _ptr(state_in), _ptr(state_out), B, H, N, d, _dt(k),
        _ptr(ws), ws.numel(), _stream(stream)))


def la_decode(q, k, v, slopes, state, o, stream=None):
    B, H, d = q.shape
    _check("la_decode", lib().la_decode(
        _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(state), _ptr(o), B, H, d, _dt(q), _dt(o),
        _stream(stream)))


def la_backward(dout, q, k, v, slopes, dq, dk, dv, ws, stream=None):
    B, H, N, d = q.shape
    _check("la_backward", lib().la_backward(
        _ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(dq), _ptr(dk), _ptr(dv),
        B, H, N, d, _dt(q), _dt(dq), _ptr(ws), ws.numel(), _stream(stream)))


def la_prefill_noalloc(q, k, v, slopes, o, state_out, stream=None):
    """la_prefill on the library's built-in scratch (for callers that cannot
    allocate device memory; see include/lightning.h)."""
    B, H, N, d = q.shape
    _check("la_prefill_noalloc", lib().la_prefill_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(slopes), _ptr(o), _ptr(state_out), B, H, N, d,
        _dt(q), _dt(o), _stream(stream)))


def la_noalloc_device_status(stream=None) -> int:
    """Device-side status of the last la_prefill_noalloc on the current device."""
    return int(lib().la_noalloc_device_status(_stream(stream)))


def la_read_device_status(ws, stream=None) -> int:
    return int(lib().la_read_device_status(_ptr(ws), _stream(stream)))


def la_set_tuning(block_tokens=0, segment_tokens=0):
    _check("la_set_tuning", lib().la_set_tuning(block_tokens, segment_tokens))


def la_get_tuning():
    b, s = ctypes.c_int(), ctypes.c_int()
    lib().la_get_tuning(ctypes.byref(b), ctypes.byref(s))
    return b.value, s.value


def la_set_fault_injection(skip_publish=0, wait_limit_us=0):
    """Test-only: make the scan's inter-segment waits run out (see lightning.h)."""
    _check("la_set_fault_injection", lib().la_set_fault_injection(int(skip_publish),
                                                                 int(wait_limit_us)))


def la_last_launch_count() -> int:
    return int(lib().la_last_launch_count())


def la_status_string(status) -> str:
    return lib().la_status_string(status).decode()


# ---------------------------------------------------------------- conveniences

def prefill(q, k, v, slopes, out_dtype=None, want_state=True, stream=None, state_in=None):
    """Allocate outputs and workspace, run la_prefill (la_prefill_with_state when
    state_in [B,H,d,d] is given). Returns (O, state or None)."""
    B, H, N, d = q.shape
    o = torch.empty_like(q, dtype=out_dtype or q.dtype)
    st = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device) if want_state else None
    ws = workspace(LA_OP_PREFILL, B, H, N, d, 0, q.dtype, q.device)
    if state_in is None:
        la_prefill(q, k, v, slopes, o, st, ws, stream)
    else:
        la_prefill_with_state(q, k, v, slopes, state_in, o, st, ws, stream)
    return o, st


def prefill_varlen(cu_seqlens, q, k, v, slopes, out_dtype=None, want_state=True, stream=None,
                   state_in=None):
    H, T, d = q.shape
    S = cu_seqlens.numel() - 1
    o = torch.empty_like(q, dtype=out_dtype or q.dtype)
    st = torch.empty((S, H, d, d), dtype=torch.float32, device=q.device) if want_state else None
    ws = workspace(LA_OP_PREFILL_VARLEN, 1, H, T, d, S, q.dtype, q.device)
    if state_in is None:
        la_prefill_varlen(cu_seqlens, q, k, v, slopes, o, st, ws, stream)
    else:
        la_prefill_varlen_with_state(cu_seqlens, q, k, v, slopes, state_in, o, st, ws, stream)
    return o, st


def decode(q, k, v, slopes, state, out_dtype=None, stream=None):
    o = torch.empty_like(q, dtype=out_dtype or q.dtype)
    la_decode(q, k, v, slopes, state, o, stream)
    return o


def backward(dout, q, k, v, slopes, out_dtype=None, stream=None):
    B, H, N, d = q.shape
    dt = out_dtype or q.dtype
    dq, dk, dv = (torch.empty_like(q, dtype=dt) for _ in range(3))
    ws = workspace(LA_OP_BACKWARD, B, H, N, d, 0, q.dtype, q.device)
    la_backward(dout, q, k, v, slopes, dq, dk, dv, ws, stream)
    return dq, dk, dv


# ---------------------------------------------------------------- state space layer
#
# Token tensors are [B, N, ...] (num_seqs = B sequences of N tokens) or, with
# cu_seqlens, [T, ...]; a token input may be a column slice of a wider tensor
# (any stride between tokens, its last dimensions contiguous).

def _rows(t, shape, lead, dense, what):
    """Pointer of a token tensor and the elements between its tokens, of which
    each has `dense` elements in the dimensions behind the `lead` first ones."""
    if t.shape != shape:
        raise ValueError(f"{what} is {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), dense
    stride, size = t.stride(), 1
    for n, st in zip(reversed(shape[lead:]), reversed(stride[lead:])):
        if n != 1 and st != size:
            raise ValueError(f"{what}: the elements of a token must be contiguous")
        size *= n
    if lead == 2 and shape[1] > 1:
        ld = stride[1]
        if shape[0] > 1 and stride[0] != shape[1] * ld:
            raise ValueError(f"{what}: the tokens of all sequences must be evenly spaced")
    else:
        ld = stride[0] if shape[0] > 1 else dense
    return t.data_ptr(), ld


def _flat(t, shape, dtype, what):
    """Pointer of a dense tensor of a given shape and dtype; 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what} is {t.dtype} {tuple(t.shape)}, expected {dtype} {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


_HERE_AND_NOW = contextlib.nullcontext()


def _on(stream, *tensors):
    """(device index, context, raw stream) of a call on these tensors, None among
    them, which are all on one GPU. Within the context that device is current
    and allocations belong to the stream (default: the device's current one).
    Inputs that a caller frees while the call runs on another stream than theirs
    stay allocated until it is done."""
    index = tensors[0].get_device()
    if index < 0:
        raise ValueError(f"tensors must be on a GPU, not on {tensors[0].device}")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {tensors[0].device} and on {t.device}")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
        if torch.cuda.current_device() == index:
            return index, _HERE_AND_NOW, raw
        return index, torch.cuda.device(index), raw
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    if stream != torch.cuda.current_stream(index):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    return index, torch.cuda.stream(stream), stream.cuda_stream  # makes its device current too


def _sequences(x, cu_seqlens):
    """(shape of the rows, number of sequences, rows, pointer of cu_seqlens)."""
    shape = x.shape
    if cu_seqlens is None:
        if len(shape) != 3:
            raise ValueError(f"expected [B, N, D] without cu_seqlens, got {tuple(shape)}")
        return shape[:2], shape[0], shape[0] * shape[1], 0
    if len(shape) != 2:
        raise ValueError(f"expected [T, D] with cu_seqlens, got {tuple(shape)}")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be int32 [num_seqs + 1]")
    return shape[:1], cu_seqlens.numel() - 1, shape[0], _flat(cu_seqlens, cu_seqlens.shape,
                                                              torch.int32, "cu_seqlens")


def _new(like, shape, dtype):
    """An output like a token input, of another dtype where one is given."""
    if (dtype is None or dtype == like.dtype) and like.is_contiguous():
        return torch.empty_like(like)
    return like.new_empty(shape, dtype=dtype)


def _scan_inputs(u, delta, A, B, C, D, z, delta_bias, softplus, lead):
    """(packed la_scan_inputs, D, G, n, in_t) after checking every shape."""
    shape, ashape, dtype = u.shape, A.shape, u.dtype
    if len(ashape) != 2 or B.dim() != lead + 2:
        raise ValueError(f"A is [D, n] and B [tokens, G, n], got {tuple(ashape)}, {tuple(B.shape)}")
    width, n, G = shape[-1], ashape[1], B.shape[-2]
    if delta.dtype != dtype or B.dtype != dtype or C.dtype != dtype or (
            z is not None and z.dtype != dtype):
        raise ValueError(f"delta, z, B and C must be {dtype} as u is")
    bc = (*shape[:-1], G, n)
    up, ld_u = _rows(u, shape, lead, width, "u")
    dp, ld_d = _rows(delta, shape, lead, width, "delta")
    bp, ld_b = _rows(B, bc, lead, G * n, "B")
    cp, ld_c = _rows(C, bc, lead, G * n, "C")
    zp, ld_z = (0, 0) if z is None else _rows(z, shape, lead, width, "z")
    f32, vector = torch.float32, (width,)
    packed = SCAN_INPUTS.pack(up, dp, zp, bp, cp, ld_u, ld_d, ld_z, ld_b, ld_c,
                              _flat(A, (width, n), f32, "A"), _flat(D, vector, f32, "D"),
                              _flat(delta_bias, vector, f32, "delta_bias"), 1 if softplus else 0)
    return packed, width, G, n, _dt(u)


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                   state_in=None, cu_seqlens=None, want_state=True, out_dtype=None, stream=None):
    """Allocate outputs and workspace and run la_selective_scan. u, delta, z
    [B, N, D] (packed [T, D] with cu_seqlens), A [D, n], B and C [B, N, G, n],
    D and delta_bias [D], state_in [num_seqs, D, n]. Returns (y, state or None)."""
    rows_shape, seqs, rows, cu = _sequences(u, cu_seqlens)
    dev, ctx, handle = _on(stream, u, delta, A, B, C, D, z, delta_bias, state_in, cu_seqlens)
    s, width, G, n, in_t = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, softplus,
                                        len(rows_shape))
    states = (seqs, width, n)
    sp = _flat(state_in, states, torch.float32, "state_in")
    fn = lib()
    with ctx:
        y = _new(u, u.shape, out_dtype)
        state = A.new_empty(states) if want_state else None
        need = fn.la_workspace_bytes(LA_OP_SCAN, G, width, rows, n, seqs, in_t)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        status = fn.la_selective_scan(
            cu, seqs, s, sp, y.data_ptr(), state.data_ptr() if want_state else 0, rows, width, G,
            n, in_t, _dt(y), ws.data_ptr() if need else 0, need, handle)
    _check("la_selective_scan", status)
    return y, state


def selective_scan_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None, softplus=True,
                        out_dtype=None, stream=None):
    """la_selective_scan_step: one token for each of B sequences (u, delta, z
    [B, D], B and C [B, G, n]); state [B, D, n] is advanced in place. Returns y [B, D]."""
    if u.dim() != 2:
        raise ValueError(f"u is [B, D], got {tuple(u.shape)}")
    _, ctx, handle = _on(stream, u, delta, A, B, C, D, z, delta_bias, state)
    s, width, G, n, in_t = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, softplus, 1)
    seqs = u.shape[0]
    sp = _flat(state, (seqs, width, n), torch.float32, "state")
    with ctx:
        y = _new(u, u.shape, out_dtype)
        status = lib().la_selective_scan_step(s, sp, y.data_ptr(), seqs, width, G, n, in_t,
                                              _dt(y), handle)
    _check("la_selective_scan_step", status)
    return y


def selective_scan_backward(dy, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                            state_in=None, dstate_out=None, cu_seqlens=None, out_dtype=None,
                            stream=None):
    """Gradients of selective_scan for the output gradient dy (and dstate_out,
    that of the returned state). Returns a dict: du, ddelta, dB, dC, dA, and dz,
    dD, ddelta_bias, dstate_in where the call has that input."""
    rows_shape, seqs, rows, cu = _sequences(u, cu_seqlens)
    dev, ctx, handle = _on(stream, u, dy, delta, A, B, C, D, z, delta_bias, state_in, dstate_out,
                           cu_seqlens)
    lead = len(rows_shape)
    s, width, G, n, in_t = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, softplus, lead)
    if dy.dtype != u.dtype:
        raise ValueError(f"dy is {dy.dtype}, u is {u.dtype}")
    dyp, ld_dy = _rows(dy, u.shape, lead, width, "dy")
    f32, states = torch.float32, (seqs, width, n)
    sp = _flat(state_in, states, f32, "state_in")
    dsp = _flat(dstate_out, states, f32, "dstate_out")
    fn = lib()
    with ctx:
        t = out_dtype or u.dtype
        bc = (*rows_shape, G, n)
        out = {"du": _new(u, u.shape, t), "ddelta": _new(u, u.shape, t),
               "dB": u.new_empty(bc, dtype=t), "dC": u.new_empty(bc, dtype=t), "dA": torch.empty_like(A)}
        if z is not None:
            out["dz"] = _new(u, u.shape, t)
        if D is not None:
            out["dD"] = torch.empty_like(D)
        if delta_bias is not None:
            out["ddelta_bias"] = torch.empty_like(delta_bias)
        if state_in is not None:
            out["dstate_in"] = torch.empty_like(state_in)
        g = SCAN_GRADS.pack(*[out[f].data_ptr() if f in out else 0 for f in (
            "du", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddelta_bias", "dstate_in")])
        need = fn.la_workspace_bytes(LA_OP_SCAN_BACKWARD, G, width, rows, n, seqs, in_t)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        status = fn.la_selective_scan_backward(
            cu, seqs, s, sp, dyp, ld_dy, dsp, g, rows, width, G, n, in_t, _dt(out["du"]),
            ws.data_ptr() if need else 0, need, handle)
    _check("la_selective_scan_backward", status)
    return out


def _conv_weights(x, weight, bias):
    width = x.shape[-1]
    if weight.dim() != 2:
        raise ValueError(f"weight is [D, W], got {tuple(weight.shape)}")
    W = weight.shape[1]
    return (width, W, _flat(weight, (width, W), torch.float32, "weight"),
            _flat(bias, (width,), torch.float32, "bias"))


def short_conv(x, weight, bias=None, silu=True, state_in=None, cu_seqlens=None, want_state=True,
               out_dtype=None, stream=None):
    """Allocate outputs and run la_short_conv. x [B, N, D] (packed [T, D] with
    cu_seqlens), weight [D, W], bias [D], state_in [num_seqs, W-1, D] of x's
    dtype. Returns (y, state or None)."""
    rows_shape, seqs, rows, cu = _sequences(x, cu_seqlens)
    _, ctx, handle = _on(stream, x, weight, bias, state_in, cu_seqlens)
    width, W, wp, bp = _conv_weights(x, weight, bias)
    xp, ld_x = _rows(x, x.shape, len(rows_shape), width, "x")
    states = (seqs, max(W - 1, 0), width)
    sp = _flat(state_in, states, x.dtype, "state_in")
    with ctx:
        y = _new(x, x.shape, out_dtype)
        state = x.new_empty(states) if want_state else None
        status = lib().la_short_conv(
            cu, seqs, xp, ld_x, wp, bp, sp, y.data_ptr(), state.data_ptr() if want_state else 0,
            rows, width, W, 1 if silu else 0, _dt(x), _dt(y), handle)
    _check("la_short_conv", status)
    return y, state


def short_conv_step(x, weight, bias, state, silu=True, out_dtype=None, stream=None):
    """la_short_conv_step: one token for each of B sequences (x [B, D]); state
    [B, W-1, D] is advanced in place. Returns y [B, D]."""
    if x.dim() != 2:
        raise ValueError(f"x is [B, D], got {tuple(x.shape)}")
    _, ctx, handle = _on(stream, x, weight, bias, state)
    width, W, wp, bp = _conv_weights(x, weight, bias)
    seqs = x.shape[0]
    xp, ld_x = _rows(x, x.shape, 1, width, "x")
    sp = _flat(state, (seqs, W - 1, width), x.dtype, "state")
    with ctx:
        y = _new(x, x.shape, out_dtype)
        status = lib().la_short_conv_step(xp, ld_x, wp, bp, sp, y.data_ptr(), seqs, width, W,
                                          1 if silu else 0, _dt(x), _dt(y), handle)
    _check("la_short_conv_step", status)
    return y


def short_conv_backward(dy, x, weight, bias=None, silu=True, state_in=None, dstate_out=None,
                        cu_seqlens=None, out_dtype=None, stream=None):
    """Gradients of short_conv. Returns a dict: dx, dweight, and dbias,
    dstate_in where the call has that input."""
    rows_shape, seqs, rows, cu = _sequences(x, cu_seqlens)
    dev, ctx, handle = _on(stream, x, dy, weight, bias, state_in, dstate_out, cu_seqlens)
    width, W, wp, bp = _conv_weights(x, weight, bias)
    if dy.dtype != x.dtype:
        raise ValueError(f"dy is {dy.dtype}, x is {x.dtype}")
    xp, ld_x = _rows(x, x.shape, len(rows_shape), width, "x")
    dyp, ld_dy = _rows(dy, x.shape, len(rows_shape), width, "dy")
    states = (seqs, W - 1, width)
    sp = _flat(state_in, states, x.dtype, "state_in")
    dsp = _flat(dstate_out, states, x.dtype, "dstate_out")
    fn, in_t = lib(), _dt(x)
    with ctx:
        t = out_dtype or x.dtype
        out = {"dx": _new(x, x.shape, t), "dweight": torch.empty_like(weight)}
        if bias is not None:
            out["dbias"] = torch.empty_like(bias)
        if state_in is not None:
            out["dstate_in"] = x.new_empty(states, dtype=t)
        need = fn.la_workspace_bytes(LA_OP_CONV_BACKWARD, 1, width, rows, W, seqs, in_t)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        status = fn.la_short_conv_backward(
            cu, seqs, dyp, ld_dy, xp, ld_x, wp, bp, sp, dsp, out["dx"].data_ptr(),
            out["dweight"].data_ptr(), out["dbias"].data_ptr() if bias is not None else 0,
            out["dstate_in"].data_ptr() if state_in is not None else 0, rows, width, W,
            1 if silu else 0, in_t, _dt(out["dx"]), ws.data_ptr() if need else 0, need, handle)
    _check("la_short_conv_backward", status)
    return out


def layer_norm(x, weight, bias=None, eps=1e-5, want_stats=True, out_dtype=None, stream=None):
    """la_layer_norm over the last dimension of x (dense). Returns (y, mean,
    rstd); the last two, fp32 of x's leading shape, are what
    layer_norm_backward takes (None without want_stats)."""
    _, ctx, handle = _on(stream, x, weight, bias)
    shape, f32 = x.shape, torch.float32
    if not shape:
        raise ValueError("x has no dimension to normalise over")
    F = shape[-1]
    xp = _flat(x, shape, x.dtype, "x")
    wp, bp = _flat(weight, (F,), f32, "weight"), _flat(bias, (F,), f32, "bias")
    rows = x.numel() // F if F else 0
    with ctx:
        y = _new(x, shape, out_dtype)
        mean = rstd = None
        mp = rp = 0
        if want_stats:
            mean = weight.new_empty(shape[:-1])
            rstd = torch.empty_like(mean)
            mp, rp = mean.data_ptr(), rstd.data_ptr()
        status = lib().la_layer_norm(xp, wp, bp, eps, y.data_ptr(), mp, rp, rows, F, _dt(x),
                                     _dt(y), handle)
    _check("la_layer_norm", status)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, want_bias=True, out_dtype=None, stream=None):
    """Gradients of layer_norm: (dx, dweight, dbias); dbias is None without want_bias."""
    dev, ctx, handle = _on(stream, x, dy, weight, mean, rstd)
    shape, f32 = x.shape, torch.float32
    if not shape:
        raise ValueError("x has no dimension to normalise over")
    F = shape[-1]
    xp, dyp = _flat(x, shape, x.dtype, "x"), _flat(dy, shape, x.dtype, "dy")
    wp = _flat(weight, (F,), f32, "weight")
    mp, rp = _flat(mean, shape[:-1], f32, "mean"), _flat(rstd, shape[:-1], f32, "rstd")
    rows = x.numel() // F if F else 0
    fn, in_t = lib(), _dt(x)
    with ctx:
        dx, dw = _new(x, shape, out_dtype), torch.empty_like(weight)
        db = torch.empty_like(weight) if want_bias else None
        need = fn.la_workspace_bytes(LA_OP_NORM_BACKWARD, 1, F, rows, 1, 1, in_t)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        status = fn.la_layer_norm_backward(
            dyp, xp, wp, mp, rp, dx.data_ptr(), dw.data_ptr(), db.data_ptr() if want_bias else 0,
            rows, F, in_t, _dt(dx), ws.data_ptr() if need else 0, need, handle)
    _check("la_layer_norm_backward", status)
    return dx, dw, db
