"""Python binding of the vector-state recurrence of libgdn.so
(include/gdn_linrec.h): whole sequences, their gradients, and one token in place.

As in the package's other bindings, arguments are only marshalled and there is
no fallback.  Tensors may be views whose rows are contiguous: row strides are
arguments of the calls.  All tensors of a call must be on one GPU; the call is
made with that GPU current and, unless a stream is given, on its current stream.
"""
from __future__ import annotations

import ctypes

import torch

import linear_attention_ssm_gated_amd as _gdn

from .train import _bytes, _Call, _code, _shaped

LINREC_PLAIN, LINREC_COMPLEMENT, LINREC_ROOT = 0, 1, 2
_SCALES = {"plain": LINREC_PLAIN, "complement": LINREC_COMPLEMENT, "root": LINREC_ROOT}

P, I, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
# name -> (restype, argtypes) of every entry point include/gdn_linrec.h declares
LINREC_SIGNATURES = {
    "gdn_linrec_workspace_bytes": (Z, [I] * 4),
    "gdn_linrec_forward": (I, [P] * 5 + [I] * 3 + [L] * 3 + [P, I, I, I, P, Z, P]),
    "gdn_linrec_forward_plan": (I, [P] * 5 + [I] * 3 + [L] * 3 + [P, I, I, I, P, Z]),
    "gdn_linrec_backward": (I, [P] * 9 + [I] * 3 + [L] * 6 + [P, I, I, I, P, Z, P]),
    "gdn_linrec_backward_plan": (I, [P] * 9 + [I] * 3 + [L] * 6 + [P, I, I, I, P, Z]),
    "gdn_linrec_step": (I, [P] * 4 + [I] * 2 + [L] * 3 + [I] * 3 + [P]),
    "gdn_linrec_step_plan": (I, [P] * 4 + [I] * 2 + [L] * 3 + [I] * 3),
}

_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = _gdn.library()
        for name, (res, args) in LINREC_SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _bound = lib
    return _bound


# ---- entry points, same names as the C ABI ----------------------------------

def _ints(B, T, D):
    """Sizes that the C call takes as ints (ctypes would cut them to 32 bits)."""
    if max(B, T, D) > 0x7fffffff:
        raise ValueError("B, T and D must fit in 32 bits")


def gdn_linrec_workspace_bytes(B, T, D, packed=False) -> int:
    _ints(B, T, D)
    return _lib().gdn_linrec_workspace_bytes(B, T, D, int(bool(packed)))


def gdn_linrec_forward(x, log_a, h0, y, h_final, B, T, D, x_stride, a_stride, y_stride, cu_seqlens=None,
                       input_scale=LINREC_PLAIN, workspace=None, stream=None):
    """Enqueue one recurrence over sequences (layouts in include/gdn_linrec.h).  Returns the route line."""
    _ints(B, T, D)
    if y.dtype != x.dtype:
        raise TypeError("x and y must have one dtype")
    c = _Call(x)
    f32 = torch.float32
    args = (c.ptr(x), c.ptr(log_a), c.dense(h0, f32), c.ptr(y), c.dense(h_final, f32), B, T, D, x_stride, a_stride,
            y_stride, c.dense(cu_seqlens, torch.int32), input_scale, _code(x), _code(log_a), c.dense(workspace),
            _bytes(workspace))
    return c.run(_lib().gdn_linrec_forward, args, stream)


def gdn_linrec_backward(x, log_a, y, h0, dy, dh_final, dx, dlog_a, dh0, B, T, D, x_stride, a_stride, y_stride,
                        dy_stride, dx_stride, da_stride, cu_seqlens=None, input_scale=LINREC_PLAIN, workspace=None,
                        stream=None):
    """Enqueue the gradients of one recurrence; x may be None with LINREC_PLAIN.  Returns the route line."""
    _ints(B, T, D)
    dt = dy.dtype
    if y.dtype is not dt or dx.dtype is not dt or (x is not None and x.dtype is not dt):
        raise TypeError("x, y, dy and dx must have one dtype")
    if dlog_a.dtype is not log_a.dtype:
        raise TypeError("log_a and dlog_a must have one dtype")
    c = _Call(dy)
    f32 = torch.float32
    args = (c.ptr(x), c.ptr(log_a), c.ptr(y), c.dense(h0, f32), c.ptr(dy), c.dense(dh_final, f32), c.ptr(dx),
            c.ptr(dlog_a), c.dense(dh0, f32), B, T, D, x_stride, a_stride, y_stride, dy_stride, dx_stride, da_stride,
            c.dense(cu_seqlens, torch.int32), input_scale, _code(dy), _code(log_a), c.dense(workspace),
            _bytes(workspace))
    return c.run(_lib().gdn_linrec_backward, args, stream)


def gdn_linrec_step(h_table, x, log_a, y, B, D, x_stride, a_stride, y_stride, input_scale=LINREC_PLAIN, stream=None):
    """Enqueue one token of B sequences, states in place through h_table (int64 tensor of
    device pointers, 0 for a padding row).  Returns the route line."""
    _ints(B, 0, D)
    if y.dtype != x.dtype:
        raise TypeError("x and y must have one dtype")
    c = _Call(x)
    args = (c.dense(h_table, torch.int64), c.ptr(x), c.ptr(log_a), c.ptr(y), B, D, x_stride, a_stride, y_stride,
            input_scale, _code(x), _code(log_a))
    return c.run(_lib().gdn_linrec_step, args, stream)


# ---- allocation conveniences (torch allocates, the library computes) --------
# With stream= they behave like torch operators under torch.cuda.stream(stream).

def _scale(input_scale):
    try:
        return _SCALES[input_scale]
    except (KeyError, TypeError):
        raise ValueError(f"input_scale must be one of {sorted(_SCALES)}, got {input_scale!r}") from None


def _rows(t, lead):
    """Row stride of a [..., D] tensor whose leading dimensions step through rows evenly."""
    D = t.shape[-1]
    if t.stride(-1) != 1 and D > 1:
        raise ValueError("a tensor's last dimension must be contiguous")
    if len(lead) == 1:
        return t.stride(0) if lead[0] > 1 else D
    B, T = lead
    if T > 1:
        if B > 1 and t.stride(0) != T * t.stride(1):
            raise ValueError("the sequences of a dense tensor must follow each other row by row")
        return t.stride(1)
    return t.stride(0) if B > 1 else D


def _sizes(x, cu_seqlens):
    if cu_seqlens is not None:
        T, D = x.shape
        B = cu_seqlens.numel() - 1
    else:
        B, T, D = x.shape
    _ints(B, T, D)
    return B, T, D


def linrec_forward(x, log_a, h0=None, cu_seqlens=None, input_scale="plain", want_state=True, stream=None):
    """The recurrence over x [B, T, D] (or packed [T, D] with cu_seqlens), log_a of the same
    shape.  Returns (y, h_final [B, D] fp32 or None).  Packed rows that belong to no sequence
    are zeros in y."""
    B, T, D = _sizes(x, cu_seqlens)
    _shaped(log_a=(log_a, x.shape), h0=(h0, (B, D)))
    with _gdn._on_stream(stream, x.device):
        new = torch.empty if cu_seqlens is None else torch.zeros
        y = new(x.shape, dtype=x.dtype, device=x.device)
        hf = torch.empty((B, D), dtype=torch.float32, device=x.device) if want_state else None
        n = gdn_linrec_workspace_bytes(B, T, D, packed=cu_seqlens is not None)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
        lead = x.shape[:-1]
        gdn_linrec_forward(x, log_a, h0, y, hf, B, T, D, _rows(x, lead), _rows(log_a, lead), D, cu_seqlens=cu_seqlens,
                           input_scale=_scale(input_scale), workspace=ws, stream=stream)
    return y, hf


def linrec_backward(dy, x, log_a, y, h0=None, dh_final=None, cu_seqlens=None, input_scale="plain", want_dh0=None,
                    stream=None):
    """Gradients of linrec_forward; y is its output, x may be None with input_scale "plain".
    Returns a dict of dx, dlog_a and, with want_dh0 (default: where h0 is given), dh0."""
    B, T, D = _sizes(dy, cu_seqlens)
    _shaped(x=(x, dy.shape), log_a=(log_a, dy.shape), y=(y, dy.shape), h0=(h0, (B, D)), dh_final=(dh_final, (B, D)))
    scale = _scale(input_scale)
    with _gdn._on_stream(stream, dy.device):
        new = torch.empty if cu_seqlens is None else torch.zeros
        g = dict(dx=new(dy.shape, dtype=dy.dtype, device=dy.device),
                 dlog_a=new(dy.shape, dtype=log_a.dtype, device=dy.device))
        if h0 is not None if want_dh0 is None else want_dh0:
            g["dh0"] = torch.empty((B, D), dtype=torch.float32, device=dy.device)
        n = gdn_linrec_workspace_bytes(B, T, D, packed=cu_seqlens is not None)
        ws = torch.empty(n, dtype=torch.uint8, device=dy.device) if n else None
        lead = dy.shape[:-1]
        gdn_linrec_backward(x, log_a, y, h0, dy, dh_final, g["dx"], g["dlog_a"], g.get("dh0"), B, T, D,
                            D if x is None else _rows(x, lead), _rows(log_a, lead), _rows(y, lead), _rows(dy, lead),
                            D, D, cu_seqlens=cu_seqlens, input_scale=scale, workspace=ws, stream=stream)
    return g


def linrec_step(h_table, x, log_a, input_scale="plain", stream=None):
    """One token x [B, D] of B sequences whose states h_table [B] points at, in place.
    Returns y [B, D]; padding rows (a pointer 0) are zeros in it."""
    B, D = x.shape
    _ints(B, 0, D)
    _shaped(h_table=(h_table, (B,)), log_a=(log_a, x.shape))
    with _gdn._on_stream(stream, x.device):
        y = torch.zeros((B, D), dtype=x.dtype, device=x.device)
        gdn_linrec_step(h_table, x, log_a, y, B, D, _rows(x, (B,)), _rows(log_a, (B,)), D,
                        input_scale=_scale(input_scale), stream=stream)
    return y
