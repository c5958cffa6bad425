"""Python binding of the training entry points of libgdn.so
(include/gdn_train.h): the delta rule's gradients, the norm of its outputs with
its gradients, and 8-bit activation checkpoints.

As in the package's other bindings, arguments are only marshalled and there is
no fallback.  Tensors may be views: strides are arguments of the calls, and a
tensor's values start at its data pointer.  All tensors of a call must be on
one GPU; the call is made with that GPU current and, unless a stream is given,
on its current stream.
"""
from __future__ import annotations

import ctypes

import torch

import linear_attention_ssm_gated_amd as _gdn

GDN_E4M3 = 2
CKPT8_GROUP = 128   # GDN_CKPT8_GROUP of include/gdn_train.h

P, I, Z, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64, ctypes.c_float
# name -> (restype, argtypes) of every entry point include/gdn_train.h declares
TRAIN_SIGNATURES = {
    "gdn_ckpt8_store": (I, [P, P, P, L, I, L, I, P]),
    "gdn_ckpt8_store_plan": (I, [P, P, P, L, I, L, I]),
    "gdn_ckpt8_load": (I, [P, P, P, L, I, L, I, P]),
    "gdn_ckpt8_load_plan": (I, [P, P, P, L, I, L, I]),
    "gdn_norm_workspace_bytes": (Z, [I, I, I]),
    "gdn_norm_forward": (I, [P] * 9 + [I] * 3 + [L] * 3 + [F, I, I, P]),
    "gdn_norm_forward_plan": (I, [P] * 9 + [I] * 3 + [L] * 3 + [F, I, I]),
    "gdn_norm_backward": (I, [P] * 11 + [I] * 3 + [L] * 5 + [F, I, I, I, P, Z, P]),
    "gdn_norm_backward_plan": (I, [P] * 11 + [I] * 3 + [L] * 5 + [F, I, I, I, P, Z]),
    "gdn_backward_workspace_bytes": (Z, [I] * 9),
    "gdn_chunk_backward": (I, [P] * 17 + [I] * 6 + [P, I, I, P, Z, P]),
    "gdn_chunk_backward_plan": (I, [P] * 17 + [I] * 6 + [P, I, I, P, Z]),
}

_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = _gdn.library()
        for name, (res, args) in TRAIN_SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _bound = lib
    return _bound


# The current stream's handle without a Stream object where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Call:
    """Pointers of one call's tensors, which must all be on one GPU."""
    __slots__ = ("device",)

    def __init__(self, first):
        self.device = first.get_device()
        if self.device < 0:
            raise ValueError("tensors must live on the GPU")

    def ptr(self, t, dtype=None):
        """A tensor whose values along the last dimension are contiguous."""
        if t is None:
            return None
        if t.get_device() != self.device:
            raise ValueError("tensors of one call must live on one GPU")
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"expected {dtype}, got {t.dtype}")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("a tensor's last dimension must be contiguous")
        return t.data_ptr()

    def dense(self, t, dtype=None):
        if t is None:
            return None
        if t.get_device() != self.device:
            raise ValueError("tensors of one call must live on one GPU")
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"expected {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return t.data_ptr()

    def run(self, fn, args, stream):
        dev = self.device
        if dev == torch.cuda.current_device():
            if stream is None and _raw_stream is not None:
                status = fn(*args, _raw_stream(dev))
            else:
                status = fn(*args, _gdn._stream(stream))
        else:
            with torch.cuda.device(dev):
                status = fn(*args, _gdn._stream(stream))
        if status != 0:
            raise _gdn.GdnError(status, _gdn.last_route())
        return _bound.gdn_last_route().decode()


_CODES = {torch.float32: 0, torch.bfloat16: 1}


def _code(t):
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _is_codes(t):
    return t is not None and t.dtype in (torch.uint8, torch.float8_e4m3fn)


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


# ---- entry points, same names as the C ABI ----------------------------------

def gdn_ckpt8_store(x, codes, exps, rows, d, x_stride, stream=None):
    """Enqueue one 8-bit checkpoint of x [rows][x_stride].  Returns the route line."""
    c = _Call(x)
    args = (c.ptr(x), c.dense(codes), c.dense(exps, torch.uint8), rows, d, x_stride, _code(x))
    return c.run(_lib().gdn_ckpt8_store, args, stream)


def gdn_ckpt8_load(codes, exps, y, rows, d, y_stride, stream=None):
    """Enqueue the reading back of one 8-bit checkpoint.  Returns the route line."""
    c = _Call(y)
    args = (c.dense(codes), c.dense(exps, torch.uint8), c.ptr(y), rows, d, y_stride, _code(y))
    return c.run(_lib().gdn_ckpt8_load, args, stream)


def gdn_norm_workspace_bytes(T, H, d) -> int:
    return _lib().gdn_norm_workspace_bytes(T, H, d)


def gdn_norm_forward(x, z, w, b, y, x_codes, x_exps, z_codes, z_exps, T, H, d, x_stride, z_stride, y_stride,
                     eps, center, stream=None):
    """Enqueue one norm (layouts in include/gdn_train.h).  Returns the route line."""
    if y.dtype != x.dtype or (z is not None and z.dtype != x.dtype):
        raise TypeError("x, z and y must have one dtype")
    c = _Call(x)
    u8, f32 = torch.uint8, torch.float32
    args = (c.ptr(x), c.ptr(z), c.dense(w, f32), c.dense(b, f32), c.ptr(y), c.dense(x_codes),
            c.dense(x_exps, u8), c.dense(z_codes), c.dense(z_exps, u8), T, H, d, x_stride, z_stride, y_stride,
            eps, int(bool(center)), _code(x))
    return c.run(_lib().gdn_norm_forward, args, stream)


def gdn_norm_backward(x, x_exps, z, z_exps, w, b, dy, dx, dz, dw, db, T, H, d, x_stride, z_stride, dy_stride,
                      dx_stride, dz_stride, eps, center, workspace=None, stream=None):
    """Enqueue the gradients of one norm; x and z may be code tensors (uint8 or
    float8_e4m3fn) with their exps.  Returns the route line."""
    if dx.dtype != dy.dtype or (dz is not None and dz.dtype != dy.dtype):
        raise TypeError("dy, dx and dz must have one dtype")
    io = _code(dy)
    act = GDN_E4M3 if _is_codes(x) else _code(x)
    if z is not None and (GDN_E4M3 if _is_codes(z) else _code(z)) != act:
        raise TypeError("x and z must have one dtype")
    c = _Call(dy)
    u8, f32 = torch.uint8, torch.float32
    args = (c.ptr(x), c.dense(x_exps, u8), c.ptr(z), c.dense(z_exps, u8), c.dense(w, f32), c.dense(b, f32),
            c.ptr(dy), c.ptr(dx), c.ptr(dz), c.dense(dw, f32), c.dense(db, f32), T, H, d, x_stride, z_stride,
            dy_stride, dx_stride, dz_stride, eps, int(bool(center)), act, io, c.dense(workspace),
            _bytes(workspace))
    return c.run(_lib().gdn_norm_backward, args, stream)


def gdn_backward_workspace_bytes(B, T, Hk, Hv, dk, dv, io_dtype, grad_dtype, packed=False) -> int:
    return _lib().gdn_backward_workspace_bytes(B, T, Hk, Hv, dk, dv, io_dtype, grad_dtype, int(bool(packed)))


def gdn_chunk_backward(q, k, v, q_exps, k_exps, v_exps, log_g, beta, h0, dout, dh_final, dq, dk_out, dv_out,
                       dlog_g, dbeta, dh0, B, T, Hk, Hv, dk, dv, cu_seqlens=None, workspace=None, stream=None):
    """Enqueue the gradients of one chunked prefill (include/gdn_train.h); q, k
    and v may be code tensors (uint8 or float8_e4m3fn) with their exps.  Returns
    the route line."""
    io = GDN_E4M3 if _is_codes(q) else _code(q)
    for t in (k, v):
        if (GDN_E4M3 if _is_codes(t) else _code(t)) != io:
            raise TypeError("q, k and v must have one dtype")
    grad = _code(dout)
    for t in (dq, dk_out, dv_out, dlog_g, dbeta):
        if t.dtype != dout.dtype:
            raise TypeError("dout, dq, dk, dv, dlog_g and dbeta must have one dtype")
    c = _Call(dout)
    u8, f32 = torch.uint8, torch.float32
    p = c.dense
    args = (p(q), p(k), p(v), p(q_exps, u8), p(k_exps, u8), p(v_exps, u8), p(log_g, f32), p(beta, f32),
            p(h0, f32), p(dout), p(dh_final, f32), p(dq), p(dk_out), p(dv_out), p(dlog_g), p(dbeta),
            p(dh0, f32), B, T, Hk, Hv, dk, dv, p(cu_seqlens, torch.int32), io, grad, p(workspace),
            _bytes(workspace))
    return c.run(_lib().gdn_chunk_backward, args, stream)


# ---- allocation conveniences (torch allocates, the library computes) --------
# With stream= they behave like torch operators under torch.cuda.stream(stream):
# workspace and outputs come from that stream's memory pool.

def _shaped(**want):
    """Refuse a tensor whose shape the kernels would read beyond."""
    for name, (t, shape) in want.items():
        if t is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _row_width(t):
    """Width of t's rows, which the C call takes as an int."""
    d = t.shape[-1]
    if d > 1 << 30:
        raise ValueError("a row has at most 2^30 values: give a long tensor rows")
    return d


def _exps_shape(rows, d):
    return rows, -(-d // CKPT8_GROUP)


def _token_rows(t):
    """Token stride of a [T, H, d] tensor whose heads lie next to each other."""
    T, H, d = t.shape
    if T and ((H > 1 and t.stride(1) != d) or (d > 1 and t.stride(2) != 1)):
        raise ValueError("a token's heads must be contiguous")
    return t.stride(0) if T > 1 else H * d


def ckpt8_store(x, stream=None):
    """8-bit checkpoint of a contiguous x [..., d].  Returns (codes
    float8_e4m3fn of x's shape, exps uint8 [rows, ceil(d / 128)])."""
    if not x.is_contiguous():
        raise ValueError("tensors must be contiguous")
    d = _row_width(x)
    rows = x.numel() // d if d else 0
    with _gdn._on_stream(stream, x.device):
        codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        exps = torch.empty(_exps_shape(rows, d), dtype=torch.uint8, device=x.device)
        gdn_ckpt8_store(x, codes, exps, rows, d, d, stream=stream)
    return codes, exps


def ckpt8_load(codes, exps, dtype=torch.bfloat16, stream=None):
    """The values of an 8-bit checkpoint as a tensor of codes' shape."""
    d = _row_width(codes)
    rows = codes.numel() // d if d else 0
    _shaped(exps=(exps, _exps_shape(rows, d)))
    with _gdn._on_stream(stream, codes.device):
        y = torch.empty(codes.shape, dtype=dtype, device=codes.device)
        gdn_ckpt8_load(codes, exps, y, rows, d, d, stream=stream)
    return y


def norm_forward(x, w, z=None, b=None, eps=1e-6, center=False, ckpt=False, stream=None):
    """Norm of x [T, H, d], times silu(z).  Returns (y, checkpoints), the
    checkpoints a dict of x_codes, x_exps (and z_codes, z_exps) with ckpt=True."""
    T, H, d = x.shape
    _shaped(z=(z, x.shape), w=(w, (d,)), b=(b, (d,)))
    with _gdn._on_stream(stream, x.device):
        y = torch.empty((T, H, d), dtype=x.dtype, device=x.device)
        kept = {}
        if ckpt:
            for name, t in (("x", x), ("z", z)):
                if t is not None:
                    kept[name + "_codes"] = torch.empty((T, H, d), dtype=torch.float8_e4m3fn, device=x.device)
                    kept[name + "_exps"] = torch.empty(_exps_shape(T * H, d), dtype=torch.uint8, device=x.device)
        gdn_norm_forward(x, z, w, b, y, kept.get("x_codes"), kept.get("x_exps"), kept.get("z_codes"),
                         kept.get("z_exps"), T, H, d, _token_rows(x), H * d if z is None else _token_rows(z),
                         H * d, eps, center, stream=stream)
    return y, kept


def norm_backward(dy, x, w, z=None, b=None, x_exps=None, z_exps=None, eps=1e-6, center=False, stream=None):
    """Gradients of norm_forward from x and z, or from their code tensors with
    exps.  Returns a dict of dx, dw (and dz, db)."""
    T, H, d = x.shape
    exps = _exps_shape(T * H, d)
    _shaped(dy=(dy, x.shape), z=(z, x.shape), w=(w, (d,)), b=(b, (d,)), x_exps=(x_exps, exps), z_exps=(z_exps, exps))
    with _gdn._on_stream(stream, dy.device):
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=dy.device)  # noqa: E731
        g = dict(dx=new((T, H, d), dy.dtype), dw=new(d, torch.float32))
        if z is not None:
            g["dz"] = new((T, H, d), dy.dtype)
        if b is not None:
            g["db"] = new(d, torch.float32)
        n = gdn_norm_workspace_bytes(T, H, d)
        ws = new(n, torch.uint8) if n else None
        gdn_norm_backward(x, x_exps, z, z_exps, w, b, dy, g["dx"], g.get("dz"), g["dw"], g.get("db"), T, H, d,
                          _token_rows(x), H * d if z is None else _token_rows(z), _token_rows(dy), H * d, H * d,
                          eps, center, workspace=ws, stream=stream)
    return g


def chunk_backward(q, k, v, log_g, beta, dout, h0=None, dh_final=None, cu_seqlens=None, q_exps=None,
                   k_exps=None, v_exps=None, want_dh0=None, stream=None):
    """Gradients of chunk_prefill.  Dense or packed layouts as there; q, k, v
    may be code tensors with their exps.  Returns (dict of dq, dk, dv, dlog_g,
    dbeta and, with want_dh0 (default: where h0 is given), dh0; route line)."""
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        T, Hk, dk = q.shape
    else:
        B, T, Hk, dk = q.shape
    Hv, dv = v.shape[-2], v.shape[-1]
    rows, state = q.shape[:-2], (B, Hv, dk, dv)
    _shaped(k=(k, q.shape), v=(v, (*rows, Hv, dv)), log_g=(log_g, (*rows, Hv)), beta=(beta, (*rows, Hv)),
            dout=(dout, v.shape), h0=(h0, state), dh_final=(dh_final, state))
    n = rows.numel()
    _shaped(q_exps=(q_exps, _exps_shape(n * Hk, dk)), k_exps=(k_exps, _exps_shape(n * Hk, dk)),
            v_exps=(v_exps, _exps_shape(n * Hv, dv)))
    dt, dev = dout.dtype, dout.device
    with _gdn._on_stream(stream, dev):
        new = lambda shape, t=dt: torch.empty(shape, dtype=t, device=dev)  # noqa: E731
        g = dict(dq=new(q.shape), dk=new(k.shape), dv=new(v.shape), dlog_g=new(log_g.shape), dbeta=new(beta.shape))
        if h0 is not None if want_dh0 is None else want_dh0:
            g["dh0"] = new(state, torch.float32)
        io = GDN_E4M3 if _is_codes(q) else _code(q)
        n = gdn_backward_workspace_bytes(B, T, Hk, Hv, dk, dv, io, _code(dout), packed=cu_seqlens is not None)
        ws = new(n, torch.uint8) if n else None
        route = gdn_chunk_backward(q, k, v, q_exps, k_exps, v_exps, log_g, beta, h0, dout, dh_final, g["dq"],
                                   g["dk"], g["dv"], g["dlog_g"], g["dbeta"], g.get("dh0"), B, T, Hk, Hv, dk, dv,
                                   cu_seqlens=cu_seqlens, workspace=ws, stream=stream)
    return g, route
