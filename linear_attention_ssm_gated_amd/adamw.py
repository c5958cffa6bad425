"""Python binding of the AdamW step of libgdn.so (include/gdn_adamw.h): one
update over many tensors, states in fp32 or in 8 bits.

As in the package's other bindings, arguments are only marshalled and there is
no fallback.  A table holds the tensors' descriptions as the C call takes them;
build it once and hand it to every step.
"""
from __future__ import annotations

import ctypes
import struct

import torch

import linear_attention_ssm_gated_amd as _gdn

from .train import GDN_E4M3, _Call, _code, _is_codes

ADAMW_GROUP = 128   # GDN_ADAMW_GROUP of include/gdn_adamw.h

P, I, L, D, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_uint32
# name -> (restype, argtypes) of every entry point include/gdn_adamw.h declares
ADAMW_SIGNATURES = {
    "gdn_adamw_step": (I, [P, I, D, D, D, D, L, D, P, I, I, I, I, U, P]),
    "gdn_adamw_step_plan": (I, [P, I, D, D, D, D, L, D, P, I, I, I, I, U]),
}


class AdamwTensor(ctypes.Structure):
    """gdn_adamw_tensor of include/gdn_adamw.h."""
    _fields_ = [("w", P), ("master", P), ("g", P), ("m", P), ("v", P), ("m_scale", P), ("v_scale", P), ("n", L),
                ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = _gdn.library()
        for name, (res, args) in ADAMW_SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _bound = lib
    return _bound


class AdamwTable:
    """The tensors of a step: lists of contiguous tensors on one GPU, in the same order.

    weights: fp32 or bf16, updated in place; grads: fp32 or bf16; m, v: the states, fp32, or
    float8_e4m3fn (or uint8) codes with m_scales, v_scales fp32 [ceil(n / 128)]; masters: fp32,
    with bf16 weights only; weight_decay: one number, or one for each tensor.  The table keeps
    the tensors' memory alive, and steps on that memory: a tensor that gets other memory
    (t.data = ...) needs a new table, or set_grads, and one in a table must not be resized.  A
    captured step keeps the addresses it was captured with: keep its table, and its gradients
    where they are."""

    def __init__(self, weights, grads, m, v, masters=None, m_scales=None, v_scales=None, weight_decay=0.0):
        weights = list(weights)
        n = len(weights)
        decays = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(d) for d in weight_decay]
        lists = dict(grads=grads, m=m, v=v, masters=masters, m_scales=m_scales, v_scales=v_scales)
        lists = {k: None if t is None else list(t) for k, t in lists.items()}
        for k, t in lists.items():
            if t is not None and len(t) != n:
                raise ValueError(f"{k} must have one tensor for each of the {n} weights, got {len(t)}")
        if len(decays) != n:
            raise ValueError(f"weight_decay must be one number, or one for each of the {n} weights")
        if (m_scales is None) != (v_scales is None):
            raise ValueError("8-bit states need both scales")
        self.weights, self._lists, self._n = weights, lists, n
        self.entries = (AdamwTensor * max(n, 1))()
        self.w_dtype = self.state_dtype = 0
        if not n:
            self.g_dtype, self._call = 0, None
            return
        self._call = c = _Call(weights[0])
        eight = lists["m_scales"] is not None
        self.w_dtype, self.state_dtype = _code(weights[0]), GDN_E4M3 if eight else 0
        f32 = torch.float32
        if masters is not None and self.w_dtype == 0:
            raise TypeError("masters go with bf16 weights")
        for i, w in enumerate(weights):
            e, size = self.entries[i], w.numel()
            e.w, e.n, e.weight_decay = c.dense(w, weights[0].dtype), size, decays[i]
            for k, field in (("m", "m"), ("v", "v")):
                t = lists[k][i]
                if eight and not _is_codes(t):
                    raise TypeError(f"{k}: expected 8-bit codes, got {t.dtype}")
                setattr(e, field, c.dense(self._sized(t, size, k), None if eight else f32))
            if eight:
                groups = -(-size // ADAMW_GROUP)
                e.m_scale = c.dense(self._sized(lists["m_scales"][i], groups, "m_scales"), f32)
                e.v_scale = c.dense(self._sized(lists["v_scales"][i], groups, "v_scales"), f32)
            if masters is not None:
                e.master = c.dense(self._sized(lists["masters"][i], size, "masters"), f32)
        held = [p for e in self.entries if e.n for p in (e.w, e.m, e.v, e.master, e.m_scale, e.v_scale) if p]
        if len(set(held)) < len(held):
            raise ValueError("a tensor that a step changes is in the table twice")
        self._memory = [t.untyped_storage() for k in ("m", "v", "masters", "m_scales", "v_scales") for t in lists[k] or ()]
        self._memory += [w.untyped_storage() for w in weights]
        self.set_grads(lists["grads"])

    @staticmethod
    def _sized(t, n, what):
        if t.numel() != n:
            raise ValueError(f"{what} must have {n} values, got {t.numel()}")
        return t

    def set_grads(self, grads):
        """Other gradient tensors for the steps that follow."""
        grads = list(grads)
        if len(grads) != self._n:
            raise ValueError(f"grads must have one tensor for each of the {self._n} weights, got {len(grads)}")
        if not grads:
            return
        code = _code(grads[0])
        ptrs = [self._call.dense(self._sized(t, w.numel(), "grads"), grads[0].dtype) for t, w in zip(grads, self.weights)]
        for e, p in zip(self.entries, ptrs):
            e.g = p
        self._lists["grads"], self.g_dtype = grads, code
        self._grad_memory = [t.untyped_storage() for t in grads]


def gdn_adamw_step(table, lr, beta1, beta2, eps, step, grad_factor=1.0, control=None, stochastic=False, seed=0,
                   stream=None):
    """Enqueue one step over a table's tensors (formulas in include/gdn_adamw.h).  control: fp32
    [5] on the GPU (adamw_control), read in place of lr, step, grad_factor and seed.  Returns the
    route line."""
    if table._call is None:
        return "nothing to launch"
    c = table._call
    if control is not None and control.numel() != 5:
        raise ValueError("control must have 5 words")
    args = (table.entries, table._n, lr, beta1, beta2, eps, step, grad_factor, c.dense(control, torch.float32),
            table.w_dtype, table.g_dtype, table.state_dtype, int(bool(stochastic)), seed & 0xffffffff)
    return c.run(_lib().gdn_adamw_step, args, stream)


# ---- conveniences -------------------------------------------------------------

def adamw_table(weights, grads, bits=32, masters=None, weight_decay=0.0):
    """A table with new states, zeros: fp32 or, with bits=8, codes and scales.  The states are
    table.states, a dict of lists m, v (and m_scales, v_scales)."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    weights = list(weights)
    kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
    new = lambda k, d: [torch.zeros(k(w), dtype=d, device=w.device) for w in weights]  # noqa: E731
    size, groups = (lambda w: w.numel()), (lambda w: -(-w.numel() // ADAMW_GROUP))
    states = dict(m=new(size, kind), v=new(size, kind))
    if bits == 8:
        states.update(m_scales=new(groups, torch.float32), v_scales=new(groups, torch.float32))
    t = AdamwTable(weights, grads, masters=masters, weight_decay=weight_decay, **states)
    t.states = states
    return t


def adamw_control(lr, beta1, beta2, step, grad_factor=1.0, seed=0, out=None, device="cuda"):
    """The 5 words of a step's control, for steps in a captured graph: written to out (fp32 [5]
    on the GPU, on the current stream), or to a new tensor."""
    if step < 1:
        raise ValueError("need step >= 1")
    words = struct.pack("<4fI", lr, 1 - beta1 ** step, 1 - beta2 ** step, grad_factor, seed & 0xffffffff)
    host = torch.frombuffer(bytearray(words), dtype=torch.float32)
    if out is None:
        return host.to(device)
    if out.numel() != 5 or out.dtype != torch.float32:
        raise ValueError("control must be 5 fp32 words")
    return out.copy_(host)
