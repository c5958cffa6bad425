"""Plain references of the training operators in 64 bits, on the CPU (not
collected by pytest): the delta rule token by token through autograd, the norm
from its definition, and the 8-bit checkpoint bit by bit."""
from __future__ import annotations

import math

import numpy as np
import torch

F64 = torch.float64


def delta_rule(q, k, v, log_g, beta, h0):
    """One sequence: q, k [T, Hk, dk], v [T, Hv, dv], log_g, beta [T, Hv], h0
    [Hv, dk, dv]; returns o [T, Hv, dv] and the final states."""
    T, Hk, _ = q.shape
    rep = v.shape[1] // Hk
    S, o = h0, []
    for t in range(T):
        kt, qt = k[t].repeat_interleave(rep, 0), q[t].repeat_interleave(rep, 0)
        S = S * torch.exp(log_g[t])[:, None, None]
        r = beta[t][:, None] * (v[t] - (S * kt[:, :, None]).sum(1))
        S = S + kt[:, :, None] * r[:, None, :]
        o.append((S * qt[:, :, None]).sum(1))
    return (torch.stack(o) if o else v.new_zeros(v.shape)), S


def sequences(inp):
    """(first row, end) of each sequence in flattened rows, and B."""
    if inp["cu_seqlens"] is not None:
        cu = inp["cu_seqlens"].tolist()
        return list(zip(cu[:-1], cu[1:]))
    B, T = inp["q"].shape[:2]
    return [(b * T, (b + 1) * T) for b in range(B)]


def delta_rule_grads(inp, dout, dht=None):
    """Gradients of sum(o * dout) + sum(h_T * dht) in 64 bits; a dict of tensors
    laid out like the inputs (rows outside every sequence stay zero)."""
    seqs = sequences(inp)
    flat = {n: inp[n].to(F64).reshape((-1,) + inp[n].shape[(1 if inp["cu_seqlens"] is not None else 2):])
            for n in ("q", "k", "v", "log_g", "beta")}
    do = dout.to(F64).reshape((-1,) + flat["v"].shape[1:])
    Hv, dk, dv = flat["v"].shape[1], flat["q"].shape[2], flat["v"].shape[2]
    g = {n: torch.zeros_like(t) for n, t in flat.items()}
    dh0 = torch.zeros((len(seqs), Hv, dk, dv), dtype=F64)
    for b, (a, e) in enumerate(seqs):
        leaf = {n: t[a:e].clone().requires_grad_() for n, t in flat.items()}
        h0 = (inp["h0"][b].to(F64) if inp["h0"] is not None else torch.zeros((Hv, dk, dv), dtype=F64)).clone().requires_grad_()
        o, S = delta_rule(leaf["q"], leaf["k"], leaf["v"], leaf["log_g"], leaf["beta"], h0)
        loss = (o * do[a:e]).sum()
        if dht is not None:
            loss = loss + (S * dht[b].to(F64)).sum()
        names = list(leaf)
        if loss.requires_grad:
            got = torch.autograd.grad(loss, [leaf[n] for n in names] + [h0], allow_unused=True)
            for n, t in zip(names, got):
                if t is not None:
                    g[n][a:e] = t
            if got[-1] is not None:
                dh0[b] = got[-1]
    out = {("d" + n): t.reshape(inp[n].shape) for n, t in g.items()}
    out["dh0"] = dh0
    return out


def norm(x, w, z=None, b=None, eps=1e-6, center=False):
    m = x.mean(-1, keepdim=True) if center else 0.0
    n = (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    a = n * w if b is None else n * w + b
    return a if z is None else a * z * torch.sigmoid(z)


def norm_grads(dy, x, w, z=None, b=None, eps=1e-6, center=False):
    leaf = {"x": x.to(F64).clone().requires_grad_(), "w": w.to(F64).clone().requires_grad_()}
    if z is not None:
        leaf["z"] = z.to(F64).clone().requires_grad_()
    if b is not None:
        leaf["b"] = b.to(F64).clone().requires_grad_()
    y = norm(leaf["x"], leaf["w"], leaf.get("z"), leaf.get("b"), eps, center)
    got = torch.autograd.grad(y, list(leaf.values()), dy.to(F64))
    return {"d" + n: t for n, t in zip(leaf, got)}


# e4m3's 256 values: sign, 4 exponent bits (bias 7), 3 mantissa bits, NaN at 0x7f
def e4m3_values():
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        f = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = math.nan if c & 127 == 127 else (-f if c & 128 else f)
    return out


def ckpt8(x):
    """(codes uint8, exps uint8) of fp64 rows [rows, d], by nearest search over
    the 127 positive values, ties to the even code."""
    vals = e4m3_values()[:127]
    rows, d = x.shape
    ng = -(-d // 128)
    codes, exps = np.zeros((rows, d), np.uint8), np.zeros((rows, ng), np.uint8)
    for r in range(rows):
        for g in range(ng):
            v = x[r, 128 * g: 128 * (g + 1)]
            a = np.abs(v)
            top = a[np.isfinite(a)].max(initial=0.0)
            e = 0
            if top > 0:
                e = -126
                while top > 448.0 * 2.0 ** e:
                    e += 1
            exps[r, g] = e + 127
            s = np.where(np.isfinite(v), v, 0.0) / 2.0 ** e
            hi = np.clip(np.searchsorted(vals, np.abs(s)), 1, 126)
            lo = hi - 1
            dl, dh = np.abs(s) - vals[lo], vals[hi] - np.abs(s)
            c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
            c = np.where(np.signbit(s), c | 128, c)
            codes[r, 128 * g: 128 * (g + 1)] = np.where(np.isfinite(v), c, 127)
    return codes, exps


def two_norm(got, ref):
    """|got - ref| / |ref| in the 2-norm, in 64 bits."""
    g, r = got.detach().cpu().to(F64), ref.to(F64)
    n = float(r.norm())
    d = float((g - r).norm())
    return d / n if n else d
