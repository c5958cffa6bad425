"""The vector-state recurrence and its gradients in 64 bits, row by row on the
CPU, with what an fp32 evaluation may be off (not collected by pytest).

How far fp32 may be off.  Let S_t = a_t S_{t-1} + |c x_t| be the recurrence of
the magnitudes.  At each row the decay is off by at most (2 + |l|) 2^-23 of
itself (the product with log2 e rounded, 2^-24 |l| in the exponent, and the
hardware's exp2, 2^-23), c by 2^-20 (a polynomial and a square root of values that
are each off by a few 2^-23, over 1 - a >= 0.22 where it is a difference), the
multiply-add by 2^-24.  So E_t = a_t E_{t-1} + ((4 + |l|) 2^-23 + 2^-20 [c]) S_t
bounds the row by row form.  Composing runs of rows adds one rounding of S_t's size
for each run that lies between: at most 16 in a segment and one for each segment before
it, which have 96 rows at least, or 64 under 8 channels.  64 + rows / 128 is as much for
all up to 6144 rows."""
from __future__ import annotations

import torch

F64 = torch.float64
TINY = 2.0 ** -115      # values under 2^-126 may come as zero, with factors of up to 2^10


def coefficients(l, scale):
    """a, c and dc/dl."""
    a = torch.exp(l)
    if scale == "plain":
        return a, torch.ones_like(l), torch.zeros_like(l)
    if scale == "complement":
        return a, -torch.expm1(l), -a
    c = torch.sqrt(-torch.expm1(2 * l))
    return a, c, torch.where(c > 0, -a * a / c, torch.zeros_like(c))


def runs_between(rows, D):
    return max(64 + rows / 128, 16 + rows / (64 if D < 8 else 96))


def spans(B, T, cu):
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    return list(zip(cu[:-1], cu[1:]))


def forward(x, log_a, h0, seqs, scale):
    """x, log_a [rows, D]; h0 [B, D] or None.  Returns y, h_final and what fp32 may be off for both."""
    x, l = x.to(F64), log_a.to(F64)
    D = x.shape[1]
    a, c, _ = coefficients(l, scale)
    step = (4 + l.abs().clamp(max=200)) * 2.0 ** -23 + (0.0 if scale == "plain" else 2.0 ** -20)
    y, off = torch.zeros_like(x), torch.zeros_like(x)
    hf, hoff = torch.zeros((len(seqs), D), dtype=F64), torch.zeros((len(seqs), D), dtype=F64)
    for b, (s, e) in enumerate(seqs):
        h = torch.zeros(D, dtype=F64) if h0 is None else h0[b].to(F64)
        S, E = h.abs(), torch.zeros(D, dtype=F64)
        joins = runs_between(e - s, D) * 2.0 ** -24
        for t in range(s, e):
            h = a[t] * h + c[t] * x[t]
            S = a[t] * S + (c[t] * x[t]).abs()
            E = a[t] * E + step[t] * S
            y[t], off[t] = h, E + joins * S + TINY
        hf[b], hoff[b] = h, (E + joins * S + TINY if e > s else 0 * S)
    return y, hf, off, hoff


def backward(x, log_a, y, h0, dy, dht, seqs, scale):
    """Gradients, with h_{t-1} = y[t-1] as given.  Returns dicts of values and of what fp32 may be off."""
    l, y, dy = log_a.to(F64), y.to(F64), dy.to(F64)
    x = torch.zeros_like(y) if x is None else x.to(F64)
    D = y.shape[1]
    a, c, dc = coefficients(l, scale)
    rel = (4 + l.abs().clamp(max=200)) * 2.0 ** -23
    step = rel + 2.0 ** -22
    crel = 0.0 if scale == "plain" else 2.0 ** -20
    v = {k: torch.zeros_like(y) for k in ("dx", "dlog_a")}
    o = {k: torch.zeros_like(y) for k in ("dx", "dlog_a")}
    v["dh0"], o["dh0"] = torch.zeros((len(seqs), D), dtype=F64), torch.zeros((len(seqs), D), dtype=F64)
    for b, (s, e) in enumerate(seqs):
        G = torch.zeros(D, dtype=F64) if dht is None else dht[b].to(F64)
        S, E = G.abs(), torch.zeros(D, dtype=F64)
        joins = runs_between(e - s, D) * 2.0 ** -24
        for t in reversed(range(s, e)):
            g = dy[t] + G
            M, Eg = dy[t].abs() + S, E + (joins + 2.0 ** -24) * (dy[t].abs() + S)
            before = y[t - 1] if t > s else (torch.zeros(D, dtype=F64) if h0 is None else h0[b].to(F64))
            k1, k2 = a[t] * before, dc[t] * x[t]
            v["dx"][t], o["dx"][t] = c[t] * g, c[t] * Eg + (crel + 2.0 ** -23) * (c[t] * g).abs() + TINY
            v["dlog_a"][t] = g * (k1 + k2)
            slope_off = (rel[t] + 2.0 ** -22) * k1.abs() + (rel[t] + 4 * crel + 2.0 ** -22) * k2.abs()
            o["dlog_a"][t] = Eg * (k1 + k2).abs() + (g.abs() + Eg) * slope_off + TINY
            G = a[t] * g
            S = a[t] * M
            E = a[t] * E + step[t] * S
        v["dh0"][b], o["dh0"][b] = G, (E + joins * S + TINY if e > s else 0 * S)
    return v, o
