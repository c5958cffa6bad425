"""The training operators of the gated delta rule, case by case: what they are
timed on, their plain forms in elementary torch operations, and their values in
64 bits.

Three operators that one training step of a layer uses together:

* ``backward``: the gradients of the chunked gated delta rule with respect to
  q, k, v, the log decays, beta and the initial state;
* ``norm_forward`` / ``norm_backward``: the layer norm (or RMS norm) of the
  recurrence's outputs, per head, times silu of a gate, and its gradients, the
  weight's and the bias's among them; with one head it is the norm over a
  hidden row;
* ``store8`` / ``load8``: activation checkpoints in 8 bits (e4m3 codes and one
  power-of-two scale per 128 values), which both backward passes read in place
  of the bf16 activations.

``run`` computes the plain form, or with ``own`` calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

CHUNK = 64      # rows of one chunk of the plain form's closed form
GROUP = 128     # values that share one scale of an 8-bit checkpoint
EPS = 1e-6

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------

def _bwd(name, dtype, B, T, Hk, Hv, dk, dv, packed=False, h0=False, ckpt=False):
    return dict(name=name, op="backward", dtype=dtype, B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv,
                packed=packed, h0=h0, ckpt=ckpt)


def _norm(name, op, dtype, T, H, d, center=False, gate=True, bias=False, ckpt=False, zpad=0):
    return dict(name=name, op=op, dtype=dtype, T=T, H=H, d=d, center=center, gate=gate, bias=bias,
                ckpt=ckpt, zpad=zpad)


def _pack(name, op, dtype, rows, d, pad=0):
    return dict(name=name, op=op, dtype=dtype, rows=rows, d=d, pad=pad)


def listed():
    return [
        # one long training sequence through a full layer: the largest call
        _bwd("backward 4576", "bf16", 1, 4576, 16, 48, 128, 128),
        # packed documents of ragged lengths, activations kept in 8 bits
        _bwd("backward packed ckpt8", "bf16", 6, 2371, 16, 48, 128, 128, packed=True, ckpt=True),
        # a narrow layer (a head-parallel share) on a short ragged batch: latency counts
        _bwd("backward narrow 200", "bf16", 2, 200, 2, 6, 128, 128),
        # fp32 with small heads, states handed over between two calls: dh0 comes back
        _bwd("backward f32 states", "f32", 2, 500, 2, 6, 64, 96, h0=True),
        # the layer's output norm with its gate, checkpoints of both kept for the backward
        _norm("norm gated 4576x48", "norm_forward", "bf16", 4576, 48, 128, ckpt=True),
        # the same norm behind a decode step of 16 sequences
        _norm("norm decode 16x48", "norm_forward", "bf16", 16, 48, 128),
        # its gradients from bf16 activations, the gate a column block of a fused projection
        _norm("norm backward 4576x48", "norm_backward", "bf16", 4576, 48, 128, zpad=640),
        # its gradients from 8-bit checkpoints
        _norm("norm backward ckpt8", "norm_backward", "bf16", 2371, 48, 128, ckpt=True),
        # layer norm over the hidden row ahead of the projections, with bias, fp32
        _norm("norm backward hidden f32", "norm_backward", "f32", 1168, 1, 5120, center=True,
              gate=False, bias=True),
        # checkpoints of v for one long sequence
        _pack("store8 v 4576x48", "store8", "bf16", 4576 * 48, 128),
        # an odd width with a ragged last group, rows of a wider buffer
        _pack("store8 odd f32", "store8", "f32", 1000, 333, pad=3),
        # reading back a checkpoint as bf16
        _pack("load8 v 2371x48", "load8", "bf16", 2371 * 48, 128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["backward", "backward", "norm_forward", "norm_backward", "norm_backward",
                     "store8", "load8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "backward":
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        packed = rng.random() < 0.4
        if dtype == "bf16":
            Hv = Hk * rng.choice([1, 2, 3])
            n = _log_int(rng, 60, min(6000, 4576 * 48 // Hv))
            dk = dv = 128
        else:
            Hk = min(Hk, 4)
            Hv = Hk * rng.choice([1, 2, 3])
            n = _log_int(rng, 1, 900)
            dk, dv = rng.choice([16, 24, 32, 40, 64, 96, 100, 128]), rng.choice([16, 20, 32, 48, 64, 96, 128])
        B = rng.randint(1, 8) if packed else rng.randint(1, 3)
        T = max(B, n) if packed else max(1, n // B)
        c = _bwd("", dtype, B, T, Hk, Hv, dk, dv, packed=packed,
                 h0=dtype == "f32" and not packed and rng.random() < 0.6,
                 ckpt=dtype == "bf16" and rng.random() < 0.5)
    elif op in ("norm_forward", "norm_backward"):
        if rng.random() < 0.6:
            H, d = rng.choice([1, 2, 6, 16, 48]), rng.choice([32, 64, 80, 100, 128, 192, 256])
        else:
            H, d = 1, _log_int(rng, 300, 8000)
        T = _log_int(rng, 1, max(1, 4576 * 48 * 128 // (H * d) // (4 if dtype == "f32" else 2)))
        gate = rng.random() < 0.6
        c = _norm("", op, dtype, min(T, 20000), H, d, center=rng.random() < 0.5, gate=gate,
                  bias=rng.random() < 0.5, ckpt=dtype == "bf16" and rng.random() < 0.5)
        if gate and not c["ckpt"]:
            c["zpad"] = rng.choice([0, 0, 8, 77])
    else:
        d = rng.choice([16, 64, 100, 128, 128, 256, 333, 1000, 5120])
        rows = _log_int(rng, 1, 4576 * 48 * 128 // d // 2)
        c = _pack("", op, dtype, rows, d, pad=rng.choice([0, 0, 0, 5, 16]))
    del c["name"]
    return c


# ---- inputs -----------------------------------------------------------------

def _lengths(case):
    """Lengths of a packed case's sequences: ragged, at least 1 each, T in all."""
    B, T = case["B"], case["T"]
    r = random.Random(T * 131 + B)
    w = [r.uniform(0.3, 1.7) for _ in range(B)]
    cut = [1 + int((T - B) * x / sum(w)) for x in w]
    cut[-1] += T - sum(cut)
    return cut


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _unit(gen, shape, dtype):
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def _pow2(e):
    """2^e as fp32, from its bits (-126 <= e <= 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes_of(x):
    """8-bit checkpoint of x [rows, d]: e4m3 codes and one exponent byte per
    128 values, the scale 2^(byte - 127) the smallest power of two that brings
    the group's largest finite magnitude to 448 or less."""
    rows, d = x.shape
    n = -(-d // GROUP)
    f = torch.zeros(rows, n * GROUP, dtype=torch.float32, device=x.device)
    f[:, :d] = x
    f = f.view(rows, n, GROUP)
    a = f.abs()
    top = torch.where(a < math.inf, a, torch.zeros_like(a)).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 119)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    f = torch.where(a < math.inf, f * _pow2(-e)[..., None], torch.full_like(f, math.nan))
    codes = f.to(torch.float8_e4m3fn).view(rows, n * GROUP)[:, :d].contiguous()
    return codes, (e + 127).to(torch.uint8)


def _values_of(codes, exps):
    """The fp32 values that an 8-bit checkpoint stands for."""
    rows, d = codes.shape
    s = _pow2(exps.to(torch.int32) - 127).repeat_interleave(GROUP, dim=1)[:, :d]
    return codes.to(torch.float32) * s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case=dict(case), op=op)
    if op == "backward":
        B, T, Hk, Hv, dk, dv = (case[x] for x in ("B", "T", "Hk", "Hv", "dk", "dv"))
        n = T if case["packed"] else B * T
        lead = (T,) if case["packed"] else (B, T)
        q, k = _unit(gen, lead + (Hk, dk), dt), _unit(gen, lead + (Hk, dk), dt)
        v = _normal(gen, lead + (Hv, dv), dt)
        s["log_g"] = -torch.nn.functional.softplus(_normal(gen, lead + (Hv,), torch.float32)) * 0.1
        s["beta"] = torch.sigmoid(_normal(gen, lead + (Hv,), torch.float32))
        s["dout"] = _normal(gen, lead + (Hv, dv), dt)
        s["q"], s["k"], s["v"] = q, k, v
        s["q_exps"] = s["k_exps"] = s["v_exps"] = None
        if case["ckpt"]:
            for x in "qkv":
                t = s[x]
                c, e = _codes_of(t.reshape(-1, t.shape[-1]))
                s[x], s[x + "_exps"] = c.view(t.shape), e
        s["h0"] = s["dht"] = s["dh0"] = None
        if case["h0"]:
            s["h0"] = _normal(gen, (B, Hv, dk, dv), torch.float32, 0.02)
            s["dht"] = _normal(gen, (B, Hv, dk, dv), torch.float32, 0.02)
            s["dh0"] = torch.empty_like(s["h0"])
        s["dq"], s["dk"] = torch.empty(q.shape, dtype=dt, device="cuda"), torch.empty(q.shape, dtype=dt, device="cuda")
        s["dv"] = torch.empty(v.shape, dtype=dt, device="cuda")
        s["dlog_g"] = torch.empty(lead + (Hv,), dtype=dt, device="cuda")
        s["dbeta"] = torch.empty(lead + (Hv,), dtype=dt, device="cuda")
        lens = _lengths(case) if case["packed"] else [T] * B
        first = [sum(lens[:i]) for i in range(B + 1)]
        s["longest"] = max(lens)
        s["cu"] = torch.tensor(first, dtype=torch.int32, device="cuda")
    elif op in ("norm_forward", "norm_backward"):
        T, H, d = case["T"], case["H"], case["d"]
        x = _normal(gen, (T, H, d), dt, 0.3)
        s["x"], s["x_exps"], s["z"], s["z_exps"] = x, None, None, None
        if case["gate"]:
            wide = _normal(gen, (T, H * d + case["zpad"]), dt)
            s["z"] = wide[:, case["zpad"]:].unflatten(1, (H, d))
        s["w"] = 1.0 + _normal(gen, (d,), torch.float32, 0.1)
        s["b"] = _normal(gen, (d,), torch.float32, 0.1) if case["bias"] else None
        n = -(-d // GROUP)
        if op == "norm_forward":
            s["y"] = torch.empty((T, H, d), dtype=dt, device="cuda")
            for a in "xz":
                keep = case["ckpt"] and s[a] is not None
                s[a + "_codes"] = torch.empty((T * H, d), dtype=torch.uint8, device="cuda") if keep else None
                s[a + "_exps"] = torch.empty((T * H, n), dtype=torch.uint8, device="cuda") if keep else None
        else:
            s["dy"] = _normal(gen, (T, H, d), dt)
            if case["ckpt"]:
                for a in "xz":
                    if s[a] is not None:
                        c, e = _codes_of(s[a].reshape(-1, d))
                        s[a], s[a + "_exps"] = c.view(T, H, d), e
            s["dx"] = torch.empty((T, H, d), dtype=dt, device="cuda")
            s["dz"] = torch.empty((T, H, d), dtype=dt, device="cuda") if case["gate"] else None
            s["dw"] = torch.empty(d, dtype=torch.float32, device="cuda")
            s["db"] = torch.empty(d, dtype=torch.float32, device="cuda") if case["bias"] else None
    else:
        rows, d, pad = case["rows"], case["d"], case["pad"]
        # rows of very different sizes, as activations of different layers and tokens are
        size = torch.exp2(torch.randint(-12, 6, (rows, 1), generator=gen, device="cuda").float())
        wide = (torch.randn((rows, d + pad), generator=gen, device="cuda") * size).to(dt)
        n = -(-d // GROUP)
        if op == "store8":
            s["x"] = wide[:, :d]
            s["codes"] = torch.empty((rows, d), dtype=torch.uint8, device="cuda")
            s["exps"] = torch.empty((rows, n), dtype=torch.uint8, device="cuda")
        else:
            s["codes"], s["exps"] = _codes_of(wide[:, :d])
            s["y"] = torch.empty((rows, d), dtype=dt, device="cuda")
    return s


# ---- the calls --------------------------------------------------------------

def _own(s):
    import linear_attention_ssm_gated_amd as gdn
    c, op = s["case"], s["op"]
    code = {torch.bfloat16: gdn.GDN_BF16, torch.float32: gdn.GDN_F32}
    if op == "backward":
        B, T, Hk, Hv, dk, dv = (c[x] for x in ("B", "T", "Hk", "Hv", "dk", "dv"))
        io = gdn.GDN_E4M3 if c["ckpt"] else code[DTYPES[c["dtype"]]]
        if "ws" not in s:
            n = gdn.gdn_backward_workspace_bytes(B, T, Hk, Hv, dk, dv, io, code[s["dq"].dtype], c["packed"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        gdn.gdn_chunk_backward(s["q"], s["k"], s["v"], s["q_exps"], s["k_exps"], s["v_exps"], s["log_g"],
                               s["beta"], s["h0"], s["dout"], s["dht"], s["dq"], s["dk"], s["dv"],
                               s["dlog_g"], s["dbeta"], s["dh0"], B, T, Hk, Hv, dk, dv,
                               cu_seqlens=s["cu"] if c["packed"] else None, workspace=s["ws"])
        out = {x: s[x] for x in ("dq", "dk", "dv", "dlog_g", "dbeta")}
        if s["dh0"] is not None:
            out["dh0"] = s["dh0"]
        return out
    if op == "norm_forward":
        T, H, d = c["T"], c["H"], c["d"]
        gdn.gdn_norm_forward(s["x"], s["z"], s["w"], s["b"], s["y"], s["x_codes"], s["x_exps"], s["z_codes"],
                             s["z_exps"], T, H, d, H * d, H * d + c["zpad"], H * d, EPS, c["center"])
        out = {"y": s["y"]}
        for a in "xz":
            if s[a + "_codes"] is not None:
                out[a + "_codes"], out[a + "_exps"] = s[a + "_codes"].view(torch.float8_e4m3fn), s[a + "_exps"]
        return out
    if op == "norm_backward":
        T, H, d = c["T"], c["H"], c["d"]
        if "ws" not in s:
            s["ws"] = torch.empty(gdn.gdn_norm_workspace_bytes(T, H, d), dtype=torch.uint8, device="cuda")
        gdn.gdn_norm_backward(s["x"], s["x_exps"], s["z"], s["z_exps"], s["w"], s["b"], s["dy"], s["dx"],
                              s["dz"], s["dw"], s["db"], T, H, d, H * d, H * d + c["zpad"], H * d, H * d,
                              H * d, EPS, c["center"], workspace=s["ws"])
        return {x: s[x] for x in ("dx", "dz", "dw", "db") if s[x] is not None}
    if op == "store8":
        gdn.gdn_ckpt8_store(s["x"], s["codes"], s["exps"], c["rows"], c["d"], c["d"] + c["pad"])
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "exps": s["exps"]}
    gdn.gdn_ckpt8_load(s["codes"], s["exps"], s["y"], c["rows"], c["d"], c["d"])
    return {"y": s["y"]}


def _plain_backward(s):
    """Per chunk of 64 rows, with G the running sum of log_g, B_rs =
    exp(G_r - G_s) k_r.k_s (s < r), P_rs = exp(G_r - G_s) q_r.k_s (s <= r),
    T = (I + B diag(beta))^-1, E_s = exp(G_L - G_s):
        u = T (v - exp(G) K h),   delta = beta u,   h' = exp(G_L) h + K^T E delta
    and the adjoints of these lines.  The chunk states follow one affine map
    each, h' = M h + N, and their adjoints its transpose."""
    c = s["case"]
    B, Hk, Hv, dk, dv = (c[x] for x in ("B", "Hk", "Hv", "dk", "dv"))
    f32, dev = torch.float32, s["dout"].device
    N = -(-s["longest"] // CHUNK)
    cu = s["cu"].long()
    t = torch.arange(N * CHUNK, device=dev)
    at = cu[:-1, None] + t                                   # row of (sequence, place)
    there = t < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(there, at, torch.zeros_like(at))

    def take(x, heads, dtype=f32):                           # [B, heads, N, CHUNK, ...]
        x = x.reshape((-1,) + x.shape[-(x.dim() - (1 if c["packed"] else 2)):]).to(dtype)
        x = x[at] * there.view(there.shape + (1,) * (x.dim() - 1)).to(dtype)
        return x.unflatten(1, (N, CHUNK)).movedim(3, 1)

    vals = {}
    for x in "qkv":
        y = s[x]
        if s[x + "_exps"] is not None:
            y = _values_of(y.reshape(-1, y.shape[-1]), s[x + "_exps"]).view(y.shape)
        vals[x] = take(y, y.shape[-2])
    rep = Hv // Hk
    q, k, v = vals["q"].repeat_interleave(rep, 1), vals["k"].repeat_interleave(rep, 1), vals["v"]
    do = take(s["dout"], Hv)
    beta, G = take(s["beta"], Hv), take(s["log_g"], Hv, torch.float64).cumsum(-1)
    ga, E = torch.exp(G).to(f32), torch.exp(G[..., -1:] - G).to(f32)
    gL = ga[..., -1:, None]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    gam = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).to(f32)
    kk = ((k @ k.mT) * gam).tril(-1)
    P = (q @ k.mT) * gam
    eye = torch.eye(CHUNK, device=dev)
    T = torch.linalg.solve_triangular(eye + kk * beta[..., None, :], eye.expand_as(kk), upper=False, unitriangular=True)
    col = lambda x: x[..., None]  # noqa: E731
    W = col(E * beta) * (T @ (col(ga) * k))
    U = col(E * beta) * (T @ v)
    M = gL * torch.eye(dk, device=dev) - k.mT @ W
    add = k.mT @ U
    PT = (P * beta[..., None, :]) @ T
    back = col(ga) * q - PT @ (col(ga) * k)
    dadd = back.mT @ do
    h = s["h0"] if s["h0"] is not None else torch.zeros(B, Hv, dk, dv, device=dev)
    dh = s["dht"] if s["dht"] is not None else torch.zeros(B, Hv, dk, dv, device=dev)
    hs, dhs = [], []
    for i in range(N):                                       # the recurrence, one product a chunk
        hs.append(h)
        h = add[:, :, i] + M[:, :, i] @ h
    for i in reversed(range(N)):
        dhs.append(dh)
        dh = dadd[:, :, i] + M[:, :, i].mT @ dh
    h, dh1 = torch.stack(hs, 2), torch.stack(dhs[::-1], 2)   # state before, its gradient after, each chunk
    kh, kdh = k @ h, k @ dh1
    u = T @ (v - col(ga) * kh)
    delta = col(beta) * u
    ddelta = P.mT @ do + col(E) * kdh
    dx = T.mT @ (col(beta) * ddelta)                         # gradient of v - exp(G) K h
    zu = (dx @ u.mT).tril(-1)
    dB = -zu * beta[..., None, :]
    dP = (do @ delta.mT).tril()
    X = (dB * kk + dP * P).tril(-1)
    dP, dB = dP * gam, dB * gam
    doh = do @ h.mT
    dq = col(ga) * doh + dP @ k
    dk_ = col(E * beta) * (u @ dh1.mT) - col(ga) * (dx @ h.mT) + dP.mT @ q + (dB + dB.mT) @ k
    dbeta = (ddelta * u).sum(-1) - (kk * zu).sum(-2)
    Y = E * (delta * kdh).sum(-1)
    dG = (ga * (doh * q).sum(-1) - ga * (dx * kh).sum(-1) - Y).double() + X.sum(-1).double() - X.sum(-2).double()
    dG[..., -1] += (Y.sum(-1) + ga[..., -1] * (h * dh1).sum((-1, -2))).double()
    dg = dG.flip(-1).cumsum(-1).flip(-1)
    dq, dk_ = dq.unflatten(1, (Hk, rep)).sum(2), dk_.unflatten(1, (Hk, rep)).sum(2)

    def give(x, like):
        x = x.movedim(1, 3).flatten(1, 2)[there]
        return x.reshape(like.shape).to(like.dtype)

    out = {"dq": give(dq, s["dq"]), "dk": give(dk_, s["dk"]), "dv": give(dx, s["dv"]),
           "dlog_g": give(dg, s["dlog_g"]), "dbeta": give(dbeta, s["dbeta"])}
    if s["dh0"] is not None:
        out["dh0"] = dh
    return out


def _plain(s):
    c, op, f32 = s["case"], s["op"], torch.float32
    if op == "backward":
        return _plain_backward(s)
    if op == "store8":
        codes, exps = _codes_of(s["x"])
        return {"codes": codes, "exps": exps}
    if op == "load8":
        return {"y": _values_of(s["codes"].view(torch.float8_e4m3fn), s["exps"]).to(s["y"].dtype)}
    d = c["d"]
    vals = {}
    for a in "xz":
        t = s[a]
        if t is not None and op == "norm_backward" and s[a + "_exps"] is not None:
            t = _values_of(t.reshape(-1, d), s[a + "_exps"]).view(t.shape)
        vals[a] = None if t is None else t.to(f32)
    x, z, w = vals["x"], vals["z"], s["w"]
    if c["center"]:
        x = x - x.sum(-1, keepdim=True) / d
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    n = x * r
    a = n * w if s["b"] is None else n * w + s["b"]
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
    if op == "norm_forward":
        out = {"y": (a if z is None else a * (z * sg)).to(s["y"].dtype)}
        for name in "xz":
            if s[name + "_codes"] is not None:
                out[name + "_codes"], out[name + "_exps"] = _codes_of(s[name].reshape(-1, d))
        return out
    dy, dt = s["dy"].to(f32), s["dx"].dtype
    out = {}
    g = dy
    if z is not None:
        g = dy * (z * sg)
        out["dz"] = (dy * a * (sg * (1 + z * (1 - sg)))).to(dt)
    dn = g * w
    dx = dn - n * ((dn * n).sum(-1, keepdim=True) / d)
    if c["center"]:
        dx = dx - dn.sum(-1, keepdim=True) / d
    out["dx"] = (dx * r).to(dt)
    out["dw"] = (g * n).sum((0, 1), dtype=torch.float64).to(f32)
    if s["b"] is not None:
        out["db"] = g.sum((0, 1), dtype=torch.float64).to(f32)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op, s = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "backward":
        B, T, Hk, Hv, dk, dv = (case[x] for x in ("B", "T", "Hk", "Hv", "dk", "dv"))
        lens = _lengths(case) if case["packed"] else [T] * B
        n, act = sum(lens), 1 if case["ckpt"] else s
        b = n * (2 * Hk * dk + Hv * dv) * (act + s) + n * Hv * dv * s + n * Hv * (8 + 2 * s)
        if case["ckpt"]:
            b += n * (2 * Hk * -(-dk // GROUP) + Hv * -(-dv // GROUP))
        if case["h0"]:
            b += 3 * 4 * B * Hv * dk * dv
        mac = 0.0
        for t in lens:
            for L in [CHUNK] * (t // CHUNK) + ([t % CHUNK] if t % CHUNK else []):
                tri = L * (L + 1) / 2
                # states: K h, K^T delta, K dh, Q^T do, K^T dx, do h^T, dx h^T, delta dh^T; rows of the
                # chunk against each other: u, delta's gradient, dx, dx u^T, do u^T over dv, four
                # products over dk, and the two Gram matrices, which the heads of a group share
                mac += 8 * L * dk * dv + tri * (5 * dv + 4 * dk + 2 * dk * Hk / Hv) + L ** 3 / 6
        return {"bytes": b, "flops": 2 * mac * Hv}
    if op in ("norm_forward", "norm_backward"):
        n = case["T"] * case["H"] * case["d"]
        groups = case["T"] * case["H"] * -(-case["d"] // GROUP)
        streams = 2 if case["gate"] else 1                    # x, and the gate
        if op == "norm_forward":
            b = n * s * (streams + 1) + (streams * (n + groups) if case["ckpt"] else 0)
            return {"bytes": b + case["d"] * 8, "flops": n * 12}
        act = n + groups if case["ckpt"] else n * s
        return {"bytes": streams * (act + n * s) + n * s + case["d"] * 16, "flops": n * 25}
    n, groups = case["rows"] * case["d"], case["rows"] * -(-case["d"] // GROUP)
    return {"bytes": n * (s + 1) + groups, "flops": n * 2}


# ---- values in 64 bits ------------------------------------------------------

def _two_to(e):
    """2^e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, exps, d):
    """e4m3 bytes read bit by bit: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    bits = codes.reshape(-1, d).view(torch.uint8).long()
    e, m = (bits >> 3) & 15, bits & 7
    f = torch.where(e == 0, m.double() * 2.0 ** -9, (8 + m).double() * _two_to(e - 10))
    f = torch.where((bits & 127) == 127, math.nan, f) * (1 - 2 * (bits >> 7)).double()
    which = torch.arange(d, device=codes.device) // GROUP
    return f * _two_to(exps.long() - 127)[:, which]


def _exact_codes(x):
    """Nearest e4m3 value, ties to even, of x over its group's scale, in 64 bits."""
    rows, d = x.shape
    pad = -d % GROUP
    v = torch.nn.functional.pad(x.double(), (0, pad)).view(rows, -1, GROUP)
    top = v.abs().amax(-1)
    # the exponents that log2 gives may be one off next to a power of two: put right by comparing
    e = torch.ceil(torch.log2(torch.where(top > 0, top / 448, 1.0))).clamp(-1000, 1000)
    e = torch.where(top > 448 * _two_to(e), e + 1, e)
    e = torch.where(top <= 448 * _two_to(e - 1), e - 1, e)
    e = torch.where(top > 0, e.clamp(-126, 119), 0.0)
    v = v * _two_to(-e)[..., None]
    place = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    place = torch.where(_two_to(place) > v.abs().clamp_min(2.0 ** -6), place - 1, place)
    place = torch.where(_two_to(place + 1) <= v.abs(), place + 1, place)
    step = _two_to(place - 3)
    v = torch.round(v / step) * step
    return v.view(rows, -1)[:, :d], (e + 127).to(torch.uint8)


def _exact_backward(s):
    """Token by token: S' = alpha S, r = v - S'^T k, S_t = S' + beta k r^T,
    o = S_t^T q, walked forwards with every state kept, then backwards."""
    c = s["case"]
    B, Hk, Hv, dk, dv = (c[x] for x in ("B", "Hk", "Hv", "dk", "dv"))
    dev, T, rep = s["dout"].device, s["longest"], Hv // Hk
    first = s["cu"].tolist()

    def rows(x, tail):
        flat = x.reshape((-1,) + tail).double()
        y = torch.zeros((T, B) + tail, dtype=torch.float64, device=dev)
        for b in range(B):
            y[: first[b + 1] - first[b], b] = flat[first[b]: first[b + 1]]
        return y

    def act(name, heads, d):
        x = s[name]
        if s[name + "_exps"] is not None:
            x = _exact_values(x, s[name + "_exps"], d)
        x = rows(x, (heads, d))
        return x.repeat_interleave(rep, 2) if heads != Hv else x

    q, k, v = act("q", Hk, dk), act("k", Hk, dk), act("v", Hv, dv)
    do, al, be = rows(s["dout"], (Hv, dv)), torch.exp(rows(s["log_g"], (Hv,))), rows(s["beta"], (Hv,))
    S = s["h0"].double() if s["h0"] is not None else torch.zeros(B, Hv, dk, dv, dtype=torch.float64, device=dev)
    kept = torch.empty((T,) + S.shape, dtype=torch.float64, device=dev)
    for t in range(T):
        kept[t] = S
        S = S * al[t][..., None, None]
        r = be[t][..., None] * (v[t] - (S * k[t][..., None]).sum(-2))
        S = S + k[t][..., None] * r[..., None, :]
    D = s["dht"].double() if s["dht"] is not None else torch.zeros_like(S)
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(al), torch.zeros_like(be)
    for t in reversed(range(T)):
        S1 = kept[t] * al[t][..., None, None]
        r = v[t] - (S1 * k[t][..., None]).sum(-2)
        S2 = S1 + k[t][..., None] * (be[t][..., None] * r)[..., None, :]
        dq[t] = (S2 * do[t][..., None, :]).sum(-1)
        D = D + q[t][..., None] * do[t][..., None, :]
        Dk = (D * k[t][..., None]).sum(-2)
        db[t] = (Dk * r).sum(-1)
        dv_[t] = be[t][..., None] * Dk
        dk_[t] = be[t][..., None] * (D * r[..., None, :]).sum(-1) - (S1 * dv_[t][..., None, :]).sum(-1)
        D = D - k[t][..., None] * dv_[t][..., None, :]
        dg[t] = (D * S1).sum((-1, -2))
        D = D * al[t][..., None, None]

    def back(x, like, group=False):
        if group:
            x = x.unflatten(2, (Hk, rep)).sum(3)
        return torch.cat([x[: first[b + 1] - first[b], b] for b in range(B)]).reshape(like.shape)

    out = {"dq": back(dq, s["dq"], True), "dk": back(dk_, s["dk"], True), "dv": back(dv_, s["dv"]),
           "dlog_g": back(dg, s["dlog_g"]), "dbeta": back(db, s["dbeta"])}
    if s["dh0"] is not None:
        out["dh0"] = D
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "backward":
        if s["longest"] * case["B"] * case["Hv"] * case["dk"] * case["dv"] * 8 > 80e9:
            return None
        return _exact_backward(s)
    if op == "store8":
        codes, exps = _exact_codes(s["x"])
        return {"codes": codes, "exps": exps}
    if op == "load8":
        return {"y": _exact_values(s["codes"], s["exps"], case["d"])}
    d = case["d"]
    leaves = {}
    for a in "xz":
        if s[a] is not None:
            coded = op == "norm_backward" and s[a + "_exps"] is not None
            t = _exact_values(s[a], s[a + "_exps"], d).view(s[a].shape) if coded else s[a].double()
            leaves[a] = t.detach().requires_grad_(op == "norm_backward")
    w = s["w"].double().requires_grad_(op == "norm_backward")
    b = None if s["b"] is None else s["b"].double().requires_grad_(op == "norm_backward")
    x = leaves["x"]
    mean = x.mean(-1, keepdim=True) if case["center"] else 0.0
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS) * w
    y = y if b is None else y + b
    if "z" in leaves:
        y = y * leaves["z"] * torch.sigmoid(leaves["z"])
    if op == "norm_forward":
        out = {"y": y}
        for a in leaves:
            if s[a + "_codes"] is not None:
                out[a + "_codes"], out[a + "_exps"] = _exact_codes(s[a].reshape(-1, d))
        return out
    named = {"dx": x, "dw": w}
    if "z" in leaves:
        named["dz"] = leaves["z"]
    if b is not None:
        named["db"] = b
    return dict(zip(named, torch.autograd.grad(y, list(named.values()), s["dy"].double())))
