"""Host-side checks of the training entry points, no GPU needed: the library
exports what include/gdn_train.h declares, the plans refuse each bad argument
with its own status, the routes are named, and the binding refuses tensors that
the kernels cannot take.  Pointers are dummies: plans only compare them with
NULL and look at their alignment."""
import os
import re

import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
from linear_attention_ssm_gated_amd import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_train.h")
X = 0x1000
BIG = 1 << 42
S = {v: k for k, v in gdn._STATUS.items()}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn.so is not built (run __graft_entry__.build())")
    return train._lib()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdn_\w+)\s*\(", text))
    assert names == set(gdn.TRAIN_SIGNATURES)
    for n in names:
        assert hasattr(lib, n)
    # what was there before keeps its own table
    assert not names & set(gdn.SIGNATURES)


# ---- 8-bit checkpoints

def store(lib, **kw):
    a = dict(x=X, codes=X, exps=X, rows=10, d=128, stride=128, dt=1)
    a.update(kw)
    return lib.gdn_ckpt8_store_plan(a["x"], a["codes"], a["exps"], a["rows"], a["d"], a["stride"], a["dt"])


def load(lib, **kw):
    a = dict(codes=X, exps=X, y=X, rows=10, d=128, stride=128, dt=1)
    a.update(kw)
    return lib.gdn_ckpt8_load_plan(a["codes"], a["exps"], a["y"], a["rows"], a["d"], a["stride"], a["dt"])


@pytest.mark.parametrize("kw,status", [
    (dict(), "GDN_OK"), (dict(rows=0), "GDN_OK"), (dict(rows=1 << 33), "GDN_OK"),
    (dict(dt=2), "GDN_ERR_DTYPE"), (dict(rows=-1), "GDN_ERR_SHAPE"), (dict(d=0), "GDN_ERR_SHAPE"),
    (dict(stride=127), "GDN_ERR_STRIDE"), (dict(codes=None), "GDN_ERR_NULL"), (dict(exps=None), "GDN_ERR_NULL"),
])
def test_ckpt8_refusals(lib, kw, status):
    assert store(lib, **kw) == S[status], gdn.last_route()
    assert load(lib, **kw) == S[status], gdn.last_route()


def test_ckpt8_routes(lib):
    store(lib)
    assert gdn.last_route().startswith("gdn_ckpt8_store_kernel ")
    for kw in (dict(d=100, stride=100), dict(x=X + 2), dict(stride=129), dict(codes=X + 8)):
        assert store(lib, **kw) == 0
        assert gdn.last_route().startswith("gdn_ckpt8_store_any_kernel ")
    load(lib)
    assert gdn.last_route().startswith("gdn_ckpt8_load_kernel ")
    load(lib, y=X + 4)
    assert gdn.last_route().startswith("gdn_ckpt8_load_any_kernel ")


# ---- norm

def fwd(lib, **kw):
    a = dict(x=X, z=X, w=X, b=None, y=X, xc=None, xe=None, zc=None, ze=None, T=5, H=4, d=128, xs=512, zs=512,
             ys=512, eps=1e-6, center=0, dt=1)
    a.update(kw)
    return lib.gdn_norm_forward_plan(*a.values())


def bwd(lib, **kw):
    a = dict(x=X, xe=None, z=X, ze=None, w=X, b=None, dy=X, dx=X, dz=X, dw=X, db=None, T=5, H=4, d=128, xs=512,
             zs=512, dys=512, dxs=512, dzs=512, eps=1e-6, center=0, act=1, io=1, ws=X, wsb=BIG)
    a.update(kw)
    return lib.gdn_norm_backward_plan(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(), "GDN_OK"), (dict(T=0, x=None, y=None), "GDN_OK"), (dict(z=None, zs=0), "GDN_OK"),
    (dict(dt=2), "GDN_ERR_DTYPE"), (dict(T=-1), "GDN_ERR_SHAPE"), (dict(H=0), "GDN_ERR_SHAPE"),
    (dict(d=0), "GDN_ERR_SHAPE"), (dict(T=1 << 30, H=2), "GDN_ERR_SHAPE"), (dict(d=8193, xs=1 << 20, zs=1 << 20, ys=1 << 20), "GDN_ERR_DIM_LIMIT"),
    (dict(eps=-1.0), "GDN_ERR_SHAPE"), (dict(eps=float("inf")), "GDN_ERR_SHAPE"), (dict(eps=float("nan")), "GDN_ERR_SHAPE"),
    (dict(xs=511), "GDN_ERR_STRIDE"), (dict(zs=511), "GDN_ERR_STRIDE"), (dict(ys=511), "GDN_ERR_STRIDE"),
    (dict(w=None), "GDN_ERR_NULL"), (dict(x=None), "GDN_ERR_NULL"), (dict(xc=X), "GDN_ERR_NULL"),
    (dict(ze=X), "GDN_ERR_NULL"), (dict(z=None, zc=X, ze=X), "GDN_ERR_NULL"),
])
def test_norm_forward_refusals(lib, kw, status):
    assert fwd(lib, **kw) == S[status], gdn.last_route()


@pytest.mark.parametrize("kw,status", [
    (dict(), "GDN_OK"), (dict(T=0, x=None, dy=None, dx=None, ws=None, wsb=0), "GDN_OK"),
    (dict(act=2, xe=X, ze=X), "GDN_OK"), (dict(act=2, xe=X, ze=X, io=0), "GDN_OK"),
    (dict(act=0), "GDN_ERR_DTYPE"), (dict(io=2), "GDN_ERR_DTYPE"), (dict(act=3), "GDN_ERR_DTYPE"),
    (dict(act=2, xe=X), "GDN_ERR_NULL"), (dict(act=2, ze=X), "GDN_ERR_NULL"),
    (dict(act=2, xe=X, ze=X, xs=520), "GDN_ERR_STRIDE"), (dict(dzs=511), "GDN_ERR_STRIDE"),
    (dict(dxs=511), "GDN_ERR_STRIDE"), (dict(dys=511), "GDN_ERR_STRIDE"),
    (dict(dw=None), "GDN_ERR_NULL"), (dict(b=X), "GDN_ERR_NULL"), (dict(db=X), "GDN_ERR_NULL"),
    (dict(dz=None), "GDN_ERR_NULL"), (dict(z=None), "GDN_ERR_NULL"), (dict(dx=None), "GDN_ERR_NULL"),
    (dict(ws=None), "GDN_ERR_WORKSPACE"), (dict(wsb=16), "GDN_ERR_WORKSPACE"), (dict(ws=X + 4), "GDN_ERR_WORKSPACE"),
])
def test_norm_backward_refusals(lib, kw, status):
    assert bwd(lib, **kw) == S[status], gdn.last_route()


def test_norm_routes(lib):
    fwd(lib)
    assert gdn.last_route().startswith("gdn_norm_forward_kernel<8> grid=[2,1,1]")
    for kw in (dict(x=X + 2), dict(zs=513), dict(d=100, xs=400, zs=400, ys=400)):
        assert fwd(lib, **kw) == 0
        assert gdn.last_route().startswith("gdn_norm_forward_kernel<1>")
    bwd(lib)
    assert gdn.last_route().startswith("gdn_norm_backward_kernel<8>+gdn_norm_weight_kernel")
    assert gdn.gdn_norm_workspace_bytes(0, 4, 128) == 0
    assert gdn.gdn_norm_workspace_bytes(5, 4, 128) == 2 * 2 * 128 * 4


# ---- chunk backward

def chunk(lib, **kw):
    a = dict(q=X, k=X, v=X, qe=None, ke=None, ve=None, lg=X, be=X, h0=None, do=X, dht=None, dq=X, dk=X, dv=X,
             dg=X, db=X, dh0=None, B=1, T=128, Hk=2, Hv=6, dk_=128, dv_=128, cu=None, io=1, grad=1, ws=X, wsb=BIG)
    a.update(kw)
    return lib.gdn_chunk_backward_plan(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(), "GDN_OK"), (dict(T=0, q=None, dq=None), "GDN_OK"), (dict(io=0, grad=0, dk_=1, dv_=3), "GDN_OK"),
    (dict(io=2, qe=X, ke=X, ve=X), "GDN_OK"),
    (dict(io=3), "GDN_ERR_DTYPE"), (dict(grad=2), "GDN_ERR_DTYPE"), (dict(io=-1), "GDN_ERR_DTYPE"),
    (dict(B=0), "GDN_ERR_SHAPE"), (dict(T=-1), "GDN_ERR_SHAPE"), (dict(dk_=0), "GDN_ERR_SHAPE"),
    (dict(B=65536), "GDN_ERR_SHAPE"), (dict(Hv=65540, Hk=2), "GDN_ERR_SHAPE"),
    (dict(Hv=5), "GDN_ERR_HEAD_GROUPS"), (dict(dk_=129), "GDN_ERR_DIM_LIMIT"), (dict(dv_=200), "GDN_ERR_DIM_LIMIT"),
    (dict(q=None), "GDN_ERR_NULL"), (dict(lg=None), "GDN_ERR_NULL"), (dict(do=None), "GDN_ERR_NULL"),
    (dict(dq=None), "GDN_ERR_NULL"), (dict(db=None), "GDN_ERR_NULL"), (dict(io=2, qe=X, ke=X), "GDN_ERR_NULL"),
    (dict(ws=None), "GDN_ERR_WORKSPACE"), (dict(wsb=1000), "GDN_ERR_WORKSPACE"), (dict(ws=X + 8), "GDN_ERR_WORKSPACE"),
])
def test_chunk_backward_refusals(lib, kw, status):
    assert chunk(lib, **kw) == S[status], gdn.last_route()


def test_chunk_backward_routes(lib):
    assert chunk(lib) == 0
    r = gdn.last_route()
    assert r.startswith("gdn_bwd_prep_kernel+gdn_bwd_spine_kernel+gdn_bwd_grads_kernel grid=[12,1,2]"), r
    for kw, why in ((dict(io=0, grad=0), "bf16 or 8-bit"), (dict(grad=0), "bf16 gradients"),
                    (dict(dv_=64), "dk = dv = 128"), (dict(q=X + 2), "aligned"), (dict(dq=X + 8), "aligned")):
        assert chunk(lib, **kw) == 0
        r = gdn.last_route()
        assert r.startswith("gdn_backward_prep_kernel") and why in r, r


def test_chunk_backward_workspace(lib):
    w = gdn.gdn_backward_workspace_bytes
    assert w(1, 128, 2, 5, 128, 128, 1, 1) == 0          # refused sizes need nothing
    assert w(1, 0, 2, 6, 128, 128, 1, 1) == 0
    one = w(1, 64, 2, 6, 128, 128, 1, 1)
    assert 0 < one and w(1, 128, 2, 6, 128, 128, 1, 1) >= 2 * one - 4096
    # a packed call of B sequences may have B chunks more than T / 64
    assert w(3, 64, 2, 6, 128, 128, 1, 1, packed=True) >= 4 * one - 4096
    assert chunk(lib, wsb=w(1, 128, 2, 6, 128, 128, 1, 1) - 1) == S["GDN_ERR_WORKSPACE"]


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="GPU"):
        gdn.ckpt8_store(x)
    with pytest.raises(ValueError, match="GPU"):
        gdn.norm_forward(x.view(4, 1, 128), torch.ones(128))
    with pytest.raises(ValueError, match="contiguous"):
        gdn.ckpt8_store(x.t())
    q = torch.zeros(1, 4, 1, 8)
    with pytest.raises(ValueError, match="GPU"):
        gdn.chunk_backward(q, q, q, torch.zeros(1, 4, 1), torch.zeros(1, 4, 1), q)
    with pytest.raises(TypeError, match="one dtype"):
        gdn.gdn_chunk_backward(q, q.bfloat16(), q, None, None, None, None, None, None, q, None, q, q, q, q, q, None,
                               1, 4, 1, 1, 8, 8)
    with pytest.raises(TypeError):
        gdn.chunk_backward(q.half(), q.half(), q.half(), q[..., 0], q[..., 0], q.half())


def test_conveniences_refuse_shapes_they_would_read_beyond():
    q, v, g = torch.zeros(1, 5, 2, 8), torch.zeros(1, 5, 4, 8), torch.zeros(1, 5, 4)
    good = dict(q=q, k=q, v=v, log_g=g, beta=g, dout=v)
    bad = dict(k=q[:, :4], v=v[:, :4], log_g=g[:, :4], beta=g[..., :2], dout=v[..., :4], h0=torch.zeros(1, 2, 8, 8),
               dh_final=torch.zeros(1, 4, 8, 4), q_exps=torch.zeros(5, 1, dtype=torch.uint8),
               v_exps=torch.zeros(20, 2, dtype=torch.uint8))
    for name, t in bad.items():
        with pytest.raises(ValueError, match="must have shape"):
            gdn.chunk_backward(**{**good, name: t})
    x, w = torch.zeros(3, 2, 8), torch.zeros(8)
    for kw in (dict(w=w[:4]), dict(w=w, z=x[:2]), dict(w=w, b=w[:1])):
        with pytest.raises(ValueError, match="must have shape"):
            gdn.norm_forward(x, **kw)
    for kw in (dict(w=w[:4]), dict(w=w, z=x[:2]), dict(w=w, x_exps=torch.zeros(6, 2, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="must have shape"):
            gdn.norm_backward(x, x, **kw)
    with pytest.raises(ValueError, match="must have shape"):
        gdn.norm_backward(x[:2], x, w)
    with pytest.raises(ValueError, match="must have shape"):
        gdn.ckpt8_load(torch.zeros(4, 130, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))


def test_a_stream_for_cpu_tensors_is_refused():
    x, w = torch.zeros(4, 1, 128), torch.ones(128)
    for call in (lambda: gdn.ckpt8_store(x, stream=16), lambda: gdn.norm_forward(x, w, stream=16),
                 lambda: gdn.norm_backward(x, x, w, stream=16)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_rows_of_more_than_2_30_values_are_refused(lib):
    # (a group's and a column's number are formed in 32 bits)
    for d in ((1 << 30) + 1, (1 << 31) - 64, (1 << 31) - 1):
        assert store(lib, rows=1, d=d, stride=1 << 33) == S["GDN_ERR_DIM_LIMIT"], gdn.last_route()
        assert load(lib, rows=1, d=d, stride=1 << 33) == S["GDN_ERR_DIM_LIMIT"], gdn.last_route()
    assert store(lib, rows=1, d=1 << 30, stride=1 << 30) == 0
    # an int of the C call would wrap: 2^32 + 128 values of one row would be 128
    x = torch.empty((1 << 32) + 128, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="2\\^30"):
        gdn.ckpt8_store(x)
    with pytest.raises(ValueError, match="2\\^30"):
        gdn.ckpt8_load(x.to(torch.uint8), torch.empty((1, 1), dtype=torch.uint8, device="meta"))
