"""GPU tests of the norm and its gradients against the definition in 64 bits.

Bounds.  fp32: every output is formed by about 2 log2(d) + 20 dependent fp32
operations, each off by at most 2^-24 (the hardware's exp2, reciprocal and
rsqrt by 2^-23), so 64 * 2^-24 = 4e-6 of the row's largest term; the bound is
1e-5 in the 2-norm over a tensor.  bf16: one rounding more, at most 2^-8 of
each value.  dx is a difference, r (dn - mean(dn) - n mean(dn n)), whose terms
are each at most r max|dn| (1 + |n|) and off by 64 * 2^-24 of that, however much
of them cancels (an RMS norm of one value keeps only eps / (x^2 + eps) of its
terms): it is held to 1e-5 of that term bound, entry by entry, and its rounding.
dw and db are fp32 sums over rows of values that are off by the
same 4e-6: 1e-5 in the 2-norm."""
import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
import train_ref
from gpu_common import dev, say
from train_ref import two_norm

pytestmark = pytest.mark.gpu


def make(T, H, d, dtype, gate, bias, seed=0, mean=0.0, xpad=0, zpad=0):
    g = torch.Generator().manual_seed(seed + 31 * d + T)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = dict(x=(r(T, H * d + xpad) * 0.7 + mean).to(dtype)[:, xpad:].unflatten(1, (H, d)),
             z=(r(T, H * d + zpad) * 2).to(dtype)[:, zpad:].unflatten(1, (H, d)) if gate else None,
             w=1 + 0.2 * r(d), b=0.3 * r(d) if bias else None, dy=r(T, H, d).to(dtype))
    return c


def on(t):
    if t is None:
        return None
    if t.is_contiguous():
        return t.to(dev())
    base = torch.empty(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype, device=dev())
    v = base.as_strided(t.shape, t.stride(), t.storage_offset())
    return v.copy_(t)


def close(got, ref, what, terms=None):
    if got.dtype == torch.bfloat16 or terms is not None:
        d = (got.cpu().double() - ref).abs()
        step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
        # a gate under fp32's smallest normal, 2^-126, may come as zero: with |z|, dy,
        # w and r next to it, 2^-126 * 2^10 * 2^6 at most in these tests
        assert bool((d <= step * ref.abs() + 1e-5 * (ref.abs().max() if terms is None else terms) + 2.0 ** -110).all()), what
    else:
        assert two_norm(got, ref) <= 1e-5, (what, two_norm(got, ref))


def check(c, center, eps=1e-6, ckpt=False):
    x, z, w, b, dy = on(c["x"]), on(c["z"]), on(c["w"]), on(c["b"]), on(c["dy"])
    y, kept = gdn.norm_forward(x, w, z=z, b=b, eps=eps, center=center, ckpt=ckpt)
    f = lambda t: None if t is None else t.double()  # noqa: E731
    close(y, train_ref.norm(f(c["x"]), f(c["w"]), f(c["z"]), f(c["b"]), eps, center), "y")
    rx, rz = c["x"], c["z"]
    if ckpt:
        for n in kept:
            if n.endswith("codes"):
                a = c[n[0]]
                cc, ee = gdn.ckpt8_store(a.contiguous().to(dev()))
                assert torch.equal(kept[n].view(torch.uint8), cc.view(torch.uint8)) and torch.equal(kept[n[0] + "_exps"], ee)
        rx = gdn.ckpt8_load(kept["x_codes"], kept["x_exps"], torch.float32).cpu()
        if z is not None:
            rz = gdn.ckpt8_load(kept["z_codes"], kept["z_exps"], torch.float32).cpu()
        g = gdn.norm_backward(dy, kept["x_codes"], w, z=kept.get("z_codes"), b=b, x_exps=kept["x_exps"],
                              z_exps=kept.get("z_exps"), eps=eps, center=center)
    else:
        g = gdn.norm_backward(dy, x, w, z=z, b=b, eps=eps, center=center)
    ref = train_ref.norm_grads(c["dy"], rx, c["w"], rz, c["b"], eps, center)
    assert set(g) == set(ref)
    rx, wd = rx.double(), c["w"].double()
    rx = rx - rx.mean(-1, keepdim=True) if center else rx
    r = 1 / torch.sqrt((rx ** 2).mean(-1, keepdim=True) + eps)
    dn = c["dy"].double() * wd * (1.0 if z is None else rz.double() * torch.sigmoid(rz.double()))
    terms = r * dn.abs().amax(-1, keepdim=True) * (1 + (rx * r).abs())
    if z is not None:
        # the gate's exp2 takes z log2(e), off by 2^-24 of itself and by the
        # constant's 2^-25: 1.5 |z| 2^-24 of the gate, in each of dx's two sums
        terms = terms * (1 + 3 * rz.double().abs().amax(-1, keepdim=True) * 2.0 ** -24 / 1e-5)
    for n in g:
        close(g[n], ref[n], n, terms if n == "dx" else None)


@pytest.mark.parametrize("d", [1, 7, 8, 32, 33, 64, 80, 100, 128, 192, 256, 264, 500, 512, 520, 1000, 1024, 1030,
                               1032, 2048, 2050, 4096, 4099, 5120, 6152, 8191, 8192])
def test_widths(d):
    say("norm d", d)
    T = 37 if d < 600 else 5
    check(make(T, 1, d, torch.float32, gate=True, bias=True), center=True)
    check(make(T, 1, d, torch.bfloat16, gate=d % 2 == 0, bias=False), center=False, ckpt=d % 3 != 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("center,gate,bias,ckpt", [(False, True, False, False), (True, False, True, False),
                                                   (False, True, True, True), (True, True, False, True),
                                                   (False, False, False, False), (True, False, False, True)])
def test_heads(dtype, center, gate, bias, ckpt):
    say("norm heads", dtype, center, gate, bias, ckpt)
    for T, H, d in ((1, 1, 128), (3, 48, 128), (700, 6, 128), (33, 3, 100), (1100, 5, 64)):
        check(make(T, H, d, dtype, gate, bias), center, ckpt=ckpt)


@pytest.mark.parametrize("xpad,zpad", [(8, 640), (0, 77), (3, 0), (128, 8)])
def test_strided_views(xpad, zpad):
    say("norm strides", xpad, zpad)
    for dtype in (torch.bfloat16, torch.float32):
        check(make(40, 6, 128, dtype, gate=True, bias=False, xpad=xpad, zpad=zpad), center=False)
        check(make(40, 2, 72, dtype, gate=True, bias=True, xpad=xpad, zpad=zpad), center=True, ckpt=zpad == 0 and xpad == 0)


def test_large_mean_keeps_its_digits():
    say("norm large mean")
    # x is 1000 + noise in fp32: the noise itself is known to 2^-24 * 1000 / 0.7,
    # and the two-step statistics lose nothing more
    check(make(64, 2, 128, torch.float32, gate=False, bias=True, mean=1000.0), center=True)


def test_constant_and_zero_rows():
    say("norm constant rows")
    c = make(4, 2, 128, torch.float32, gate=True, bias=True)
    c["x"][0] = 0.0
    c["x"][1] = 3.0
    check(c, center=True, eps=1e-5)
    check(c, center=False, eps=1e-5)


def test_extreme_gates():
    say("norm extreme gates")
    c = make(6, 2, 128, torch.float32, gate=True, bias=False)
    c["z"][0], c["z"][1], c["z"][2] = 80.0, -80.0, 0.0
    c["z"][3], c["z"][4] = 300.0, -300.0
    check(c, center=False)


def test_a_bad_row_stays_alone():
    say("norm NaN row")
    c = make(40, 2, 128, torch.float32, gate=True, bias=False)
    good = gdn.norm_backward(on(c["dy"]), on(c["x"]), on(c["w"]), z=on(c["z"]))
    c["x"][7, 1, 3] = float("nan")
    c["x"][9, 0, 5] = float("inf")
    g = gdn.norm_backward(on(c["dy"]), on(c["x"]), on(c["w"]), z=on(c["z"]))
    keep = torch.ones(40, 2, dtype=torch.bool)
    keep[7, 1] = keep[9, 0] = False
    for n in ("dx", "dz"):
        assert torch.equal(g[n].cpu()[keep], good[n].cpu()[keep])
    assert bool(torch.isnan(g["dx"].cpu()[7, 1]).all())


def test_no_rows_writes_zero_sums():
    say("norm T = 0")
    x = torch.empty((0, 3, 128), device=dev())
    w, b = torch.ones(128, device=dev()), torch.ones(128, device=dev())
    y, _ = gdn.norm_forward(x, w, b=b)
    assert y.shape == x.shape
    g = gdn.norm_backward(x, x, w, b=b)
    assert bool((g["dw"] == 0).all()) and bool((g["db"] == 0).all())


def test_same_bits_each_run_and_other_stream():
    say("norm runs and streams")
    c = make(3000, 4, 128, torch.bfloat16, gate=True, bias=True)
    t = {n: on(v) for n, v in c.items()}
    a = gdn.norm_backward(t["dy"], t["x"], t["w"], z=t["z"], b=t["b"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        e = gdn.norm_backward(t["dy"], t["x"], t["w"], z=t["z"], b=t["b"])
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], e[n]), n


def test_gradient_against_differences():
    say("norm differences")
    c = make(5, 2, 24, torch.float32, gate=True, bias=True)
    g = gdn.norm_backward(on(c["dy"]), on(c["x"]), on(c["w"]), z=on(c["z"]), b=on(c["b"]), center=True)
    gen = torch.Generator().manual_seed(1)
    f = {n: c[n].double() for n in ("x", "w", "z", "b")}
    for n in f:
        step = torch.randn(f[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        loss = [float((train_ref.norm(**{**f, n: f[n] + s * h * step}, center=True) * c["dy"].double()).sum()) for s in (1, -1)]
        want = (loss[0] - loss[1]) / (2 * h)
        got = float((g["d" + n].cpu().double() * step).sum())
        # differences are off by h^2 times a third derivative of order 1 per value
        assert abs(got - want) <= 1e-4 * max(1.0, abs(want)), n


def test_heads_of_one_token_past_32_bits():
    # one token of 2^18 + 3 heads of 8192: a head's offset passes 2^31 values.  The
    # same rows as tokens of one head are the same bits
    say("norm, one token's heads past 2^31 values")
    H, d = (1 << 18) + 3, 8192
    gen = torch.Generator(dev()).manual_seed(5)
    x, dy = (torch.randn(1, H, d, generator=gen, device=dev(), dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand(d, generator=gen, device=dev()) + 0.5
    one, _ = gdn.norm_forward(x, w, z=dy)
    rows, _ = gdn.norm_forward(x.view(H, 1, d), w, z=dy.view(H, 1, d))
    assert torch.equal(one.view(H, 1, d), rows)
    close(rows[-3:], train_ref.norm(x[0, -3:, None].cpu().double(), w.cpu().double(), dy[0, -3:, None].cpu().double()), "y")
    del one, rows
    one = gdn.norm_backward(dy, x, w, z=x)
    rows = gdn.norm_backward(dy.view(H, 1, d), x.view(H, 1, d), w, z=x.view(H, 1, d))
    for n in one:
        assert torch.equal(one[n].flatten(), rows[n].flatten()), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("center,bad", [(False, "nan"), (True, "nan"), (True, "inf")])
@pytest.mark.parametrize("d", [128, 100, 2048, 4099])
def test_a_bad_row_is_nan(dtype, center, bad, d):
    # the statistics of a row that holds a NaN are NaN, and so is all that they
    # enter: the row's y, dx and dz, and dw; of a centred row, whose mean is then
    # infinite or NaN, with an infinity too
    say("norm bad row", dtype, center, bad, d)
    c = make(9, 2, d, dtype, gate=True, bias=False, seed=3)
    c["x"][4, 1, 7] = float(bad)
    x, z, w, dy = on(c["x"]), on(c["z"]), on(c["w"]), on(c["dy"])
    y, kept = gdn.norm_forward(x, w, z=z, center=center, ckpt=True)
    g = gdn.norm_backward(dy, x, w, z=z, center=center)
    h = gdn.norm_backward(dy, kept["x_codes"], w, z=kept["z_codes"], x_exps=kept["x_exps"], z_exps=kept["z_exps"], center=center)
    rows = torch.zeros(9, 2, dtype=torch.bool)
    rows[4, 1] = True
    for t in (y, g["dx"], g["dz"], h["dx"], h["dz"]):
        assert bool(torch.isnan(t.cpu()[rows]).all()) and not bool(torch.isnan(t.cpu()[~rows]).any())
    assert bool(torch.isnan(g["dw"]).all()) and bool(torch.isnan(h["dw"]).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gates_of_any_size(dtype):
    # silu'(z) = s + z s (1 - s) goes to 1 for a large z.  s and 1 - s are off by 2^-22
    # at the most and 1 - s is exactly zero from z = 18 on, so that z s (1 - s) is off
    # by 18 * 2^-22 = 4e-6, beside values of s of 1
    say("norm large gates", dtype)
    c = make(8, 2, 128, dtype, gate=True, bias=True, seed=9)
    for i, v in enumerate([5.0, 12.0, 17.0, 50.0, 1e3, 1e5, 1e8, 1e30]):
        c["z"][i] = (torch.ones(2, 128) * v).to(dtype)
    g = gdn.norm_backward(on(c["dy"]), on(c["x"]), on(c["w"]), z=on(c["z"]), b=on(c["b"]))
    ref = train_ref.norm_grads(c["dy"], c["x"], c["w"], c["z"], c["b"])["dz"]
    d = (g["dz"].cpu().double() - ref).abs()
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert bool((d <= (step + 1e-5) * ref.abs() + 1e-5 * ref.abs().amax(-1, keepdim=True)).all())
