"""GPU tests of the 8-bit checkpoints: codes and scale bytes equal, bit for bit,
a search over e4m3's values in 64 bits; reading back is exact."""
import numpy as np
import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
import train_ref
from gpu_common import dev, say

pytestmark = pytest.mark.gpu


def rows(n, d, seed, dtype):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)) * np.exp2(rng.integers(-30, 30, (n, 1)).astype(float))
    return torch.from_numpy(x).to(torch.float32).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (3, 16, 0), (7, 48, 0), (5, 100, 0), (9, 128, 0), (4, 128, 16),
                                     (3, 129, 0), (2, 333, 5), (3, 512, 0), (2, 520, 8), (1, 1000, 0), (2, 1024, 1)])
def test_store_bits(dtype, n, d, pad):
    x = rows(n, d + pad, 7 * n + d, dtype)
    say("ckpt8 store", dtype, n, d, pad)
    ng = -(-d // 128)
    codes = torch.full((n, d), 0xAA, dtype=torch.uint8, device=dev())
    exps = torch.full((n, ng), 0xAA, dtype=torch.uint8, device=dev())
    gdn.gdn_ckpt8_store(x.to(dev()), codes, exps, n, d, d + pad)
    c, e = train_ref.ckpt8(x[:, :d].double().numpy())
    assert np.array_equal(exps.cpu().numpy(), e)
    assert np.array_equal(codes.cpu().numpy(), c)


def test_store_special_values():
    inf, nan = float("inf"), float("nan")
    lines = [
        [0.0, -0.0] * 8,
        [inf, -inf, nan, 1.0] * 4,                    # the scale comes from the finite ones
        [inf, nan] * 8,                               # no finite value: as all zero
        [448.0, 449.0, 464.0, 465.0] * 4,
        [1.75 * 2.0 ** 20, 2.0 ** 20, 1.0, 2.0 ** -3] * 4,     # 1.75 2^x is the last of its scale
        [float(np.nextafter(np.float32(1.75), np.float32(2))), 1.0, 0.5, 2.0 ** -9] * 4,
        [2.0 ** -126, 2.0 ** -130, 1e-45, 0.0] * 4,   # the smallest scale
        [3.4028234663852886e38, 1e38, 2.0 ** 120, 1.0] * 4,    # the largest
        [2.0 ** -6, 1.5 * 2.0 ** -9, 0.5 * 2.0 ** -9, 448.0] * 4,   # subnormal codes and their ties
    ]
    x = torch.tensor(lines, dtype=torch.float32)
    say("ckpt8 special values")
    codes, exps = gdn.ckpt8_store(x.to(dev()))
    c, e = train_ref.ckpt8(x.double().numpy())
    assert np.array_equal(exps.cpu().numpy(), e)
    got = codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(np.where(got & 127 == 127, 127, got), np.where(c & 127 == 127, 127, c))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,pad", [(256, 0), (250, 0), (250, 6), (256, 32)])
def test_load_every_code(dtype, d, pad):
    codes = torch.arange(256, dtype=torch.uint8).repeat(6, 1)[:, :d].contiguous()
    exps = torch.tensor([[1, 120], [127, 128], [246, 7], [127, 127], [60, 200], [100, 2]], dtype=torch.uint8)
    say("ckpt8 load", dtype, d, pad)
    y = torch.full((6, d + pad), 7.0, dtype=dtype, device=dev())
    gdn.gdn_ckpt8_load(codes.to(dev()), exps.to(dev()), y, 6, d, d + pad)
    vals = train_ref.e4m3_values()[codes.numpy()] * np.exp2(exps.numpy().astype(float) - 127)[:, np.arange(d) // 128]
    ref = torch.from_numpy(vals).to(torch.float32).to(dtype)       # exact, down to the type's smallest
    got = y[:, :d].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[~torch.isnan(ref)], ref[~torch.isnan(ref)])
    assert pad == 0 or bool((y[:, d:] == 7.0).all())               # nothing behind the rows


def test_round_trip_error_and_no_rows():
    x = rows(500, 128, 3, torch.bfloat16)
    say("ckpt8 round trip")
    codes, exps = gdn.ckpt8_store(x.to(dev()))
    y = gdn.ckpt8_load(codes, exps, torch.float32).cpu().double()
    # half a step: 2^-4 of the value, and 2^-10 of the scale below 2^-6 of it
    scale = torch.exp2(exps.cpu().double() - 127)
    assert bool(((y - x.double()).abs() <= torch.maximum(x.double().abs() * 2.0 ** -4, scale * 2.0 ** -10)).all())
    c, e = gdn.ckpt8_store(torch.empty((0, 128), device=dev()))
    assert c.shape == (0, 128) and e.shape == (0, 1)
    assert gdn.ckpt8_load(c, e).shape == (0, 128)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,pad", [(128, 0), (256, 0), (100, 0), (130, 1)])
def test_the_largest_finite_values_come_back_finite(dtype, d, pad):
    # the last binade: byte 247, codes up to 256
    say("ckpt8 largest values", dtype, d, pad)
    x = torch.linspace(1.0, 2.0 - 2.0 ** -7, 5 * d).reshape(5, d).mul(2.0 ** 127).to(dtype)
    x[:, 1::2] /= 200.0
    x[:, 0] = torch.finfo(dtype).max
    x[:, d - 1] = -torch.finfo(dtype).max
    x[2, 3], x[2, 4] = float("nan"), float("inf")
    codes, exps = gdn.ckpt8_store(x.to(dev()))
    assert bool((exps == 247).all())
    y = torch.full((5, d + pad), 7.0, dtype=torch.float32, device=dev())
    gdn.gdn_ckpt8_load(codes, exps, y, 5, d, d + pad)
    got, ref = y[:, :d].cpu().double(), x.double()
    ok = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), ok) and bool(torch.isnan(got[~ok]).all())
    # half a step, and the roundings of the reciprocal and of the product with it
    assert bool(((got - ref).abs()[ok] <= (2.0 ** -4 + 2.0 ** -22) * ref.abs()[ok]).all())
    vals = train_ref.e4m3_values()[codes.view(torch.uint8).cpu().numpy()] * 255.0 * 2.0 ** 112
    assert np.array_equal(vals[ok.numpy()], got.numpy()[ok.numpy()])
    half = gdn.ckpt8_load(codes, exps, torch.bfloat16).cpu()
    assert torch.equal(half.double().nan_to_num(), got.to(torch.float32).to(torch.bfloat16).double().nan_to_num())


@pytest.mark.parametrize("d", [128, 100])
def test_the_backward_passes_read_the_largest_values_alike(d):
    # the gradients from codes of byte 247 are those of the values that
    # gdn_ckpt8_load gives, to the bit
    say("ckpt8 largest values, read by the backward passes", d)
    gen = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    big = lambda t: t.sign() * (1.9 + 0.09 * torch.rand(t.shape, generator=gen)) * 2.0 ** 127  # noqa: E731
    on = lambda t: t.to(dev())  # noqa: E731
    x, z, dy, w = r(6, 2, d), big(r(6, 2, d)).abs(), r(6, 2, d) * 2.0 ** -100, r(d)
    xc, xe = gdn.ckpt8_store(on(x))
    zc, ze = gdn.ckpt8_store(on(z))
    assert int(ze.min()) == 247
    a = gdn.norm_backward(on(dy), xc, on(w), z=zc, x_exps=xe, z_exps=ze)
    b = gdn.norm_backward(on(dy), gdn.ckpt8_load(xc, xe, torch.float32), on(w), z=gdn.ckpt8_load(zc, ze, torch.float32))
    for n in a:
        assert bool(torch.isfinite(a[n]).all()) and torch.equal(a[n], b[n]), n
    q, k, v = r(1, 70, 1, d) / d ** 0.5, r(1, 70, 1, d) / d ** 0.5, r(1, 70, 2, d)
    v[0, 30] = big(v[0, 30])
    gate, beta = on(torch.full((1, 70, 2), -0.1)), torch.full((1, 70, 2), 0.5)
    beta[0, 30] = 2.0 ** -120
    dt = torch.bfloat16 if d == 128 else torch.float32
    dout = on((r(1, 70, 2, d) * 2.0 ** -20).to(dt))
    kept = [gdn.ckpt8_store(on(t)) for t in (q, k, v)]
    vals = [gdn.ckpt8_load(*t, dt) for t in kept]
    assert int(kept[2][1].max()) == 247 and all(bool(torch.isfinite(t).all()) for t in vals)
    a, route = gdn.chunk_backward(*(t[0] for t in kept), gate, on(beta), dout, q_exps=kept[0][1], k_exps=kept[1][1],
                                  v_exps=kept[2][1])
    assert route.startswith("gdn_bwd_prep" if d == 128 else "gdn_backward_prep"), route
    b, _ = gdn.chunk_backward(*vals, gate, on(beta), dout)
    for n in a:
        assert bool(torch.isfinite(a[n].float()).all()), n
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("off", [0, 1])
def test_one_long_row(off):
    # the widest row: its groups are those of the same values in rows of 128, with
    # wide loads (off = 0) and value by value
    say("ckpt8 long row", off)
    n = 1 << 30
    x = torch.empty(n + 1, dtype=torch.bfloat16, device=dev())[off:off + n].normal_(generator=torch.Generator(dev()).manual_seed(6))
    codes, exps = gdn.ckpt8_store(x)
    c, e = gdn.ckpt8_store(x.clone().view(-1, 128))
    assert torch.equal(codes.view(torch.uint8), c.view(torch.uint8).flatten()) and torch.equal(exps.flatten(), e.flatten())
    assert torch.equal(gdn.ckpt8_load(codes, exps), gdn.ckpt8_load(c, e).flatten())
