"""GPU tests of the update's digits with 8-bit states: fp32 weights and fp32 masters
are not rounded to fewer bits, so the quotient m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
has to be a division's."""
import math

import numpy as np
import pytest
import torch

import adamw_ref
import linear_attention_ssm_gated_amd as gdn
from gpu_common import dev, say

pytestmark = pytest.mark.gpu

F64, BF = torch.float64, torch.bfloat16
B2, EPS = 0.99, 1e-8


def divided(weights, g, m, v, t, eps=EPS):
    """-u after one step of weights that are zero, with beta1 0 and a rate of 1: m and the divisor
    in fp32 as the step forms them, one operation at a time."""
    n = g.numel()
    codes = [adamw_ref.keep8(m, False, None), adamw_ref.keep8(v.sqrt(), True, None)]
    w = torch.zeros(n, dtype=torch.float32 if weights == "f32" else BF, device=dev())
    master = torch.zeros(n, device=dev()) if weights == "bf16+f32" else None
    on = lambda x: x.to(dev())  # noqa: E731
    table = gdn.AdamwTable([w], [on(g)], [on(codes[0][0])], [on(codes[1][0])], masters=None if master is None else [master],
                           m_scales=[on(codes[0][1])], v_scales=[on(codes[1][1])])
    gdn.gdn_adamw_step(table, 1.0, 0.0, B2, eps, t)
    torch.cuda.synchronize()
    f = np.float32
    r = adamw_ref.load8(*codes[1]).numpy()
    with np.errstate(all="ignore"):
        v32 = (r * r) * f(B2) + (g.numpy() * g.numpy()) * f(1 - B2)
        d = np.sqrt(v32) * f(1 / math.sqrt(1 - B2 ** t)) + f(eps)
    return (w if master is None else master).cpu(), g, torch.from_numpy(d), w


@pytest.mark.parametrize("weights", ["f32", "bf16+f32"])
@pytest.mark.parametrize("size", [1e-3, 1e-12, 1e12])
def test_quotient(weights, size):
    # half a step (2^-24 of the quotient) and, where the quotient all but lies between two floats, 2^-44 more
    say("adamw quotient", weights, size)
    gen = torch.Generator().manual_seed(2)
    n = 200001
    g = torch.randn(n, generator=gen) * size * torch.exp(torch.randn(n, generator=gen))
    got, m, d, w = divided(weights, g, g * 0.5, g.square() * torch.rand(n, generator=gen) + size ** 2, 4, eps=EPS * size)
    want = -m.to(F64) / d.to(F64)
    off = (got.to(F64) - want).abs() / want.abs()
    assert float(off.max()) <= 2.0 ** -24 * (1 + 2.0 ** -18), float(off.max() * 2 ** 24)
    if weights == "bf16+f32":
        assert torch.equal(w.cpu(), got.to(BF))


@pytest.mark.parametrize("weights", ["f32", "bf16", "bf16+f32"])
def test_quotients_without_a_value(weights):
    # 0 / 0, m / 0, an infinite divisor, an infinite or missing m: as a division has them
    say("adamw quotients without a value", weights)
    g = torch.tensor([0.0, 0.0, 1e30, -1e30, math.inf, -math.inf, math.nan, 1.0, -2.0, 1e-30, 3e38, -0.0])
    g = torch.cat([g, torch.full((250,), 0.5)])
    z = torch.zeros_like(g)
    for eps in (0.0, 1e-8):
        got, m, d, w = divided(weights, g, z, z, 1, eps=eps)
        want = -(m / d)
        if weights == "bf16":
            want = want.to(BF)
        assert torch.equal(got.isnan(), want.isnan()), eps
        both = ~want.isnan()
        assert bool(((got == want) | ((got.double() - want.double()).abs() <= 2.0 ** -8 * want.double().abs()))[both].all()), eps
