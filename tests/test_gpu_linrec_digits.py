"""GPU tests of the digits of the recurrence's decays: a = exp(log_a), 1 - a and
sqrt(1 - a^2), each read off one row or one token.

How far they may be off, in u = 2^-24.  For -1/4 < l < 0, q = expm1(l) is l + l^2 p: l^2 p is at
most l / 8 of l and carries two and a half roundings (0.3 u of q), p's polynomial is 2^-28 off
(0.1 u), the last addition rounds once (1 u): 1.5 u of q.  a = 1 + q rounds to half of u (it lies
between 1/2 and 1) and has q's share, at most 1.5 u |l|.  With the plain scale this holds for |l| < 1/64 alone: the cubic's next
term is l^4 / 24, 2.6 u |l| at most, and the factor behind the last multiply-add is 1.1 u off, times
|l|: (1/2 + 4 |l|) u.  Elsewhere a is 2 (2 + |l|) u of itself off
(the product with log2 e rounded and the hardware's exp2), and 1 - a, at least 0.22, 16 u.  A root halves
what its argument is off (1 - a's 1.5 or 16 u, 2 u of 1 + a and the product) and adds 2 u by the hardware's."""
import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
from gpu_common import dev, say

pytestmark = pytest.mark.gpu

F64, BF, F32 = torch.float64, torch.bfloat16, torch.float32
U = 2.0 ** -24


def gates(dtype):
    """Log decays from -1e-8 to -2, most of them above -1/4, the borders' neighbours among them."""
    g = torch.Generator().manual_seed(6)
    l = torch.cat([-torch.logspace(-8, -0.61, 1500), -0.25 * torch.rand(2000, generator=g), -torch.linspace(0.25, 2, 500)])
    at = torch.tensor([-0.25, -0.125], dtype=dtype)
    ulp = torch.tensor([0.25, 0.125]) * torch.finfo(dtype).eps
    return torch.cat([l.to(dtype), at, at + ulp.to(dtype), at - ulp.to(dtype), torch.zeros(2, dtype=dtype)])


def decays(l, scale):
    """In 64 bits a and 1 - a, with what each may be off."""
    l = l.to(F64)
    a, d = torch.exp(l), -torch.expm1(l)
    near = l > -0.25
    far = 2 * (2 + l.abs()) * U * a
    if scale == "plain":
        oa = torch.where(l > -1 / 64, (0.5 + 4 * l.abs()) * U, far)
    else:
        oa = torch.where(near, (0.5 + 1.5 * l.abs()) * U, far)
    od = torch.where(near, 1.5 * U * d, 16 * U * d)
    return a, d, oa, od


def call(io, l, x, h0, scale, way):
    """The state behind one row (or token), or backward dh0 with dy 0 and dh_final h0."""
    D = l.numel()
    l, x, h0 = l.to(dev()), torch.full((D,), x, dtype=io, device=dev()), torch.full((D,), h0, device=dev())
    if way == "sequence":
        return gdn.linrec_forward(x[None, None], l[None, None], h0=h0[None], input_scale=scale)[1][0].cpu().to(F64)
    if way == "token":
        table = torch.tensor([h0.data_ptr()], dtype=torch.int64, device=dev())
        gdn.linrec_step(table, x[None], l[None], input_scale=scale)
        torch.cuda.synchronize()
        return h0.cpu().to(F64)
    z = torch.zeros((1, 1, D), dtype=io, device=dev())
    return gdn.linrec_backward(z, x[None, None], l[None, None], z, dh_final=h0[None], input_scale=scale,
                               want_dh0=True)["dh0"][0].cpu().to(F64)


TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("scale", ["plain", "complement", "root"])
@pytest.mark.parametrize("way", ["sequence", "token", "backward"])
def test_decays(io, gate, scale, way):
    # h0 = 1 and no input: the state is a itself
    say("linrec decays", io, gate, scale, way)
    l = gates(gate)
    got = call(io, l, 0.0, 1.0, scale, way)
    a, _, off, _ = decays(l, scale)
    d = (got - a).abs()
    assert bool((d <= off).all()), (float((d / off).max()), l[d > off][:5], int((d > off).sum()))


@pytest.mark.parametrize("scale", ["plain", "complement", "root"])
@pytest.mark.parametrize("B", [1, 64])
def test_slow_decays_add_up_by_chance(scale, B):
    # what 20,000 slow gates leave of a state.  A decay's rounding and a product's are each at most u / 2
    # of 1/2 to 1, 0.58 u of the value as a root mean square, of either sign: 0.82 u a row, 116 u in all,
    # of which six times.  Decays that are an eighth of u too low each would be 2500 u
    say("linrec slow decays", scale, B)
    T, D = 20000 // B, 64
    g = torch.Generator().manual_seed(11)
    l = -(1e-4 + 4e-4 * torch.rand(B, T, D, generator=g))
    z, h = torch.zeros(B, T, D, device=dev()), torch.ones(B, D, device=dev())
    _, hf = gdn.linrec_forward(z, l.to(dev()), h0=h, input_scale=scale)
    got, want = hf.cpu().to(F64), torch.exp(l.to(F64).sum(1))
    off = 6 * 0.82 * T ** 0.5 * U
    e = (got - want) / want
    assert float(e.abs().max()) <= off, float(e.abs().max() / U)
    assert abs(float(e.mean())) <= off / e.numel() ** 0.5, float(e.mean() / U)


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("scale", ["complement", "root"])
@pytest.mark.parametrize("way", ["sequence", "token"])
def test_input_scales(io, gate, scale, way):
    # an input of 1 and no state before: the state is 1 - a or sqrt(1 - a^2)
    say("linrec input scales", io, gate, scale, way)
    l = gates(gate)
    got = call(io, l, 1.0, 0.0, scale, way)
    _, d, _, od = decays(l, scale)
    want, off = d, od
    if scale == "root":
        want = torch.sqrt(-torch.expm1(2 * l.to(F64)))
        off = want * (od / d.clamp(min=1e-300) / 2 + U + 2 * U)
    e = (got - want).abs()
    assert bool((e <= off).all()), (float((e / off.clamp(min=1e-300)).max()), l[e > off][:5], int((e > off).sum()))


@pytest.mark.parametrize("scale", ["complement", "root"])
def test_input_scales_of_the_gradients(scale):
    # dx = c dy with dy 1
    say("linrec input scales, gradients", scale)
    l = gates(F32)
    one = torch.ones((1, 1, l.numel()), device=dev())
    got = gdn.linrec_backward(one, one, l.to(dev())[None, None], one, input_scale=scale)["dx"].cpu().to(F64).view(-1)
    _, d, _, od = decays(l, scale)
    want, off = d, od
    if scale == "root":                              # by the reciprocal root: its u and two products
        want = torch.sqrt(-torch.expm1(2 * l.to(F64)))
        off = want * (od / d.clamp(min=1e-300) / 2 + U + 4 * U)
    e = (got - want).abs()
    assert bool((e <= off).all()), (float((e / off.clamp(min=1e-300)).max()), l[e > off][:5], int((e > off).sum()))
