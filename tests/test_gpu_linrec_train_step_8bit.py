"""Training steps of a layer of the vector-state recurrence with 8-bit optimizer
states, each step against 64 bits from the states that the codes stand for: the
rounding of the states is in both, so that a step is as close as one with fp32
states."""
import pytest
import torch

import adamw_ref
import linear_attention_ssm_gated_amd as gdn
from gpu_common import dev, say
from test_gpu_linrec_train_step import B1, B2, EPS, LR, WD, F64, layer64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stochastic", [False, True])
def test_steps_from_what_the_codes_stand_for(stochastic):
    say("training steps of the linear recurrence, 8-bit states", stochastic)
    D, cu = 96, [0, 70, 70, 200]
    g = torch.Generator().manual_seed(77)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, r, z, dy = rn(200, D), rn(200, D), rn(200, D), rn(200, D)
    names = ("decay", "w")
    p = dict(decay=rn(D).to(dev()), w=(1 + 0.1 * rn(D)).to(dev()))
    grads = {k: torch.zeros_like(t) for k, t in p.items()}
    table = gdn.adamw_table([p[k] for k in names], [grads[k] for k in names], bits=8, weight_decay=[0.0, WD])
    gx, gr, gz, gdy = (t.to(dev()) for t in (x, r, z, dy))
    g_cu = torch.tensor(cu, dtype=torch.int32, device=dev())
    for t in range(1, 6):
        before = {k: p[k].cpu().to(F64).requires_grad_() for k in names}
        codes = {k: [table.states[s][i].cpu().clone() for s in ("m", "m_scales", "v", "v_scales")] for i, k in enumerate(names)}
        decay = p["decay"].detach().clone().requires_grad_()
        l = -torch.nn.functional.softplus(decay) * torch.sigmoid(gr)
        h, _ = gdn.linrec_forward(gx, l.detach(), cu_seqlens=g_cu, input_scale="root")
        nb = gdn.norm_backward(gdy[:, None], h[:, None], p["w"], z=gz[:, None])
        lb = gdn.linrec_backward(nb["dx"][:, 0], gx, l.detach(), h, cu_seqlens=g_cu, input_scale="root")
        l.backward(lb["dlog_a"])
        grads["decay"].copy_(decay.grad)
        grads["w"].copy_(nb["dw"])
        gdn.gdn_adamw_step(table, LR, B1, B2, EPS, t, stochastic=stochastic, seed=t)
        ry = layer64(before, x.to(F64), r.to(F64), z.to(F64), cu)
        got = torch.autograd.grad(ry, [before[k] for k in names], dy.to(F64))
        for k, gk in zip(names, got):
            assert float((grads[k].cpu().double() - gk).abs().max() / gk.abs().max()) <= 1e-4, k
            cm, sm, cv, sv = codes[k]
            m = B1 * adamw_ref.load8(cm.view(torch.uint8), sm).double() + (1 - B1) * gk
            v = B2 * adamw_ref.load8(cv.view(torch.uint8), sv).double() ** 2 + (1 - B2) * gk * gk
            c1, c2 = 1 - B1 ** t, 1 - B2 ** t
            d = torch.sqrt(v / c2) + EPS
            u = m / c1 / d
            want = before[k].detach() * (1 - LR * (WD if k == "w" else 0.0)) - LR * u
            # A gradient is e = 1e-4 of the largest off.  m moves by (1 - b1) e, and the root of v, by v's
            # change 2 (1 - b2) |g| e + (1 - b2) e^2, by at most sqrt(1 - b2) e, both over d; everything else
            # in fp32: 32 roundings of the update, and two of the weight
            e = 1e-4 * float(gk.abs().max())
            off = ((1 - B1) / c1 * e + u.abs() * ((1 - B2) / c2) ** 0.5 * e) / (d - ((1 - B2) / c2) ** 0.5 * e).clamp(min=1e-30)
            off = LR * (off + 32 * 2.0 ** -24 * u.abs()).clamp(max=1e3) + 2.0 ** -22 * want.abs()
            assert bool(((p[k].cpu().double() - want).abs() <= off).all()), (k, t)
            assert float(off.median()) <= 2e-3 * LR, (k, t)          # (the bound says something)
