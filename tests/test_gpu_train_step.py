"""A training step of one gated delta rule layer, its operators together as they
are used: checkpoints of q, k, v; the prefill; the gated norm with checkpoints of
its inputs; and back through the norm and the recurrence.  Checked against
autograd through the whole step in 64 bits."""
import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
import synth
import train_ref
from gpu_common import rel_err, say, to_dev
from train_ref import F64, two_norm

pytestmark = pytest.mark.gpu


def reference(inp, z, w, dy, x_at=None, z_at=None):
    """Gradients of sum(norm(rule(...)) * silu(z) * dy); with x_at the norm's
    gradients are taken there (what a checkpoint stands for) and handed on."""
    o64 = None
    leaf = {n: inp[n].to(F64).clone().requires_grad_() for n in ("q", "k", "v", "log_g", "beta")}
    outs = []
    for b in range(inp["q"].shape[0]):
        Hv, dk, dv = inp["v"].shape[2], inp["q"].shape[3], inp["v"].shape[3]
        o, _ = train_ref.delta_rule(*(leaf[n][b] for n in ("q", "k", "v", "log_g", "beta")), torch.zeros((Hv, dk, dv), dtype=F64))
        outs.append(o)
    o64 = torch.stack(outs)
    B, T, Hv, dv = o64.shape
    x = (o64.detach() if x_at is None else x_at.to(F64)).reshape(B * T, Hv, dv)
    ng = train_ref.norm_grads(dy.reshape(B * T, Hv, dv), x, w, (z if z_at is None else z_at).reshape(B * T, Hv, dv))
    got = torch.autograd.grad(o64, list(leaf.values()), ng["dx"].reshape(B, T, Hv, dv))
    return o64.detach(), ng, {"d" + n: t for n, t in zip(leaf, got)}


def test_step_fp32():
    # fp32 throughout: 1e-4 of the largest entry, the generic kernels' bound
    say("training step fp32")
    B, T, Hk, Hv, d = 2, 130, 1, 3, 32
    inp = synth.prefill_inputs(B, T, Hk, Hv, d, d, io=torch.float32, seed=21)
    gen = torch.Generator().manual_seed(22)
    z, dy, w = torch.randn(B, T, Hv, d, generator=gen), torch.randn(B, T, Hv, d, generator=gen), 1 + 0.1 * torch.randn(d, generator=gen)
    g = to_dev(inp)
    o, _, _ = gdn.chunk_prefill(g["q"], g["k"], g["v"], g["log_g"], g["beta"], chunk=32)
    rows = lambda t: t.reshape(B * T, Hv, d)  # noqa: E731
    y, _ = gdn.norm_forward(rows(o), w.to(o.device), z=rows(z.to(o.device)))
    n = gdn.norm_backward(rows(dy.to(o.device)), rows(o), w.to(o.device), z=rows(z.to(o.device)))
    c, _ = gdn.chunk_backward(g["q"], g["k"], g["v"], g["log_g"], g["beta"], n["dx"].view(o.shape))
    o64, ng, rg = reference(inp, z, w, dy)
    y64 = train_ref.norm(rows(o64), w.double(), rows(z).double())
    assert rel_err(y, y64.numpy()) <= 1e-4
    for k in ("dw", "dz"):
        assert rel_err(n[k], ng[k].numpy()) <= 1e-4, k
    for k in rg:
        assert rel_err(c[k], rg[k].numpy()) <= 1e-4, k


def test_step_bf16_with_checkpoints():
    # bf16 and 8-bit checkpoints: q, k, v replaced by what their codes stand for
    # ahead of the step, the norm's gradients taken at its own checkpoints; then
    # the recurrence's gradients are those of the bf16 route for the norm's dx,
    # itself rounded once more: 1e-2 in the 2-norm, and as much again for dx
    say("training step bf16, checkpoints")
    B, T, Hk, Hv, d = 1, 200, 1, 3, 128
    inp = synth.prefill_inputs(B, T, Hk, Hv, d, d, seed=23)
    gen = torch.Generator().manual_seed(24)
    bf = torch.bfloat16
    z, dy = torch.randn(B, T, Hv, d, generator=gen).to(bf), torch.randn(B, T, Hv, d, generator=gen).to(bf)
    w = 1 + 0.1 * torch.randn(d, generator=gen)
    g = to_dev(inp)
    dv = g["q"].device
    kept = {n: gdn.ckpt8_store(g[n]) for n in "qkv"}
    for n in "qkv":
        g[n] = gdn.ckpt8_load(*kept[n])
        inp[n] = g[n].cpu()
    rows = lambda t: t.reshape(B * T, Hv, d)  # noqa: E731
    o, _, _ = gdn.chunk_prefill(g["q"], g["k"], g["v"], g["log_g"], g["beta"])
    y, ck = gdn.norm_forward(rows(o), w.to(dv), z=rows(z.to(dv)), ckpt=True)
    n = gdn.norm_backward(rows(dy.to(dv)), ck["x_codes"], w.to(dv), z=ck["z_codes"], x_exps=ck["x_exps"], z_exps=ck["z_exps"])
    c, route = gdn.chunk_backward(kept["q"][0], kept["k"][0], kept["v"][0], g["log_g"], g["beta"], n["dx"].view(o.shape),
                                  q_exps=kept["q"][1], k_exps=kept["k"][1], v_exps=kept["v"][1])
    assert route.startswith("gdn_bwd_prep"), route
    x_at, z_at = gdn.ckpt8_load(ck["x_codes"], ck["x_exps"], torch.float32).cpu(), gdn.ckpt8_load(ck["z_codes"], ck["z_exps"], torch.float32).cpu()
    o64, ng, rg = reference(inp, z, w, dy, x_at, z_at)
    assert two_norm(o, o64) <= 1e-2
    assert two_norm(n["dw"], ng["dw"]) <= 1e-5
    for k in ("dx", "dz"):
        assert two_norm(n[k].cpu().reshape(ng[k].shape), ng[k]) <= 2.0 ** -8, k
    for k in rg:
        assert two_norm(c[k], rg[k]) <= 2e-2, (k, two_norm(c[k], rg[k]))
