"""GPU tests of the delta rule's gradients against autograd through the token
recurrence in 64 bits.

Bounds.  Generic route (fp32): an entry is a sum over at most 128 columns, 64
rows of a chunk and the chunks behind it, formed by a chain of about 400 fp32
operations a chunk, each off by at most 2^-24 of the terms it adds: 400 * 2^-24
= 2.4e-5 of the largest entry a chunk; 1e-4 of it bounds the few chunks that a
decaying state remembers.
MFMA route (bf16): on the way to an entry about nine values are rounded to
bf16 (T, P, x, u, delta's gradient, dx, h, dh', the masked products, the
output), each off by at most 2^-8 and, as rounding errors of random sign, by
2^-8 / 3 of its size in the root mean square over a tensor: sqrt(9) * 2^-8 / 3 =
4e-3 in the 2-norm, bounded by 1e-2; a single entry is off by at most 9 * 2^-8 =
3.5e-2 of the largest one.  dlog_g sums products of such values over whole rows
and columns; the same bounds hold relative to its own norm for T >= 16."""
import numpy as np
import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
import oracle
import synth
import train_ref
from gpu_common import dev, rel_err, say, to_dev
from train_ref import two_norm

pytestmark = pytest.mark.gpu

F32_MAX, BF16_TWO, BF16_MAX = 1e-4, 1e-2, 9 * 2.0 ** -8
NAMES = ("dq", "dk", "dv", "dlog_g", "dbeta")


def inputs(B, T, Hk, Hv, dk, dv, io, h0=False, dht=False, lens=None, seed=0, gate_scale=0.1):
    inp = synth.prefill_inputs(B, T, Hk, Hv, dk, dv, io=io, h0=h0, seed=seed, lengths=lens, gate_scale=gate_scale)
    rng = np.random.default_rng(seed + 1000)
    inp["dout"] = torch.from_numpy(rng.standard_normal(tuple(inp["v"].shape)).astype(np.float32)).to(io)
    inp["dht"] = torch.from_numpy((rng.standard_normal((B, Hv, dk, dv)) * 0.05).astype(np.float32)) if dht else None
    return inp


def gpu(inp, want_dh0=True, **kw):
    g = to_dev(inp)
    out, route = gdn.chunk_backward(g["q"], g["k"], g["v"], g["log_g"], g["beta"], g["dout"], h0=g["h0"],
                                    dh_final=g["dht"], cu_seqlens=g["cu_seqlens"], want_dh0=want_dh0, **kw)
    torch.cuda.synchronize()
    return out, route


def check(inp, mfma, **kw):
    out, route = gpu(inp, **kw)
    assert route.startswith("gdn_bwd_prep" if mfma else "gdn_backward_prep"), route
    ref = train_ref.delta_rule_grads(inp, inp["dout"], inp["dht"])
    for n in out:
        r = ref[n]
        assert bool(torch.isfinite(out[n].float()).all()), n
        if float(r.abs().max()) == 0.0:
            assert bool((out[n] == 0).all()), n
        elif mfma:
            assert two_norm(out[n], r) <= BF16_TWO, (n, two_norm(out[n], r))
            assert rel_err(out[n], r.numpy()) <= BF16_MAX, n
        else:
            assert rel_err(out[n], r.numpy()) <= F32_MAX, (n, rel_err(out[n], r.numpy()))
    return out, ref


GENERIC = [
    # B, T, Hk, Hv, dk, dv, h0, dht
    (1, 1, 1, 1, 1, 1, True, True),
    (1, 1, 1, 1, 16, 16, False, False),
    (2, 3, 1, 3, 3, 20, True, True),
    (1, 63, 2, 2, 33, 17, False, True),
    (1, 64, 1, 2, 32, 32, True, False),
    (2, 65, 1, 4, 48, 96, True, True),
    (1, 130, 2, 6, 64, 100, True, True),
    (1, 200, 1, 2, 128, 128, True, True),
    (3, 100, 1, 1, 100, 24, False, False),
]


@pytest.mark.parametrize("case", GENERIC, ids=lambda c: "B%d_T%d_Hk%d_Hv%d_dk%d_dv%d_h%d_t%d" % c)
def test_generic(case):
    B, T, Hk, Hv, dk, dv, h0, dht = case
    say("generic backward", case)
    check(inputs(B, T, Hk, Hv, dk, dv, torch.float32, h0, dht, seed=T), mfma=False)


@pytest.mark.parametrize("dk", [20, 50, 100])
@pytest.mark.parametrize("dv", [20, 50, 90, 120])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_generic_head_sizes(dk, dv, io):
    # every pair of padded sizes, with the end state's and the start state's gradients;
    # bf16 gradients of fp32 sums are one rounding off (2^-8 of the value)
    say("generic sizes", dk, dv, io)
    inp = inputs(1, 70, 1, 2, dk, dv, io, True, True, seed=dk + dv)
    out, route = gpu(inp)
    assert route.startswith("gdn_backward_prep"), route
    ref = train_ref.delta_rule_grads(inp, inp["dout"], inp["dht"])
    for n in out:
        bound = F32_MAX + (2.0 ** -8 if out[n].dtype == torch.bfloat16 else 0.0)
        assert rel_err(out[n], ref[n].numpy()) <= bound, (n, rel_err(out[n], ref[n].numpy()))


def test_generic_wide_and_narrow_walks():
    # 9 sequences of 8 v-heads, 64 columns: walks of 32 columns; one sequence: of 16.
    # A column's products are the same ones in the same order.
    say("generic walks")
    inp = inputs(9, 70, 4, 8, 40, 50, torch.float32, True, True, seed=12)
    a, _ = check(inp, mfma=False)
    for b in range(9):
        one = {n: t[b:b + 1] if torch.is_tensor(t) else t for n, t in inp.items()}
        c, _ = gpu(one)
        for n in a:
            assert torch.equal(a[n][b], c[n][0]), (n, b)


MFMA = [
    # B, T, Hk, Hv, h0, dht
    (1, 16, 1, 1, False, False),
    (1, 63, 1, 3, True, True),
    (2, 64, 2, 2, False, True),
    (1, 65, 1, 2, True, False),
    (1, 200, 2, 6, True, True),
    (2, 129, 1, 4, False, False),
]


@pytest.mark.parametrize("case", MFMA, ids=lambda c: "B%d_T%d_Hk%d_Hv%d_h%d_t%d" % c)
def test_mfma(case):
    B, T, Hk, Hv, h0, dht = case
    say("mfma backward", case)
    check(inputs(B, T, Hk, Hv, 128, 128, torch.bfloat16, h0, dht, seed=T), mfma=True)


@pytest.mark.parametrize("T", [1, 2, 5])
def test_mfma_short(T):
    # few values of a gate's gradient: held to the largest entry's bound alone
    say("mfma short", T)
    inp = inputs(2, T, 1, 3, 128, 128, torch.bfloat16, True, True, seed=40 + T)
    out, _ = gpu(inp)
    ref = train_ref.delta_rule_grads(inp, inp["dout"], inp["dht"])
    for n in out:
        assert rel_err(out[n], ref[n].numpy()) <= BF16_MAX, n


def test_mfma_heads_together():
    # 33 chunks x 8 v-heads: more v-heads than compute units, a workgroup takes a k-head whole
    say("mfma, k-heads whole")
    check(inputs(33, 9, 4, 8, 128, 128, torch.bfloat16, True, True, seed=77), mfma=True)


def test_mfma_heads_together_and_apart():
    # 5 x 3 chunks x 18 v-heads go by k-heads, one sequence's 3 x 18 by v-heads. What belongs
    # to a v-head is the same to the bit; dq and dk add the same fp32 products in another order
    # (3 x 64 x 128 terms at most, far below 2^-16 of the largest entry), so the roundings to
    # bf16 land at most a step apart: 2^-7 of the value.
    say("mfma, together and apart")
    inp = inputs(5, 150, 6, 18, 128, 128, torch.bfloat16, True, True, seed=78)
    a, _ = gpu(inp)
    for b in range(5):
        one = {n: t[b:b + 1] if torch.is_tensor(t) else t for n, t in inp.items()}
        c, _ = gpu(one)
        for n in a:
            x, y = a[n][b].float(), c[n][0].float()
            if n in ("dq", "dk"):
                assert bool(((x - y).abs() <= 2.0 ** -7 * x.abs() + 2.0 ** -16 * x.abs().max()).all()), (n, b)
            else:
                assert torch.equal(x, y), (n, b)


LENS = [64, 0, 1, 130, 63, 0, 40]


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_packed_with_empty_sequences(io):
    say("packed backward", io)
    d = 128 if io == torch.bfloat16 else 40
    inp = inputs(len(LENS), 0, 1, 2, d, d, io, True, True, lens=LENS, seed=5)
    out, ref = check(inp, mfma=io == torch.bfloat16)
    for b, n in enumerate(LENS):
        if n == 0:
            assert torch.equal(out["dh0"][b].cpu(), inp["dht"][b])


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_rows_behind_the_last_sequence_are_left(io):
    say("rows behind", io)
    d = 128 if io == torch.bfloat16 else 32
    inp = inputs(2, 0, 1, 2, d, d, io, lens=[70, 100], seed=6)
    inp["cu_seqlens"] = torch.tensor([0, 70, 101], dtype=torch.int32)     # rows 101 .. 169 belong to nobody
    for t in ("q", "k", "v", "dout", "log_g", "beta"):
        inp[t][101:] = float("nan")
    g = to_dev(inp)
    out = {n: torch.full(inp[n[1:]].shape, 7.0, dtype=io, device=dev()) for n in NAMES}
    code = gdn.GDN_BF16 if io == torch.bfloat16 else gdn.GDN_F32
    ws = torch.empty(gdn.gdn_backward_workspace_bytes(2, 170, 1, 2, d, d, code, code, packed=True), dtype=torch.uint8, device=dev())
    gdn.gdn_chunk_backward(g["q"], g["k"], g["v"], None, None, None, g["log_g"], g["beta"], None, g["dout"], None,
                           out["dq"], out["dk"], out["dv"], out["dlog_g"], out["dbeta"], None, 2, 170, 1, 2, d, d,
                           cu_seqlens=g["cu_seqlens"], workspace=ws)
    for n in NAMES:
        assert bool((out[n][101:] == 7.0).all()), n
        assert bool(torch.isfinite(out[n][:101].float()).all()) and not bool((out[n][:101] == 7.0).all()), n


def test_offsets_outside_the_rows_are_clamped():
    say("clamped offsets")
    inp = inputs(2, 0, 1, 1, 16, 16, torch.float32, lens=[30, 20], seed=7)
    a, _ = gpu(inp)
    inp["cu_seqlens"] = torch.tensor([0, 30, 5000], dtype=torch.int32)
    b, _ = gpu(inp)
    for n in NAMES:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_offsets_out_of_order_stay_in_the_workspace(io):
    # twice 0 .. 640 in three sequences: 20 chunks where the workspace has 10 + 3
    say("offsets out of order", io)
    d = 128 if io == torch.bfloat16 else 32
    inp = inputs(3, 0, 1, 2, d, d, io, True, True, lens=[640, 0, 0], seed=8)
    inp["cu_seqlens"] = torch.tensor([0, 640, 0, 640], dtype=torch.int32)
    g = to_dev(inp)
    out = {n: torch.zeros(inp[n[1:]].shape, dtype=io, device=dev()) for n in NAMES}
    code = gdn.GDN_BF16 if io == torch.bfloat16 else gdn.GDN_F32
    n = gdn.gdn_backward_workspace_bytes(3, 640, 1, 2, d, d, code, code, packed=True)
    ws = torch.full((n + (32 << 20),), 171, dtype=torch.uint8, device=dev())
    dh0 = torch.zeros_like(g["h0"])
    gdn.gdn_chunk_backward(g["q"], g["k"], g["v"], None, None, None, g["log_g"], g["beta"], g["h0"], g["dout"],
                           g["dht"], out["dq"], out["dk"], out["dv"], out["dlog_g"], out["dbeta"], dh0, 3, 640, 1, 2,
                           d, d, cu_seqlens=g["cu_seqlens"], workspace=ws[:n])
    torch.cuda.synchronize()
    assert bool((ws[n:] == 171).all())


@pytest.mark.parametrize("lens", [None, [70, 1, 129]])
def test_checkpoints_equal_their_values(lens):
    # a code times its power of two is a bf16 value: the MFMA route must give the
    # same bits from the codes as from those values
    say("backward from codes", lens)
    inp = inputs(1 if lens is None else 3, 150, 2, 4, 128, 128, torch.bfloat16, True, True, lens=lens, seed=8)
    g = to_dev(inp)
    kept = {n: gdn.ckpt8_store(g[n]) for n in "qkv"}
    codes, _ = gdn.chunk_backward(kept["q"][0], kept["k"][0], kept["v"][0], g["log_g"], g["beta"], g["dout"],
                                  h0=g["h0"], dh_final=g["dht"], cu_seqlens=g["cu_seqlens"], q_exps=kept["q"][1],
                                  k_exps=kept["k"][1], v_exps=kept["v"][1])
    for n in "qkv":
        inp[n] = gdn.ckpt8_load(*kept[n]).cpu()
    vals, _ = gpu(inp)
    for n in vals:
        assert torch.equal(codes[n], vals[n]), n


def test_codes_and_bf16_on_the_generic_route():
    say("generic from codes and bf16")
    for dk, dv in ((40, 24), (128, 128)):
        inp = inputs(1, 90, 1, 2, dk, dv, torch.bfloat16, True, True, seed=9)
        g = to_dev(inp)
        kept = {n: gdn.ckpt8_store(g[n]) for n in "qkv"}
        dout = g["dout"].float()
        a, route = gdn.chunk_backward(kept["q"][0], kept["k"][0], kept["v"][0], g["log_g"], g["beta"], dout, h0=g["h0"],
                                      dh_final=g["dht"], q_exps=kept["q"][1], k_exps=kept["k"][1], v_exps=kept["v"][1])
        assert route.startswith("gdn_backward_prep"), route
        for n in "qkv":
            inp[n] = gdn.ckpt8_load(*kept[n]).cpu()
        ref = train_ref.delta_rule_grads(inp, inp["dout"], inp["dht"])
        h = to_dev(inp)
        b, _ = gdn.chunk_backward(h["q"], h["k"], h["v"], h["log_g"], h["beta"], dout, h0=h["h0"], dh_final=h["dht"])
        for n in a:
            assert rel_err(a[n], ref[n].numpy()) <= F32_MAX, n
            assert torch.equal(a[n], b[n]), n


def test_unaligned_pointers_take_the_generic_route():
    say("unaligned")
    inp = inputs(1, 70, 1, 2, 128, 128, torch.bfloat16, seed=10)
    aligned, _ = gpu(inp)
    g = to_dev(inp)
    shifted = torch.empty(inp["q"].numel() + 1, dtype=torch.bfloat16, device=dev())[1:].view(inp["q"].shape)
    shifted.copy_(g["q"])
    out, route = gdn.chunk_backward(shifted, g["k"], g["v"], g["log_g"], g["beta"], g["dout"])
    assert route.startswith("gdn_backward_prep") and "aligned" in route
    for n in out:
        assert two_norm(out[n], aligned[n].cpu().double()) <= 2 * BF16_TWO


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_zero_beta_and_repeated_keys(io):
    # beta = 0 (padded or ignored tokens) divides nothing; beta = 1 with one key
    # throughout is the longest chain of the triangular inverse
    say("zero beta, repeated keys", io)
    d = 128 if io == torch.bfloat16 else 32
    inp = inputs(1, 100, 1, 2, d, d, io, True, True, seed=11)
    inp["beta"][0, ::3] = 0.0
    inp["beta"][0, 1::3] = 1.0
    check(inp, mfma=io == torch.bfloat16)
    inp["k"][:] = inp["k"][:, :1]
    if io == torch.float32:
        check(inp, mfma=False)
    else:
        out, _ = gpu(inp)
        assert all(bool(torch.isfinite(t.float()).all()) for t in out.values())


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [0.0, -5.0, -200.0])
def test_gates_from_none_to_complete(io, g):
    say("gates", io, g)
    d = 128 if io == torch.bfloat16 else 32
    inp = inputs(1, 130, 1, 2, d, d, io, True, True, seed=12)
    inp["log_g"][0, 40:] = g
    if g == 0.0:
        inp["log_g"][:] = 0.0
    check(inp, mfma=io == torch.bfloat16)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_padded_rows_change_nothing(io):
    # a batch padded at the end with k = 0, beta = 0, log_g = 0 and a zero
    # gradient: the rows before, and dh0, get the same bits
    say("padded batch", io)
    d = 128 if io == torch.bfloat16 else 32
    inp = inputs(1, 200, 1, 2, d, d, io, True, True, seed=13)
    for n in ("q", "k", "v", "log_g", "beta", "dout"):
        inp[n][:, 150:] = 0
    long, _ = gpu(inp)
    short = {n: (t[:, :150].contiguous() if torch.is_tensor(t) and n not in ("h0", "dht") else t) for n, t in inp.items()}
    a, _ = gpu(short)
    for n in NAMES:
        assert torch.equal(long[n][:, :150], a[n]), n
    # the states behind pass through two more steps of the walk, each rounding
    # what it hands on to nothing coarser than fp32
    assert rel_err(long["dh0"], a["dh0"].cpu().double().numpy()) <= 1e-6


def test_no_gradient_in_gives_none_out():
    say("zero gradient")
    for io, d in ((torch.float32, 24), (torch.bfloat16, 128)):
        inp = inputs(1, 80, 1, 2, d, d, io, True, True, seed=14)
        inp["dout"].zero_()
        inp["dht"].zero_()
        out, _ = gpu(inp)
        assert all(bool((t == 0).all()) for t in out.values())


def test_no_tokens():
    say("T = 0")
    for io, d in ((torch.float32, 24), (torch.bfloat16, 128)):
        inp = inputs(2, 0, 1, 2, d, d, io, True, True, seed=15)
        out, _ = gpu(inp)
        assert out["dq"].numel() == 0
        assert torch.equal(out["dh0"].cpu(), inp["dht"])


def test_shared_heads_sum():
    # dq and dk of a k-head are the sums over its v-heads
    say("shared heads")
    inp = inputs(1, 100, 2, 6, 32, 48, torch.float32, True, True, seed=16)
    a, _ = gpu(inp)
    wide = dict(inp, q=inp["q"].repeat_interleave(3, 2), k=inp["k"].repeat_interleave(3, 2))
    b, _ = gpu(wide)
    for n in ("dq", "dk"):
        assert rel_err(a[n], b[n].cpu().double().unflatten(2, (2, 3)).sum(3).numpy()) <= 1e-6, n
    for n in ("dv", "dlog_g", "dbeta", "dh0"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_runs_streams_and_graphs_give_the_same_bits(io):
    say("runs, streams, graph", io)
    d = 128 if io == torch.bfloat16 else 64
    inp = inputs(3, 0, 1, 3, d, d, io, True, True, lens=[150, 0, 90], seed=17)
    first, _ = gpu(inp)
    g = to_dev(inp)
    code = gdn.GDN_BF16 if io == torch.bfloat16 else gdn.GDN_F32
    out = {n: torch.empty(inp[n[1:]].shape, dtype=io, device=dev()) for n in NAMES}
    out["dh0"] = torch.empty_like(g["h0"])
    ws = torch.empty(gdn.gdn_backward_workspace_bytes(3, 240, 1, 3, d, d, code, code, packed=True), dtype=torch.uint8, device=dev())

    def call(stream=None):
        gdn.gdn_chunk_backward(g["q"], g["k"], g["v"], None, None, None, g["log_g"], g["beta"], g["h0"], g["dout"],
                               g["dht"], out["dq"], out["dk"], out["dv"], out["dlog_g"], out["dbeta"], out["dh0"],
                               3, 240, 1, 3, d, d, cu_seqlens=g["cu_seqlens"], workspace=ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    torch.cuda.synchronize()
    for n in out:
        assert torch.equal(out[n], first[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for r in range(3):
        for t in out.values():
            t.fill_(0)
        ws.fill_(0xFF)                  # a workspace needs no initialisation
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], first[n]), (r, n)


def test_two_calls_at_once():
    say("two streams")
    inp = [inputs(1, 300, 1, 3, 128, 128, torch.bfloat16, True, True, seed=18 + i) for i in range(2)]
    alone = [gpu(i)[0] for i in inp]
    on = [to_dev(i) for i in inp]
    torch.cuda.synchronize()
    got = []
    for g in on:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(gdn.chunk_backward(g["q"], g["k"], g["v"], g["log_g"], g["beta"], g["dout"], h0=g["h0"],
                                          dh_final=g["dht"])[0])
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_gradient_against_differences():
    # the 64-bit oracle's forward pass, in a random direction of all inputs
    say("differences")
    inp = inputs(1, 70, 1, 2, 16, 24, torch.float32, True, True, seed=19)
    out, _ = gpu(inp)
    rng = np.random.default_rng(20)
    step = {n: rng.standard_normal(tuple(inp[n].shape)) for n in ("q", "k", "v", "beta", "h0")}
    step["log_g"] = -np.abs(rng.standard_normal(tuple(inp["log_g"].shape))) * inp["log_g"].double().abs().numpy()

    def loss(h):
        a = {n: inp[n].double().numpy() + h * step[n] for n in step}
        o, S = oracle.prefill(torch.from_numpy(a["q"]), torch.from_numpy(a["k"]), torch.from_numpy(a["v"]),
                              torch.from_numpy(a["log_g"]), torch.from_numpy(a["beta"]), torch.from_numpy(a["h0"]))
        return float((o * inp["dout"].double().numpy()).sum() + (S * inp["dht"].double().numpy()).sum())

    got = sum(float((out["d" + n].cpu().double().numpy() * step[n]).sum()) for n in step)
    # Richardson: errors of the fourth order in h; the oracle's inputs may be fp32,
    # whose rounding (2^-24 of each of about 10^4 terms over h) sets the bound
    h = 2.0 ** -7
    d1, d2 = ((loss(s) - loss(-s)) / (2 * s) for s in (h, h / 2))
    want = (4 * d2 - d1) / 3
    assert abs(got - want) <= 2e-3 * max(1.0, abs(want)), (got, want)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [-104.0, -1e5, -1e6, -1e9, float(torch.finfo(torch.float32).min)])
@pytest.mark.parametrize("at", ["once", "twelve a chunk", "every other token"])
def test_resets_between_mild_gates(io, g, at):
    # a gate that forgets everything, of any strength, among gates of about -0.07: the
    # decays behind it are differences of sums that hold it
    say("resets", io, g, at)
    d = 128 if io == torch.bfloat16 else 32
    inp = inputs(1, 130, 1, 2, d, d, io, True, True, seed=30)
    rows = torch.tensor([20, 90]) if at == "once" else torch.arange(3, 130, 5 if at == "twelve a chunk" else 2)
    inp["log_g"][0, rows] = g
    check(inp, mfma=io == torch.bfloat16)
