"""GPU tests of the recurrence's forms that widths and lengths choose between, each
against the definition in 64 bits: blocks of channels in the order of eight XCDs,
one segment with longer runs, and single channels a lane.  The route line tells
the form: the clearing goes ahead where there are several segments, and the grid is
segments times blocks of 64 channels."""
import re

import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
import linrec_ref
from gpu_common import dev, say
from test_gpu_linrec import SCALES, check, close, inputs, on

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def segments(B, T, D, io, gate, cu=None, backward=False):
    """Segments of a call of these sizes, by the route line of its plan."""
    lib, code = gdn.linrec._lib(), {"f32": 0, "bf16": 1}
    c = (None if cu is None else 0x8000)
    if backward:
        st = lib.gdn_linrec_backward_plan(0x1000, 0x2000, 0x3000, None, 0x4000, None, 0x5000, 0x6000, None, B, T, D, D, D, D, D, D,
                                          D, c, 0, code[io], code[gate], 0x10000, 1 << 40)
    else:
        st = lib.gdn_linrec_forward_plan(0x1000, 0x2000, None, 0x3000, None, B, T, D, D, D, D, c, 0, code[io], code[gate], 0x10000,
                                         1 << 40)
    assert st == 0
    line = gdn.last_route()
    n = int(re.search(r"grid=\[(\d+),1,1\]", line)[1])
    blocks = -(-D // 64)
    assert n % blocks == 0 and ("clear" in line) == (n > blocks), line
    return n // blocks


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("B,T,D", [(1, 600, 512), (2, 290, 1000), (1, 520, 4096)])
def test_blocks_by_eight(io, gate, scale, B, T, D):
    # 8, 16 (the last one short) and 64 blocks of channels, several segments each way
    say("linrec blocks by eight", io, gate, scale, B, T, D)
    assert -(-D // 64) % 8 == 0
    assert segments(B, T, D, io, gate) > 1 and segments(B, T, D, io, gate, backward=True) > 2
    check(inputs(B * T, D, io, gate, B), scale, B, T)


def test_blocks_by_eight_packed():
    say("linrec blocks by eight, packed")
    cu, D = [0, 100, 100, 130, 555, 700], 512
    check(inputs(720, D, "bf16", "bf16", 5), "root", 5, 720, cu=cu, pad=3)


# rows of the longest call of one segment with runs as long as ever, and with longer ones
LIMITS = {("bf16", "bf16"): (256, 512), ("bf16", "f32"): (128, 384), ("f32", "f32"): (128, 384)}


def test_which_calls_take_one_segment():
    for (io, gate), (usual, brief) in LIMITS.items():
        assert [segments(1, n, 768, io, gate) for n in (1, usual, usual + 1, brief, brief + 1)] == [1, 1, 1, 1, -(-(brief + 1) // usual)]
        assert segments(1, brief, 2048, io, gate) == 1 and segments(1, brief, 2049, io, gate) == -(-brief // usual)


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("D,pad", [(72, 0), (768, 0), (333, 5)])
def test_one_segment(io, gate, scale, D, pad):
    # from the first length that takes longer runs to the last one, states in and out; two sequences
    # whose border lies inside a run, at a run's end (300 / 2 = 150 rows) and in the last run
    say("linrec one segment", io, gate, scale, D, pad)
    usual, brief = LIMITS[io, gate]
    for B, T in ((1, usual + 1), (1, 300), (2, 150), (1, brief), (brief // 3, 3), (1, brief - 5)):
        assert segments(B, T, D, io, gate) == 1 and B * T > usual
        check(inputs(B * T, D, io, gate, B), scale, B, T, pad=pad)


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("scale,D", [("plain", 768), ("complement", 72), ("root", 130)])
def test_one_segment_packed(io, gate, scale, D):
    # borders inside runs, at their ends, in the last run; empty sequences, rows behind the last one
    say("linrec one segment, packed", io, gate, scale, D)
    usual, brief = LIMITS[io, gate]
    for cu, rows in (([0, 0, 3, 8, 12, 96, 97, 251, 251, brief - 2], brief), ([0, 64, 128, usual], usual + 3),
                     ([0, brief - 1, brief], brief), ([5, 5, 6], usual + 9)):
        cu = [0] + cu[1:]
        assert segments(len(cu) - 1, rows, D, io, gate, cu) == 1
        c = inputs(rows, D, io, gate, len(cu) - 1)
        for k in ("x", "log_a", "dy"):
            c[k][cu[-1]:] = float("nan")
        y, got = check(c, scale, len(cu) - 1, rows, cu=cu)
        for t in (y, got["dx"], got["dlog_a"]):
            assert bool((t[cu[-1]:] == 0).all())


@pytest.mark.parametrize("io,gate,D", [("bf16", "bf16", 7), ("bf16", "f32", 3), ("f32", "f32", 1)])
def test_single_channels_of_long_sequences(io, gate, D):
    # one channel a lane, 64 rows a segment: 141 segments one behind the other
    say("linrec narrow and long", io, gate, D)
    rows, cu = 9000, [0, 17, 8200, 9000]
    assert segments(3, rows, D, io, gate, cu) == 141
    check(inputs(rows, D, io, gate, 3), "root", 3, rows, cu=cu)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("gate", ["bf16", "f32"])
def test_borders_of_the_decay(scale, gate):
    # gates at -1/4, where one evaluation of 1 - a takes over from the other, and at their neighbours
    say("linrec border of the decay", scale, gate)
    rows, D = 400, 64
    io = "bf16" if gate == "bf16" else "f32"
    c = inputs(rows, D, io, gate, 1)
    t = c["log_a"].dtype
    step = 0.25 * torch.finfo(t).eps
    for i, v in enumerate((-0.25, -0.25 - step, -0.25 + step / 2, -0.125, -0.125 - step / 2, -0.125 + step / 4)):
        c["log_a"][11 + 60 * i:41 + 60 * i] = torch.tensor(v, dtype=t)
    check(c, scale, 1, rows)


def test_step_and_sequence_agree_on_forms():
    # one row of many sequences next to one token of them
    say("linrec step against a row")
    B, D = 130, 1000
    c = inputs(B, D, "bf16", "bf16", B)
    y, hf = gdn.linrec_forward(on(c["x"])[:, None], on(c["log_a"])[:, None], h0=on(c["h0"]), input_scale="root")
    h = on(c["h0"]).clone()
    table = torch.tensor([h[b].data_ptr() for b in range(B)], dtype=torch.int64, device=dev())
    ys = gdn.linrec_step(table, on(c["x"]), on(c["log_a"]), input_scale="root")
    torch.cuda.synchronize()
    assert torch.equal(ys, y[:, 0]) and torch.equal(h, hf)
    ry, rh, oy, oh = linrec_ref.forward(c["x"], c["log_a"], c["h0"], linrec_ref.spans(B, 1, None), "root")
    close(hf, rh, oh, "states")
