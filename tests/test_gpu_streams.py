"""GPU tests of the allocating conveniences on a stream that is not the current
one: neither their workspace nor their outputs share memory with what the
current stream still uses, or takes next."""
import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
import synth
from gpu_common import dev, say, to_dev

pytestmark = pytest.mark.gpu

SPIN = 20_000_000      # cycles: some milliseconds, longer than the host needs for its calls


def calls():
    inp = to_dev(synth.prefill_inputs(1, 200, 2, 6, 128, 128, seed=3))
    gen = torch.Generator(dev()).manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device=dev(), dtype=torch.bfloat16)  # noqa: E731
    x, z, w = r(300, 6, 128), r(300, 6, 128), torch.rand(128, generator=gen, device=dev())
    do = r(1, 200, 6, 128)
    codes, exps = gdn.ckpt8_store(x)
    m, wt = r(64, 256), r(12, 256)
    a, b = torch.zeros(6, device=dev()), torch.zeros(6, device=dev())
    t = (inp["q"], inp["k"], inp["v"], inp["log_g"], inp["beta"])
    return {
        "chunk_backward": lambda s: list(gdn.chunk_backward(*t, do, want_dh0=True, stream=s)[0].values()),
        "norm_backward": lambda s: list(gdn.norm_backward(x, x, w, z=z, stream=s).values()),
        "norm_forward": lambda s: [y for y, kept in [gdn.norm_forward(x, w, z=z, ckpt=True, stream=s)] for y in (y, *kept.values())],
        "ckpt8_store": lambda s: list(gdn.ckpt8_store(x, stream=s)),
        "ckpt8_load": lambda s: [gdn.ckpt8_load(codes, exps, stream=s)],
        "chunk_prefill": lambda s: list(gdn.chunk_prefill(*t, stream=s)[:2]),
        "ba_gates": lambda s: [gdn.ba_gates(m, wt, a, b, 6, 3, stream=s)[0]],
    }


def workspace_bytes(name):
    if name == "chunk_backward":
        return gdn.gdn_backward_workspace_bytes(1, 200, 2, 6, 128, 128, 1, 1)
    if name == "norm_backward":
        return gdn.gdn_norm_workspace_bytes(300, 6, 128)
    if name == "chunk_prefill":
        return gdn.gdn_prefill_workspace_bytes(1, 200, 2, 6, 128, 128, 64, 1)
    return gdn.gdn_ba_gates_workspace_bytes(64, 12, 256) if name == "ba_gates" else 0


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["chunk_backward", "norm_backward", "norm_forward", "ckpt8_store", "ckpt8_load",
                                  "chunk_prefill", "ba_gates"])
def test_memory_of_another_stream(name, handle):
    say("another stream", name, handle)
    f = calls()[name]
    want = [t.clone() for t in f(None)]
    sizes = [t.numel() * t.element_size() for t in want] + [n for n in [workspace_bytes(name)] if n]
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    # the current stream has yet to write memory that the host has let go
    torch.cuda._sleep(SPIN)
    for n in sizes:
        torch.empty(n, dtype=torch.uint8, device=dev()).fill_(0xEE)
    got = f(s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del got, a
    # the side stream has yet to run the call when the current one takes memory
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    got = f(s)
    mine = [torch.empty(n, dtype=torch.uint8, device=dev()).fill_(0xEE) for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for t in mine:
        assert bool((t == 0xEE).all())


def test_the_default_streams_handle():
    say("handle 0")
    for name, f in calls().items():
        for a, b in zip(f(0), f(None)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
