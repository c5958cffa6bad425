"""Host-side checks of the linear recurrence's calls, no GPU needed: outputs at an
input's address, and sizes that 32 bits do not hold."""
import os

import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
from test_linrec_abi import S


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn.so is not built (run __graft_entry__.build())")
    return gdn.linrec._lib()


@pytest.mark.parametrize("kw", [dict(y=0x2000), dict(y=0x3000), dict(y=0x1000), dict(y=0x2000, ys=80), dict(y=0x3000, gate=0)])
def test_step_refuses_its_inputs_as_output(lib, kw):
    # (refused ahead of any launch, on a machine with a GPU too)
    a = dict(h=0x1000, x=0x2000, l=0x3000, y=0x4000, B=2, D=64, xs=64, as_=64, ys=64, scale=0, io=1, gate=1, stream=None)
    a.update(kw)
    assert lib.gdn_linrec_step(*a.values()) == S["GDN_ERR_SHAPE"], gdn.last_route()
    assert "share memory" in gdn.last_route()


def test_sizes_past_32_bits_are_refused():
    # as the C call's ints they would wrap to a short call, and leave the other rows unwritten
    n = (1 << 32) + 1000
    for B, T, D in ((1, n, 1), (n, 1, 1), (1, 1, n), (1, 1 << 31, 1)):
        with pytest.raises(ValueError, match="32 bits"):
            gdn.gdn_linrec_workspace_bytes(B, T, D)
    x = torch.zeros(1, 1)
    with pytest.raises(ValueError, match="32 bits"):
        gdn.linrec_forward(x.expand(1, n, 1), x.expand(1, n, 1))
    with pytest.raises(ValueError, match="32 bits"):
        gdn.linrec_forward(x.expand(n, 1), x.expand(n, 1), cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="32 bits"):
        gdn.linrec_backward(*[x.expand(1, n, 1)] * 4)
    with pytest.raises(ValueError, match="32 bits"):
        gdn.linrec_step(torch.zeros(1, dtype=torch.int64).expand(n), x.expand(n, 1), x.expand(n, 1))
    a = [x.expand(n, 1)] * 2
    with pytest.raises(ValueError, match="32 bits"):
        gdn.gdn_linrec_forward(*a, None, a[0], None, 1, n, 1, 1, 1, 1)
    with pytest.raises(ValueError, match="32 bits"):
        gdn.gdn_linrec_backward(None, a[0], a[0], None, a[0], None, a[0], a[0], None, 1, n, 1, 1, 1, 1, 1, 1, 1)
    with pytest.raises(ValueError, match="32 bits"):
        gdn.gdn_linrec_step(torch.zeros(1, dtype=torch.int64), a[0], a[0], a[0], n, 1, 1, 1, 1)
