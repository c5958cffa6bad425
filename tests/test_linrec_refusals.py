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
