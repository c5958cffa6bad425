"""Host-side checks of the AdamW step's derived scalars, no GPU needed: what the
arguments give in fp32 has to be finite, not the arguments alone."""
import os

import pytest

import linear_attention_ssm_gated_amd as gdn
from test_adamw_abi import S, X, entry, plan


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn.so is not built (run __graft_entry__.build())")
    return gdn.adamw._lib()


@pytest.mark.parametrize("kw,status", [
    (dict(lr=1e38, b1=0.9, step=1), "GDN_ERR_SHAPE"), (dict(lr=-1e38, b1=0.9, step=1), "GDN_ERR_SHAPE"),   # lr / 0.1
    (dict(lr=1e38, b1=0.9, step=1000), "GDN_OK"), (dict(lr=3e37, b1=0.9, step=1), "GDN_OK"),
    (dict(lr=1e31, b1=1 - 1e-8, step=1), "GDN_ERR_SHAPE"), (dict(lr=1e38, b1=0.9, step=1, control=X), "GDN_OK"),
])
def test_rates(lib, kw, status):
    assert plan(lib, [entry(weight_decay=0.0)], **kw) == S[status], gdn.last_route()
    assert plan(lib, [entry(weight_decay=0.0, m_scale=X, v_scale=X)], s=2, **kw) == S[status], gdn.last_route()


@pytest.mark.parametrize("wd,lr,status", [
    (1e30, 1e9, "GDN_ERR_SHAPE"), (1e30, -1e9, "GDN_ERR_SHAPE"), (1e30, 1e8, "GDN_OK"), (3e38, 1.0, "GDN_OK"), (3e38, 2.0, "GDN_ERR_SHAPE"),
])
def test_decays(lib, wd, lr, status):
    # the second of two tensors; a control's lr is not known here; a tensor without values is not touched
    assert plan(lib, [entry(), entry(weight_decay=wd)], lr=lr) == S[status], gdn.last_route()
    assert plan(lib, [entry(), entry(weight_decay=wd)], lr=lr, control=X) == 0
    assert plan(lib, [entry(), entry(weight_decay=wd, n=0)], lr=lr) == 0
