"""GPU tests of the memory that an AdamW table steps on."""
import pytest
import torch

import linear_attention_ssm_gated_amd as gdn
from gpu_common import dev, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_that_get_other_memory(bits):
    # the table goes on with the memory it was built on, which nobody else gets meanwhile
    say("adamw, other memory", bits)
    n = 3 << 20
    w, g = torch.ones(n, device=dev()), torch.ones(n, device=dev())
    table = gdn.adamw_table([w], [g], bits=bits)
    states = [t for k in table.states.values() for t in k]
    old = [t.data_ptr() for t in (w, g, *states)]
    for t in (w, g, *states):
        t.data = torch.zeros_like(t)
    others = [torch.full((n * size,), 7, dtype=torch.uint8, device=dev()) for size in (4, 4, 4, 4, 1, 1) for _ in range(2)]
    assert not {t.data_ptr() for t in others} & set(old)
    gdn.gdn_adamw_step(table, 1e-2, 0.9, 0.999, 1e-8, 1)
    torch.cuda.synchronize()
    for t in others:
        assert bool((t == 7).all())
    for t in (w, g, *states):
        assert not bool(t.view(torch.uint8).any())
    table.set_grads([torch.ones(n, device=dev())])
    gdn.gdn_adamw_step(table, 1e-2, 0.9, 0.999, 1e-8, 2)
    torch.cuda.synchronize()
    assert not bool(w.any())
