"""The norms about a block without rows: whatever has a row a token is an empty tensor, whose pointer is null."""
import pytest

from test_gpu_norm import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("save", [False, True])
def test_no_rows(gate, save):
    import torch
    c = Case(0, 96, "layer", "layer", gate)
    n = c.make()
    n.reserve()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    e, st = torch.empty(0, 96, **bf), torch.empty(0, 4, device="cuda")
    p = c.params()
    held = (torch.empty(0, 96, dtype=torch.int8, device="cuda"), torch.empty(0, 1, **bf)) if save else None
    n.forward(e, e, e, e, **p, stats=st, out8=held, y8=held)
    grads = {k: torch.full((96,), 9.0, device="cuda") for k in ("grad_pre_gain", "grad_pre_shift", "grad_post_gain",
                                                                "grad_post_shift")}
    own = dict(none={}, channel=dict(grad_gate=torch.full((96,), 9.0, device="cuda")),
               token=dict(grad_gate=torch.empty(0, device="cuda")), element=dict(grad_gate=e))[gate]
    n.backward(e, e, e, e, stats=st, out=held if save else e, y=held if save else e, **p, **grads, **own)
    assert all(torch.all(t == 0) for t in (*grads.values(), *own.values()))
