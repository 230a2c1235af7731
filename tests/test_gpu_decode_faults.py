"""The layer for a few tokens when a wait inside its kernel runs out: one block is told not to arrive, the limit is short, the
kernel returns by itself.  The status says so, passes until it is asked for do nothing, and the one after it is right."""
import numpy as np
import pytest

from persistent_megakernel_sm_gb300 import MOE_E_TIMEOUT, MOE_OK, MoEError
from test_gpu_decode import Case, dev

pytestmark = pytest.mark.gpu

NONE, LOGITS, H = -1, 0, 1


@pytest.mark.parametrize("shape", [(3, 256, 24, 4, 512, 1), (12, 1024, 8, 2, 1408, 0)])
@pytest.mark.parametrize("routed,drop", [(False, LOGITS), (False, H), (True, H)])
def test_a_wait_that_runs_out(shape, routed, drop):
    import torch
    c = Case(*shape, bias=True)
    T, d, _, k = shape[:4]
    n, weights = c.make(), c.weights()
    x, router, bias, given, given_w = dev(c.x), dev(c.router), dev(c.bias, "float32"), dev(c.idx), dev(c.w, "float32")
    out, idx, w = torch.empty_like(x), torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")

    def run():
        for t in (out, idx, w):
            t.fill_(5)
        if routed:
            n.forward_routed(x, given, given_w, *weights, out)
        else:
            n.forward(x, router, *weights, out, bias=bias, idx=idx, w=w)

    run()
    n.check()
    want = [t.clone() for t in (out, idx, w)]
    n.set_option("timeout_ns", 50_000_000)
    n.set_option("fault_drop_task", drop)
    run()
    n.set_option("fault_drop_task", NONE)
    for _ in range(2):  # these would be let through their waits early
        run()
        assert all(torch.all(t == 5) for t in (out, idx, w))
    assert n.status() == MOE_E_TIMEOUT
    assert n.status() == MOE_OK
    for _ in range(3):
        run()
        assert n.status() == MOE_OK
        assert all(torch.equal(a, b) for a, b in zip(want, (out, idx, w)))
    n.set_option("fault_drop_task", drop)
    run()
    with pytest.raises(MoEError) as err:
        n.check()
    assert err.value.code == MOE_E_TIMEOUT
    n.set_option("fault_drop_task", NONE)
    n.reserve(T)
    run()
    n.check()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, idx, w)))


def test_a_given_routing_has_no_wait_for_logits():
    c = Case(3, 256, 24, 4, 512, 1)
    n, weights = c.make(), c.weights()
    want = c.routed(n, weights)
    n.set_option("fault_drop_task", LOGITS)
    assert np.array_equal(c.routed(n, weights), want)
