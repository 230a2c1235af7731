"""A routing that the plan refuses ends the pass before anything reads through
the tables that the plan would have led to: those of the handle's last pass."""
import numpy as np
import pytest

import _harness as hz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", ["negative", "twice"])
@pytest.mark.parametrize("S", [0, 1])
@pytest.mark.parametrize("pair", [1, 2])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_a_refused_routing_after_a_longer_pass(mode, pair, S, bad):
    import torch
    from persistent_megakernel_sm_gb300 import MOE_E_DEVICE
    T, few = 3000, 40
    w, inp = hz.custom_case(T, 256, 16, 2, 128, S)
    dev = hz.upload(inp)
    layer = hz.make_layer(w, mode=mode, pair=pair, timeout_ns=200_000_000)
    want, routing = hz.run_layer(layer, w, dev)
    mats = (dev["w_gate"], dev["w_up"], dev["w_down"])
    idx, wt = torch.from_numpy(routing["idx"]).cuda(), torch.from_numpy(routing["w"]).cuda()
    no = idx[:few].clone()
    no[few - 1, 1] = -1 if bad == "negative" else no[few - 1, 0]
    out = torch.full((T, w.d), 7.0, dtype=torch.bfloat16, device="cuda")
    layer.forward_routed(dev["x"][:few], no, wt[:few], *mats, out)
    assert layer.status() == MOE_E_DEVICE
    assert bool((out == 7.0).all())
    layer.forward_routed(dev["x"], idx, wt, *mats, out)
    layer.check()
    assert np.array_equal(hz.from_dev_bf16(out), want)
    layer.close()
