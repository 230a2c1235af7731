"""The router's result for a batch with masked and padding rows, in the bf16
layer and in the 4-bit experts."""
import numpy as np
import pytest

import _harness as hz
import _ops_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [0, 1])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_slots_without_an_expert_as_weights_of_zero(mode, S):
    """Rows masked out altogether and rows with fewer than k experts left: the
    layer takes them once each empty slot names another expert with weight 0."""
    import torch
    from persistent_megakernel_sm_gb300 import MoERouter
    T, d, E, k, f = 70, 256, 16, 4, 256
    w, inp = hz.custom_case(T, d, E, k, f, S)
    dev = hz.upload(inp)
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[60:] = -np.inf                                # padding
    logits[7] = -np.inf
    logits[7, [3, 9]] = [0.5, 0.25]                      # two experts are left
    idx, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    MoERouter(E, k).forward(torch.from_numpy(logits).cuda(), idx, wt)
    torch.cuda.synchronize()
    want_idx, want_w = ref.route(logits, dict(E=E, k=k, score="softmax", groups=1, groups_kept=1, group_score="max",
                                              renormalise=True, scale=1.0))
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    # the experts in ascending order, those that the row has chosen last: as
    # many of the others as there are slots to fill, on the device
    taken = torch.zeros(T, E + 1, device="cuda").scatter_(1, torch.where(idx < 0, E, idx).long(), 1.0)[:, :E]
    others = taken.sort(dim=1, stable=True).indices[:, :k].to(torch.int32)
    filled = torch.where(idx < 0, others, idx)
    layer = hz.make_layer(w, mode=mode)
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    layer.forward_routed(dev["x"], filled, wt, dev["w_gate"], dev["w_up"], dev["w_down"], out)
    layer.check()
    layer.close()
    got = hz.bf16_to_f64(hz.from_dev_bf16(out))
    x, g, u, dn = (hz.bf16_to_f64(inp[n]) for n in ("x", "w_gate", "w_up", "w_down"))
    want = np.zeros((T, d))
    for t in range(T):
        slots = [(e, v) for e, v in zip(want_idx[t], want_w[t]) if e >= 0]
        for e, v in slots + [(E, 1.0)] * S:
            z = g[e] @ x[t]
            want[t] += v * (dn[e] @ ref.bf16(z / (1 + np.exp(-z)) * (u[e] @ x[t])))
    assert np.all(np.abs(got - want) <= hz.ATOL + hz.RTOL * np.abs(want))
    assert S or np.all(got[60:] == 0)
