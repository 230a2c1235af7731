"""moe_layer_forward_routed: the layer on a routing that the caller gives."""
import numpy as np
import pytest

import _harness as hz
import _ops_ref as ref

pytestmark = pytest.mark.gpu

CASES = {
    # T, d, E, k, f, S, router-bias std, options
    "small": (64, 256, 8, 2, 512, 0, 0.3, {}),
    "shared_ragged": (300, 384, 16, 3, 256, 1, 0.6, {"tokens_per_tile": 64}),
    "many_experts": (257, 256, 128, 8, 128, 0, 0.0, {}),
    "one_token": (1, 256, 8, 2, 256, 0, 0.0, {}),
    "top16_small_tiles": (40, 128, 32, 16, 128, 1, 0.0, {"route_tokens": 64}),
}


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("pair", [1, 2])
@pytest.mark.parametrize("name", list(CASES))
def test_the_layers_own_routing_gives_the_same_bits(name, pair, mode):
    import torch
    T, d, E, k, f, S, b, opts = CASES[name]
    w, inp = hz.custom_case(T, d, E, k, f, S, b)
    dev = hz.upload(inp)
    layer = hz.make_layer(w, mode=mode, pair=pair, **opts)
    want, routing = hz.run_layer(layer, w, dev)
    idx, wt = torch.from_numpy(routing["idx"]).cuda(), torch.from_numpy(routing["w"]).cuda()
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    layer.set_router_bias(None)
    layer.forward_routed(dev["x"], idx, wt, dev["w_gate"], dev["w_up"], dev["w_down"], out)
    layer.check()
    assert np.array_equal(hz.from_dev_bf16(out), want)
    # the routing read back is the given one, the plan's tables those of the layer
    back = {"idx": torch.empty_like(idx), "w": torch.empty_like(wt),
            "counts": torch.empty(E, dtype=torch.int32, device="cuda"),
            "perm": torch.empty(T * k, dtype=torch.int32, device="cuda"),
            "pos": torch.empty(T, k, dtype=torch.int32, device="cuda")}
    layer.get_routing(**back)
    torch.cuda.synchronize()
    for key, v in back.items():
        assert np.array_equal(v.cpu().numpy(), routing[key]), key
    # and the layer's own router still runs on the same handle
    again, _ = hz.run_layer(layer, w, dev)
    assert np.array_equal(again, want)
    layer.close()


def test_grouped_sigmoid_router_into_the_layer():
    """A router that the layer does not have: sigmoid scores, a balance bias,
    groups, scaled weights; against the definition in 64 bits."""
    import torch
    from persistent_megakernel_sm_gb300 import MoERouter
    T, d, E, k, f, S = 70, 256, 32, 4, 256, 1
    w, inp = hz.custom_case(T, d, E, k, f, S)
    dev = hz.upload(inp)
    rng = np.random.default_rng(2)
    r = dict(E=E, k=k, score="sigmoid", groups=4, groups_kept=2, group_score="top2", renormalise=True, scale=2.5)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32).astype(np.float64)
    logits = ref.clear_logits(rng, T, r, bias)
    idx, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    MoERouter(**r).forward(torch.from_numpy(logits.astype(np.float32)).cuda(), idx, wt,
                           bias=torch.from_numpy(bias.astype(np.float32)).cuda())
    layer = hz.make_layer(w)
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    layer.forward_routed(dev["x"], idx, wt, dev["w_gate"], dev["w_up"], dev["w_down"], out)
    layer.check()
    layer.close()
    want_idx, want_w = ref.route(logits, r, bias)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    x, g, u, dn = (hz.bf16_to_f64(inp[n]) for n in ("x", "w_gate", "w_up", "w_down"))
    want = np.zeros((T, d))
    for t in range(T):
        for e, v in [*zip(want_idx[t], want_w[t]), (E, 1.0)]:
            z = g[e] @ x[t]
            want[t] += v * (dn[e] @ ref.bf16(z / (1 + np.exp(-z)) * (u[e] @ x[t])))
    got = hz.bf16_to_f64(hz.from_dev_bf16(out))
    assert np.all(np.abs(got - want) <= hz.ATOL + hz.RTOL * np.abs(want))


@pytest.mark.parametrize("bad", ["outside", "negative", "twice"])
def test_a_routing_that_is_not_one_is_reported(bad):
    import torch
    T, d, E, k, f, S, b, _ = CASES["small"]
    w, inp = hz.custom_case(T, d, E, k, f, S, b)
    dev = hz.upload(inp)
    layer = hz.make_layer(w, timeout_ns=50_000_000)
    want, routing = hz.run_layer(layer, w, dev)
    idx = routing["idx"].copy()
    if bad == "outside":
        idx[17, 1] = E
    elif bad == "negative":
        idx[0, 0] = -1
    else:
        idx[63] = 5
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    wt = torch.from_numpy(routing["w"]).cuda()
    layer.forward_routed(dev["x"], torch.from_numpy(idx).cuda(), wt, dev["w_gate"], dev["w_up"], dev["w_down"], out)
    from persistent_megakernel_sm_gb300 import MOE_E_DEVICE
    assert layer.status() == MOE_E_DEVICE
    # the handle is usable afterwards
    layer.forward_routed(dev["x"], torch.from_numpy(routing["idx"]).cuda(), wt, dev["w_gate"], dev["w_up"],
                         dev["w_down"], out)
    layer.check()
    assert np.array_equal(hz.from_dev_bf16(out), want)
    layer.close()


def test_no_tokens_and_a_graph():
    import torch
    T, d, E, k, f, S, b, _ = CASES["small"]
    w, inp = hz.custom_case(T, d, E, k, f, S, b)
    dev = hz.upload(inp)
    layer = hz.make_layer(w)
    want, routing = hz.run_layer(layer, w, dev)
    idx, wt = torch.from_numpy(routing["idx"]).cuda(), torch.from_numpy(routing["w"]).cuda()
    out = torch.full((T, d), 3.0, dtype=torch.bfloat16, device="cuda")
    mats = (dev["w_gate"], dev["w_up"], dev["w_down"])
    layer.forward_routed(dev["x"][:0], idx[:0], wt[:0], *mats, out)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer.forward_routed(dev["x"], idx, wt, *mats, out)
    for _ in range(2):
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(hz.from_dev_bf16(out), want)
    layer.close()
