"""Several router tiles to a CTA, one after another, in the static mode (whose
CTAs take tiles round-robin): each tile's token masks are read to the end before
the next tile's are begun."""
import numpy as np
import pytest

import _harness as hz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("pair", [1, 2])
@pytest.mark.parametrize("route_tokens,T,k", [(64, 1000, 2), (128, 3000, 8)])
def test_static_mode_with_many_router_tiles_a_cta(route_tokens, T, k, pair, given):
    import torch
    w, inp = hz.custom_case(T, 128, 64, k, 128, 0)
    dev = hz.upload(inp)
    layer = hz.make_layer(w, mode=0, pair=pair, route_tokens=route_tokens, route_splits=1)
    want, routing = hz.run_layer(layer, w, dev)          # the persistent mode
    idx, wt = torch.from_numpy(routing["idx"]).cuda(), torch.from_numpy(routing["w"]).cuda()
    layer.set_option("mode", 2)
    layer.set_option("grid_ctas", 2 * pair)              # two workers for all tiles
    for _ in range(20):
        if given:
            out = torch.empty(T, w.d, dtype=torch.bfloat16, device="cuda")
            layer.forward_routed(dev["x"], idx, wt, dev["w_gate"], dev["w_up"], dev["w_down"], out)
            layer.check()
            got = {key: torch.empty_like(torch.from_numpy(routing[key])).cuda() for key in ("counts", "perm", "pos")}
            layer.get_routing(**got)
            torch.cuda.synchronize()
            got, bits = {key: v.cpu().numpy() for key, v in got.items()}, hz.from_dev_bf16(out)
        else:
            bits, got = hz.run_layer(layer, w, dev)
        for key in ("counts", "perm", "pos"):
            assert np.array_equal(got[key], routing[key]), key
        assert np.array_equal(bits, want)
    layer.close()
