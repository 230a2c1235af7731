"""A workspace reserved again: what the last pass left in the old one is gone."""
import numpy as np
import pytest

import _harness as hz

pytestmark = pytest.mark.gpu


def test_status_and_routing_between_reserve_and_the_next_pass():
    import torch
    from persistent_megakernel_sm_gb300 import MOE_E_STATE, MOE_OK, MoEError
    w, inp = hz.named_case("tiny")
    dev = hz.upload(inp)
    layer = hz.make_layer(w)
    want, routing = hz.run_layer(layer, w, dev)
    layer.reserve(4 * w.T)
    assert layer.status() == MOE_OK
    idx = torch.full((w.T, w.k), 7, dtype=torch.int32, device="cuda")
    with pytest.raises(MoEError) as e:
        layer.get_routing(idx=idx)
    assert e.value.code == MOE_E_STATE
    got, again = hz.run_layer(layer, w, dev)
    assert np.array_equal(got, want)
    assert np.array_equal(again["idx"], routing["idx"])
    layer.close()
