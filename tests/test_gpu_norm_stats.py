"""The norms' gradient without stats, where no norm is passed through."""
import pytest

from test_gpu_norm import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,pad", [(264, 0), (77, 3)])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("res", ["bfloat16", "float32"])
def test_the_residuals_gradient_alone_needs_no_stats(d, pad, post, res):
    """Nothing but the residual's gradient is wanted and none comes through the pre norm: it is grad_out."""
    import torch
    c = Case(9, d, "rms", post, "token", res=res, pad=pad)
    n, p = c.make(), c.params()
    go = torch.randn(9, d + pad, device="cuda").to(getattr(torch, res))[:, :d]
    gr = torch.full_like(go, 9.0)
    n.backward(go, None, gr, None, **p)
    assert torch.equal(gr, go)


def test_gradients_through_the_post_norm_need_stats():
    import torch
    from persistent_megakernel_sm_gb300 import MOE_E_INVAL, MoEError
    c = Case(9, 64, "rms", "rms", "token")
    n, p = c.make(), c.params()
    n.reserve()
    t = torch.zeros(9, 64, dtype=torch.bfloat16, device="cuda")
    for how in (dict(grad_post_gain=torch.empty(64, device="cuda")), dict(grad_gate=torch.empty(9, device="cuda"))):
        with pytest.raises(MoEError) as err:
            n.backward(t, None, torch.empty_like(t), None, y=t, **p, **how)
        assert err.value.code == MOE_E_INVAL
    with pytest.raises(MoEError) as err:
        n.backward(t, None, None, torch.empty_like(t), y=t, **p)
    assert err.value.code == MOE_E_INVAL
