"""The routing gradient of long batches in every form, against its definition in
64 bits."""
import pytest

import _ops_ref as ref
from test_gpu_router import make, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("T,E,k", [(32768, 256, 8), (30011, 60, 6), (9001, 9, 3)])
def test_gradient_of_a_long_batch(T, E, k, score, renorm, bf16):
    """More rows than the grid holds at once."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + k)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits = logits.bfloat16() if bf16 else logits
    idx = logits.float().sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
    gw = torch.randn(T, k, generator=g, device="cuda")
    got = torch.full_like(logits, 77.0)
    make(settings(E, k, score, renorm=renorm, scale=2.5)).backward(logits, idx, gw, got)
    x, at, g64 = logits.double(), idx.long(), gw.double()
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    kept = s.gather(1, at)
    if renorm:
        a = kept / kept.sum(1, keepdim=True)
        slot, size = a * (g64 - (a * g64).sum(1, keepdim=True)), a * (g64.abs() + (a * g64.abs()).sum(1, keepdim=True))
    else:
        slot, size = kept * g64, kept * g64.abs()
    if score == "sigmoid":
        slot, size = slot * (1 - kept), size * (1 - kept)
    want = torch.zeros_like(x).scatter_(1, at, slot)
    mag = torch.zeros_like(x).scatter_(1, at, size)
    if score == "softmax" and not renorm:
        want, mag = want - s * slot.sum(1, keepdim=True), mag + s * size.sum(1, keepdim=True)
    # as for short batches: the weights' error twice and the sums over k slots
    spread = x.amax(1, keepdim=True) - x.amin(1, keepdim=True) + x.abs().amax(1, keepdim=True)
    tol = (2 * (24 + 2 * spread) + 2 * (k + 4)) * ref.U32 * 2.5 * mag + (ref.U16 if bf16 else ref.U32) * 2.5 * want.abs()
    assert bool(((got.double() - 2.5 * want).abs() <= tol + 2.0 ** -126).all())
