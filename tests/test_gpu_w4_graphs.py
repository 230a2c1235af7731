"""A decode step in one captured graph: copies, counts, routing and the 4-bit
experts' kernels, each of which may start before the one in front has ended."""
import numpy as np
import pytest

import _ops_ref as ref
from test_gpu_w4 import Case, dev, dev_bf16, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 13, 60])
def test_a_step_with_copies_and_forks_in_one_graph(T):
    """x and the logits come in by copies inside the graph; the routing runs on a
    forked stream and joins; two layers follow one another, the second one's x
    the first one's output."""
    import torch
    from persistent_megakernel_sm_gb300 import MoERouter
    a, b = (Case(T, 256, 8, 2, 256, S, 64, True, seed=T + S) for S in (0, 1))
    la, lb = a.layer(), b.layer()
    router = MoERouter(8, 2)
    x_in, l_in = torch.empty(T, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(T, 8, device="cuda")
    x, l = torch.empty_like(x_in), torch.empty_like(l_in)
    idx, w = torch.empty(T, 2, dtype=torch.int32, device="cuda"), torch.empty(T, 2, device="cuda")
    counts = torch.empty(8, dtype=torch.int32, device="cuda")
    mid, out = torch.empty_like(x), torch.empty_like(x)
    last = torch.empty_like(x)

    def step(fork):
        x.copy_(x_in)
        here = torch.cuda.current_stream()
        fork.wait_stream(here)
        with torch.cuda.stream(fork):
            l.copy_(l_in)
            router.forward(l, idx, w, counts=counts)
        here.wait_stream(fork)
        la.forward(x, idx, w, mid)
        lb.forward(mid, idx, w, out)
        last.copy_(out)

    side, fork = torch.cuda.Stream(), torch.cuda.Stream()
    rng = np.random.default_rng(T)
    inputs = [(dev_bf16(rng.standard_normal((T, 256))), dev(rng.standard_normal((T, 8)).astype(np.float32)))
              for _ in range(3)]
    wants = []
    for xi, li in inputs:
        x_in.copy_(xi), l_in.copy_(li)
        step(fork)
        torch.cuda.synchronize()
        assert int(counts.sum()) == 2 * T
        wants.append(last.clone())
        want, off = ref.experts(host(mid), idx.cpu().numpy(), w.cpu().numpy().astype(np.float64), b.gate, b.up, b.down,
                                8, 1)
        assert np.all(np.abs(host(last) - want) <= off)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(fork)
    for (xi, li), want in [*zip(inputs, wants)] * 2:
        x_in.copy_(xi), l_in.copy_(li)
        last.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(last, want)
    la.check(), lb.check()


def test_a_graph_sees_weights_set_again_in_the_same_place():
    """set_weights copies scales and zero points to where the captured pass reads
    them; the codes are read where they were."""
    import torch
    c = Case(5, 256, 4, 2, 256, 0, 32, True, seed=3)
    layer = c.layer()
    x, idx, w = dev_bf16(c.x), dev(c.idx), dev(c.w)
    out = torch.empty(5, 256, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            layer.forward(x, idx, w, out)
    g.replay()
    torch.cuda.synchronize()
    c.check(host(out))
    other = Case(5, 256, 4, 2, 256, 0, 32, True, seed=4)
    for (codes, scales, zeros), m in zip(c.dev, (other.gate, other.up, other.down)):
        codes.copy_(dev(m[0])), scales.copy_(dev_bf16(m[1])), zeros.copy_(dev(m[2]))
    layer.set_weights(*c.dev)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    c.gate, c.up, c.down = other.gate, other.up, other.down
    c.check(host(out))
