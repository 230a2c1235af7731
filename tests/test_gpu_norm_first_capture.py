"""The first calls that a process makes of the norms' kernels, in a capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
from persistent_megakernel_sm_gb300 import MoEBlockNorm
T, d = 37, {d}
g = torch.Generator(device="cuda").manual_seed(1)
def rows(dtype):
    return torch.randn(T, d, generator=g, device="cuda").to(dtype)
bf, f32 = torch.bfloat16, torch.float32
n = MoEBlockNorm(d, pre="layer", post="layer", gate="channel")
n.reserve()
r, y, go, gn = rows(f32), rows(bf), rows(f32), rows(bf)
v = [torch.randn(d, generator=g, device="cuda") for _ in range(5)]
p = dict(zip(("pre_gain", "pre_shift", "post_gain", "post_shift", "gate"), v))
out, norm, gr, gy = (torch.zeros(T, d, dtype=k, device="cuda") for k in (f32, bf, f32, bf))
stats = torch.zeros(T, 4, device="cuda")
grads = {{"grad_" + k: torch.zeros(d, device="cuda") for k in p}}
every = [out, norm, stats, gr, gy, *grads.values()]
def step():
    n.forward(r, y, out, norm, **p, stats=stats)
    n.backward(go, gn, gr, gy, stats=stats, out=out, y=y, **p, **grads)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
assert all(not t.any() for t in every)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in every]
for t in every:
    t.zero_()
step()
torch.cuda.synchronize()
assert all(t.any() and torch.isfinite(t).all() for t in every)
assert all(torch.equal(a, b) for a, b in zip(got, every))
print("the same bits")
"""


@pytest.mark.parametrize("d", [4096, 16384, 77])
def test_a_process_may_begin_with_a_capture(d):
    """Wide rows take more shared memory than a kernel has unasked, which its first call asks for."""
    done = subprocess.run([sys.executable, "-c", PROGRAM.format(d=d)], cwd=REPO, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "the same bits" in done.stdout, done.stdout + done.stderr
