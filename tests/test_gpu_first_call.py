"""The first call of an operator in a process may be one that a graph captures."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
import torch
import bit_diffusion_transformer_nvfp4_b200 as w4
g = torch.Generator(device="cuda")
g.manual_seed(1)
def normal(*shape):
    return torch.randn(*shape, device="cuda", generator=g).bfloat16()
x, r, k, codes, scales = normal(300, 256), normal(300, 256), normal(77, 256), None, None
w = w4.PackedWeightFp8(torch.full((512, 256), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(512, device="cuda"))
if sys.argv[1] == "after W4A4":
    w4.linear(x, w4.pack_weight(normal(256, 256)))
torch.cuda.synchronize()
def call():
    a, h = w4.rms_norm_fp8(x, residual=r)
    return [a.codes, a.scales, h, w4.linear_fp8(a, w), w4.cross_attention(x, k, k, heads=4),
            w4.cross_attention(x[:2], k, k, heads=4)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(out, call()):
    assert torch.equal(a, b)
assert w4.w4a4_device_status() == 0
print("ok")
"""


@pytest.mark.parametrize("state", ["after W4A4", "first of all"])
def test_first_call_under_capture(state):
    run = subprocess.run([sys.executable, "-c", PROGRAM, state], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout == "ok\n", run.stdout + run.stderr
