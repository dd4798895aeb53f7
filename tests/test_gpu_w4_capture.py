"""The first call of a process is one that is captured into a graph."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import rank_binary_factorization_b200 as nq
from w4_common import acts, layer, stack
_, (q, s, z) = layer(300, 1024, 64, True, 1)
GU = stack(4, 2 * 96, 128, 64, True, 2)[1]
DN = stack(4, 128, 96, 64, True, 3)[1]
W = acts(64, 256, torch.float32, 4).cuda()
X = {{b: acts(b, 1024, torch.bfloat16, b).cuda() for b in (1, 100)}}
T = acts(3, 128, torch.bfloat16, 5).cuda()
R = acts(4, 128, torch.bfloat16, 6).cuda()
calls = dict(
    few=lambda: nq.nq_w4_matmul(q, s, X[1], group=64, zeros=z),
    many=lambda: nq.nq_w4_matmul(q, s, X[100], group=64, zeros=z),
    moe=lambda: nq.nq_moe_w4(T, R, GU[0], GU[1], DN[0], DN[1], 2, group=64, gate_up_zeros=GU[2],
                             down_zeros=DN[2]),
    quantize=lambda: nq.nq_w4_quantize(W, group=32, grid=4)["packed"],
    dequantize=lambda: nq.nq_w4_dequantize(q, s, 1024, 64, z),
)
torch.cuda.synchronize()
call = calls[{what!r}]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, call())
"""


@pytest.mark.parametrize("what", ["few", "many", "moe", "quantize", "dequantize"])
def test_first_call_in_a_capture(what):
    run = subprocess.run([sys.executable, "-c", SETUP.format(root=ROOT, what=what)], capture_output=True,
                         text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
