"""The first call of a process may be a captured one, at every head size, with a
bias of a short and of a wide reach and without one."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys, numpy as np, torch
import transformer_encoder_forward_gb300 as te
hd, reach = int(sys.argv[1]), int(sys.argv[2])
torch.manual_seed(1)
rows, nq = 1300, 3
cu = np.array([0, 1200, 1300], np.int32)
cu_dev = torch.from_numpy(cu).cuda()
qkv = torch.randn(rows, 3 * nq * hd, device="cuda").bfloat16()
out = torch.zeros(rows, nq * hd, dtype=torch.bfloat16, device="cuda")
plan = te.relpos_plan(64, reach) if reach else None
table = torch.randn(64, nq, device="cuda")
def call():
    if reach:
        te.attn_relbias_fwd(qkv, 3 * nq * hd, 0, nq * hd, 2 * nq * hd, cu, cu_dev, nq, nq, hd, -1, -1, 0, hd ** -0.5, plan,
                            table, out, nq * hd)
    else:
        te.attn_sink_fwd(qkv, 3 * nq * hd, 0, nq * hd, 2 * nq * hd, cu, cu_dev, nq, nq, hd, 100, 0, 4, hd ** -0.5, out,
                         nq * hd)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
got = out.clone()
out.zero_()
call()
torch.cuda.synchronize()
te.check()
assert bool((got != 0).any()) and torch.equal(got, out)
print("same")
"""


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("reach", [0, 128, 2048])
def test_the_first_call_of_a_process_is_captured(hd, reach):
    r = subprocess.run([sys.executable, "-c", SCRIPT, str(hd), str(reach)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
