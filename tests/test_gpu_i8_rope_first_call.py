"""The first call of a process may be a captured one: no kernel choice of the
8-bit and rotation entry points needs an eager call before.  And the binding
holds the leading dimensions it is given to the tensors'."""
import os
import subprocess
import sys

import pytest

import transformer_encoder_forward_gb300 as te

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys, torch
import transformer_encoder_forward_gb300 as te
what = sys.argv[1]
torch.manual_seed(1)
m, k, n = {"small": (5, 512, 96), "mid": (60, 768, 256), "resident": (2000, 512, 128), "large": (2000, 1024, 256),
           "gated": (2000, 1024, 256), "quant": (300, 512, 32), "norm": (300, 3840, 32), "rope": (300, 512, 256),
           "rope_odd": (300, 512, 256)}[what]
i8 = lambda *s: torch.randint(-127, 128, s, dtype=torch.int8, device="cuda")
x, xs, w, sw = i8(m, k), torch.rand(m, device="cuda"), i8(2, n, k), torch.rand(2, n, device="cuda")
qw = [te.q8w(w[i], sw[i]) for i in range(2)]
ws = torch.empty(te.i8_workspace(m, k, 2 * n) + 256, dtype=torch.uint8, device="cuda")
y = torch.zeros(m, n, device="cuda")
out = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
v, one = torch.randn(m, k, device="cuda"), torch.ones(k, device="cuda")
q, s = torch.zeros(m, k, dtype=torch.int8, device="cuda"), torch.zeros(m, device="cuda")
plan = te.rope_axes_plan(64, (16, 24, 24) if what == "rope" else (22, 22, 20))
pos = torch.randint(0, 99, (m, 3), dtype=torch.int32, device="cuda")
r = torch.zeros(m, k, device="cuda")
def call():
    if what in ("small", "mid", "resident", "large"):
        te.i8_linear(x, xs, [dict(w=qw[0], y=y, ldy=n)], ws)
    elif what == "gated":
        te.i8_gated_linear(x, xs, qw[0], qw[1], 1, out, ws)
    elif what == "quant":
        te.quant_rows(v, q, s)
    elif what == "norm":
        te.rownorm_quant(v, one, None, 0, 1e-6, q, s)
    else:
        te.qk_rope_axes(v, k, r, k, 0, k // 2, 4, 4, 64, None, None, 1e-6, plan, pos, 1.0, m)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
outs = (y, out, q, s, r)
graph.replay()
got = [t.clone() for t in outs]
for t in outs:
    t.zero_()
call()
torch.cuda.synchronize()
te.check()
assert any(bool((t != 0).any()) for t in outs)
assert all(bool((a == b).all()) for a, b in zip(got, outs))
print("same")
"""


@pytest.mark.parametrize("what", ["small", "mid", "resident", "large", "gated", "quant", "norm", "rope", "rope_odd"])
def test_the_first_call_of_a_process_is_captured(what):
    r = subprocess.run([sys.executable, "-c", SCRIPT, what], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


def test_leading_dimensions_are_those_of_the_tensors():
    import torch
    x = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(4, device="cuda")
    w, sw = torch.zeros(32, 64, dtype=torch.int8, device="cuda"), torch.zeros(32, device="cuda")
    qw = te.q8w(w, sw)
    y = torch.zeros(4, 64, device="cuda")
    te.i8_linear(x, s, [dict(w=qw, y=y[:, :32], ldy=64)], None)
    with pytest.raises(ValueError):
        te.i8_linear(x, s, [dict(w=qw, y=y[:, :32], ldy=128)], None)
    with pytest.raises(ValueError):
        te.i8_linear(x, s, [dict(w=qw, y=y[:, :32], ldy=64, residual=y[:, 32:], ldr=96)], None)
    with pytest.raises(ValueError):                          # a residual of fewer features
        te.i8_linear(x, s, [dict(w=qw, y=y[:, :32], ldy=64, residual=y[:, 32:48], ldr=64)], None)
    te.i8_linear(x[:1], s[:1], [dict(w=qw, y=y[:1, :32], ldy=32)], None)     # one row: any stride
    plan = te.rope_axes_plan(32, (16, 16))
    pos = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    rope = lambda src, lds, off=0, nq=1, nkv=1: te.qk_rope_axes(src, lds, src, lds, off, off + 32, nq, nkv, 32, None, None,
                                                                1e-6, plan, pos, 1.0, 4)
    rope(y, 64)
    rope(y[:, :32], 64, nkv=0)
    with pytest.raises(ValueError):
        rope(y, 128)
    with pytest.raises(ValueError):
        rope(y, 64, off=32)
    with pytest.raises(ValueError):
        rope(y[:, :32], 64)
    te.check()


def test_an_empty_batch_is_no_error():
    import torch
    z = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")
    w, sw = torch.zeros(32, 64, dtype=torch.int8, device="cuda"), torch.zeros(32, device="cuda")
    qw = te.q8w(w, sw)
    x, xs, y = z(0, 64, t=torch.int8), z(0), z(0, 32)
    te.quant_rows(z(0, 64), x, xs)
    te.rownorm_quant(z(0, 64), z(64), None, 0, 1e-6, x, xs)
    te.i8_linear(x, xs, [dict(w=qw, y=y, ldy=32)], None)
    te.i8_gated_linear(x, xs, qw, qw, 1, z(0, 32, t=torch.bfloat16), None)
    plan = te.rope_axes_plan(32, (16, 16))
    te.qk_rope_axes(z(0, 64), 64, z(0, 64), 64, 0, 32, 1, 1, 32, None, None, 1e-6, plan, z(0, 2, t=torch.int32), 1.0, 0)
    te.check()
