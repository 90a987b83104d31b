"""A call may be its thread's first of CUDA: the entry points that describe their
operands to the TMA unit through a driver call need no context set up before."""
import os
import subprocess
import sys

import pytest

import transformer_encoder_forward_gb300 as te  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys, threading, torch
import numpy as np
import transformer_encoder_forward_gb300 as te
what = sys.argv[1]
torch.manual_seed(3)
m, k, n = {"mid": (60, 768, 256), "resident": (2000, 512, 128)}.get(what, (300, 1024, 256))
i8 = lambda *s: torch.randint(-127, 128, s, dtype=torch.int8, device="cuda")
x, xs, w, sw = i8(m, k), torch.rand(m, device="cuda"), i8(2, n, k), torch.rand(2, n, device="cuda")
xb = torch.randn(m, k, device="cuda").bfloat16()
qw = [te.q8w(w[i], sw[i]) for i in range(2)]
ws = torch.empty(te.i8_workspace(m, k, 2 * n) + 256, dtype=torch.uint8, device="cuda")
y = torch.zeros(m, n, device="cuda")
out = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
qkv = torch.randn(m, 3 * 128, device="cuda").bfloat16()
o = torch.zeros(m, 128, dtype=torch.bfloat16, device="cuda")
cu = np.array([0, m], dtype=np.int32)
cu_dev = torch.from_numpy(cu).cuda()
stream = torch.cuda.current_stream()
def call():
    if what in ("mid", "resident", "large"):
        te.i8_linear(x, xs, [dict(w=qw[0], y=y, ldy=n)], ws, stream=stream)
    elif what == "gated":
        te.i8_gated_linear(x, xs, qw[0], qw[1], 1, out, ws, stream=stream)
    elif what == "q8":
        te.q8_linear(xb, [dict(w=qw[0], y=y, ldy=n)], stream=stream)
    elif what == "q8_gated":
        te.q8_gated_linear(xb, qw[0], qw[1], 1, out, stream=stream)
    else:
        te.attn_varlen_fwd(qkv, 384, 0, 128, 256, cu, cu_dev, 2, 2, 64, 0, 0.125, o, 128, stream=stream)
call()
torch.cuda.synchronize()
want = [t.clone() for t in (y, out, o)]
for t in (y, out, o):
    t.zero_()
torch.cuda.synchronize()
fails = []
def first():
    try:
        call()
    except Exception as e:
        fails.append(e)
t = threading.Thread(target=first)
t.start()
t.join()
te.check()
assert not fails, fails
assert all(bool((a == b).all()) for a, b in zip(want, (y, out, o))) and any(bool((t != 0).any()) for t in want)
print("same")
"""


@pytest.mark.parametrize("what", ["mid", "resident", "large", "gated", "q8", "q8_gated", "attention"])
def test_a_threads_first_call(what):
    r = subprocess.run([sys.executable, "-c", SCRIPT, what], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
