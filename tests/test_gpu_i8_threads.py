"""Calls of the 8-bit and rotation operators from Python programs of several
threads: a call that has to wait in the library leaves the other threads
running, and first calls made at the same time give the results of calls apart."""
import os
import shutil
import subprocess
import sys

import pytest

import transformer_encoder_forward_gb300 as te  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Stands in for the library's functions: waits, three seconds at most, until
# another thread of the program has called go().
STUB = """
#include <stdatomic.h>
#include <unistd.h>
static atomic_int inside, gone;
int called(void) { return atomic_load(&inside); }
void go(void) { atomic_store(&gone, 1); }
int wait_for_go(void) {
    atomic_store(&gone, 0);
    atomic_store(&inside, 1);
    int i = 0;
    while (!atomic_load(&gone) && i++ < 3000) usleep(1000);
    atomic_store(&inside, 0);
    return atomic_load(&gone) ? 0 : 1;
}
"""

WAITING = """
import ctypes, sys, threading, time, torch
import transformer_encoder_forward_gb300 as te
stub = ctypes.CDLL(sys.argv[1])
te._marshalling().bind(*[ctypes.cast(stub.wait_for_go, ctypes.c_void_p).value] * 5)
stop = False
def other():
    while not stop:
        if stub.called():
            stub.go()
        time.sleep(0.001)
x, q, s = (torch.zeros(4, 64, device="cuda", dtype=d) for d in (torch.float32, torch.int8, torch.float32))
s = s[:, 0].contiguous()
w, sw = torch.zeros(32, 64, device="cuda", dtype=torch.int8), torch.zeros(32, device="cuda")
qw = te.q8w(w, sw)
y, o = torch.zeros(4, 32, device="cuda"), torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16)
pos, plan = torch.zeros(4, 2, device="cuda", dtype=torch.int32), te.rope_axes_plan(32, (16, 16))
t = threading.Thread(target=other)
t.start()
try:
    te.quant_rows(x, q, s)
    te.rownorm_quant(x, torch.ones(64, device="cuda"), None, 0, 1e-6, q, s)
    te.i8_linear(q, s, [dict(w=qw, y=y, ldy=32)], None)
    te.i8_gated_linear(q, s, qw, qw, 0, o, None)
    te.qk_rope_axes(x, 64, x, 64, 0, 32, 1, 1, 32, None, None, 1e-6, plan, pos, 1.0, 4)
    print("went on")
finally:
    stop = True
    t.join()
"""


def test_other_threads_run_while_a_call_waits(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "stub.c").write_text(STUB)
    so = str(tmp_path / "stub.so")
    subprocess.run([cc, "-shared", "-fPIC", "-o", so, str(tmp_path / "stub.c")], check=True)
    r = subprocess.run([sys.executable, "-c", WAITING, so], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("went on"), r.stderr[-2000:]


FIRST = """
import threading, torch
import transformer_encoder_forward_gb300 as te
torch.manual_seed(2)
i8 = lambda *s: torch.randint(-127, 128, s, dtype=torch.int8, device="cuda")
jobs = []
for m, k, n in ((5, 512, 96), (60, 768, 256), (2000, 512, 128), (2000, 1024, 256), (40, 1024, 512), (300, 512, 640)):
    x, xs, w, sw = i8(m, k), torch.rand(m, device="cuda"), i8(n, k), torch.rand(n, device="cuda")
    src, q, s = torch.randn(m, k, device="cuda"), i8(m, k), torch.zeros(m, device="cuda")
    ws = torch.empty(te.i8_workspace(m, k, 2 * n) + 256, dtype=torch.uint8, device="cuda")
    y, o = torch.zeros(m, n, device="cuda"), torch.zeros(m, n, device="cuda", dtype=torch.bfloat16)
    pos, plan = torch.randint(0, 99, (m, 2), dtype=torch.int32, device="cuda"), te.rope_axes_plan(64, (32, 32))
    jobs.append((m, k, n, x, xs, te.q8w(w, sw), w, sw, src, q, s, ws, y, o, pos, plan, torch.zeros(m, k, device="cuda"),
                 torch.zeros(m, n, device="cuda"), ws.clone()))
torch.cuda.synchronize()
def run(j, stream):
    m, k, n, x, xs, qw, _, _, src, q, s, ws, y, o, pos, plan, r, _, _ = j
    te.quant_rows(src, q, s, stream=stream)
    te.i8_linear(x, xs, [dict(w=qw, y=y, ldy=n)], ws, stream=stream)
    te.i8_gated_linear(x, xs, qw, qw, 1, o, ws, stream=stream)
    te.qk_rope_axes(src, k, r, k, 0, k // 2, 4, 4, 64, None, None, 1e-6, plan, pos, 1.0, m, stream=stream)
outs = lambda j: (j[9], j[10], j[12], j[13], j[16])
gate, fails = threading.Barrier(2 * len(jobs)), []
def one(j, first):
    stream = torch.cuda.Stream()
    gate.wait()
    try:
        if first:
            run(j, stream)
        else:                                   # the same kernel's first call, on buffers of its own
            te.i8_linear(j[3], j[4], [dict(w=j[5], y=j[17], ldy=j[2])], j[18], stream=stream)
    except Exception as e:
        fails.append(e)
    stream.synchronize()
threads = [threading.Thread(target=one, args=(j, f)) for j in jobs for f in (True, False)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not fails, fails
got = [[t.clone() for t in outs(j)] for j in jobs]
torch.cuda.synchronize()
for j, g in zip(jobs, got):
    for t in outs(j):
        t.zero_()
    run(j, None)
    torch.cuda.synchronize()
    assert all(bool((a == b).all()) and bool((a != 0).any()) for a, b in zip(g, outs(j))), j[:3]
    assert bool((j[17] == j[12]).all()), j[:3]
te.check()
print("same")
"""


def test_first_calls_from_several_threads_at_once():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
