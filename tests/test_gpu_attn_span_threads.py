"""A call of attention with sinks or relative position bias that has to wait in
the library leaves a Python program's other threads running."""
import os
import shutil
import subprocess
import sys

import pytest

from tests.test_gpu_i8_threads import STUB

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WAITING = """
import ctypes, sys, threading, time, torch
import transformer_encoder_forward_gb300 as te
stub = ctypes.CDLL(sys.argv[1])
te._marshalling().bind_attn(*[ctypes.cast(stub.wait_for_go, ctypes.c_void_p).value] * 2)
stop = False
def other():
    while not stop:
        if stub.called():
            stub.go()
        time.sleep(0.001)
qkv, out = (torch.zeros(4, n, device="cuda", dtype=torch.bfloat16) for n in (192, 64))
cu_dev = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
plan, table = te.relpos_plan(32, 128), torch.zeros(32, 1, device="cuda")
t = threading.Thread(target=other)
t.start()
try:
    te.attn_sink_fwd(qkv, 192, 0, 64, 128, [0, 4], cu_dev, 1, 1, 64, -1, -1, 0, 0.1, out, 64)
    te.attn_relbias_fwd(qkv, 192, 0, 64, 128, [0, 4], cu_dev, 1, 1, 64, -1, -1, 0, 0.1, plan, table, out, 64)
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
