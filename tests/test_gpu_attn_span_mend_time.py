"""What rows that are not the plain case cost: the time of a call beside that of
the same call on ordinary inputs.  (Limits far above what is measured, a third
of them or less, and far below a pass over the keys one by one: 400 to 1000 times a call's time.)"""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_gpu_attn_span import _lib, offsets, panel  # noqa: F401  (the library as a fixture)

pytestmark = pytest.mark.gpu


def time_of(qkv, n, nq, hd, left, right, sinks, table=None):
    """us a call, the least of several; the output."""
    import torch
    cu, cu_dev = offsets([n])
    w = nq * hd
    out = torch.empty(n, w, dtype=torch.bfloat16, device="cuda")
    args = (qkv, 3 * w, 0, w, 2 * w, cu, cu_dev, nq, nq, hd, left, right, sinks, hd ** -0.5)
    plan = te.relpos_plan(32, 128)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(5):
        a.record()
        for _ in range(3):
            if table is None:
                te.attn_sink_fwd(*args, out, w)
            else:
                te.attn_relbias_fwd(*args, plan, table, out, w)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 3 * 1000)
    te.check()
    return best, out


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads", ["one", "all"])
def test_heads_without_a_visible_key(hd, heads):
    """Table columns of -inf: nothing is left to compute."""
    import torch
    n, nq = 4096, 12
    qkv = panel(n, 3 * nq * hd, 110)
    table = torch.randn(32, nq, device="cuda")
    usual, _ = time_of(qkv, n, nq, hd, -1, -1, 0, table)
    lost = 1 if heads == "one" else nq
    table[:, :lost] = float("-inf")
    took, out = time_of(qkv, n, nq, hd, -1, -1, 0, table)
    assert bool((out[:, :lost * hd] == 0).all())
    assert took < 5 * usual, (took, usual)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("what", ["one value", "a value", "a key", "a query", "all"])
def test_rows_that_see_a_lost_key(hd, what):
    """Every row sees it."""
    import torch
    n, nq = 4096, 12
    w = nq * hd
    qkv = panel(n, 3 * w, 111)
    usual, clean = time_of(qkv, n, nq, hd, -1, -1, 0)
    if what == "one value":
        qkv[n // 2, 2 * w + 5] = float("inf")
    elif what == "a value":
        qkv[n // 2, 2 * w:] = float("nan")
    elif what == "a key":
        qkv[n // 2, w:2 * w] = float("nan")
    elif what == "a query":
        qkv[n // 2, :w] = float("inf")
    else:
        qkv[:] = float("nan")
    took, out = time_of(qkv, n, nq, hd, -1, -1, 0)
    if what == "one value":
        assert bool((out[:, 5] == float("inf")).all())
        clean[:, 5] = out[:, 5]
        assert torch.equal(out, clean)
    elif what == "a query":
        assert bool(torch.isnan(out[n // 2].float()).all())
        clean[n // 2] = out[n // 2] = 0
        assert torch.equal(out, clean)
    else:
        assert bool(torch.isnan(out.float()).all())
    assert took < 25 * usual, (took, usual)


@pytest.mark.parametrize("hd", [64, 128])
def test_rows_beside_a_lost_key(hd):
    """A key beside the sinks lies in a tile of every row, and none past the window sees it."""
    import torch
    n, nq = 4096, 12
    w = nq * hd
    qkv = panel(n, 3 * w, 112)
    usual, _ = time_of(qkv, n, nq, hd, 256, 256, 3)
    qkv[40, w:] = float("nan")
    took, out = time_of(qkv, n, nq, hd, 256, 256, 3)
    assert bool(torch.isnan(out[:297].float()).all()) and bool(torch.isfinite(out[297:].float()).all())
    assert took < 150 * usual, (took, usual)
