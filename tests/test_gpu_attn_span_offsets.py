"""The device's offsets of te.attn_sink_fwd and te.attn_relbias_fwd: not read where
the sequences' blocks travel with the launch, read and bounded where they are
too many for it."""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.attn_span_ref import attention
from tests.test_gpu_attn_span import _lib, compare, offsets, panel  # noqa: F401  (the library as a fixture)

pytestmark = pytest.mark.gpu


def run(qkv, cu, dev, nq, hd, out, bias):
    import torch
    args = (qkv, 3 * nq * hd, 0, nq * hd, 2 * nq * hd, cu, dev, nq, nq, hd, 9, 9, 1, 0.1)
    if bias:
        te.attn_relbias_fwd(*args, te.relpos_plan(32, 128), torch.zeros(32, nq, device="cuda"), out, nq * hd)
    else:
        te.attn_sink_fwd(*args, out, nq * hd)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_few_blocks_take_the_hosts_offsets(hd, bias):
    import torch
    nq, cu = 2, np.array([0, 100, 300], np.int32)
    qkv = panel(300, 3 * nq * hd, 51)
    right = torch.empty(300, nq * hd, dtype=torch.bfloat16, device="cuda")
    run(qkv, cu, torch.from_numpy(cu).cuda(), nq, hd, right, bias)
    for bad in ([0, 100, 10 ** 9], [-5, 100, 300], [0, 300, 100], [2 ** 31 - 1, -2 ** 31, 7], [0, 100, 301]):
        guard = torch.full((900, nq * hd), 7.0, dtype=torch.bfloat16, device="cuda")
        run(qkv, cu, torch.tensor(bad, dtype=torch.int32, device="cuda"), nq, hd, guard[300:600], bias)
        assert bool((guard[:300] == 7).all()) and bool((guard[600:] == 7).all()), bad
        assert torch.equal(guard[300:600], right), bad
    te.check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_many_blocks_read_the_devices_offsets(hd, bias):
    """One entry that is not the host's, at the start, within and at the end: rows outside
    the panel are neither read nor written."""
    import torch
    nq, lens = 2, [1] * 700 + [50, 3]
    cu, good = offsets(lens)
    rows, n = sum(lens), len(lens)
    qkv = panel(rows, 3 * nq * hd, 52)
    ref, mag = attention(qkv, lens, nq, nq, hd, 9, 9, 1, 0.1)
    for at in (0, 1, 350, 700, 701, n):
        for value in (-5, -2 ** 31, 2 ** 31 - 1, 10 ** 9, rows + 1, 0, int(cu[at])):
            dev = good.clone()
            dev[at] = value
            guard = torch.full((3 * rows, nq * hd), 7.0, dtype=torch.bfloat16, device="cuda")
            run(qkv, cu, dev, nq, hd, guard[rows:2 * rows], bias)
            torch.cuda.synchronize()
            assert bool((guard[:rows] == 7).all()) and bool((guard[2 * rows:] == 7).all()), (at, value)
            if value == cu[at]:
                compare(f"the device's offsets {hd} bias={bias}", guard[rows:2 * rows], ref, mag)
    for dev in (np.arange(n + 1)[::-1], np.full(n + 1, rows), np.zeros(n + 1)):   # backwards, all the end, all the start
        guard = torch.full((3 * rows, nq * hd), 7.0, dtype=torch.bfloat16, device="cuda")
        run(qkv, cu, torch.from_numpy(dev.astype(np.int32)).cuda(), nq, hd, guard[rows:2 * rows], bias)
        torch.cuda.synchronize()
        assert bool((guard[:rows] == 7).all()) and bool((guard[2 * rows:] == 7).all())
    te.check()
