"""Scores so large that f32 holds them to a hundred units only."""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_gpu_attn_span import _lib, call, compare, panel  # noqa: F401  (the library as a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_scores_of_two_to_the_31(hd, bias):
    """One key a row, so each row's output is that key's value, whatever the score.
    f32 holds scores of 2^31 to a hundred units: the score less its own rounded
    maximum may be any power to 2^+-256, and the row's sum with it.  (Within the
    bound and not to the bit: where such a weight is kept, its bf16 form is off by up
    to 2^-9 of it, and the sum that divides is not.)"""
    import torch
    n, nq = 6000, 2
    w = nq * hd
    ln = [1] * n
    qkv = panel(n, 3 * w, 91)
    rng = np.random.default_rng(92)
    # one product a score, exact in f32: 2^31 to 2^32 in log2 units
    qkv[:, :2 * w] = 0
    a, b = rng.integers(128, 256, (2, n, nq)), rng.integers(128, 256, (2, n, nq))
    for h in range(nq):
        qkv[:, h * hd] = torch.from_numpy(a[0, :, h] * b[0, :, h] % 128 + 128.0).cuda()
        qkv[:, w + h * hd] = torch.from_numpy(a[1, :, h] * 1.0).cuda()
    scale = 2.0 ** 17                                 # 2^14 .. 2^16 times 2^17
    rel = (32, 128, True) if bias else None
    table = torch.randn(32, nq, device="cuda") if bias else None
    out = call(qkv, ln, nq, nq, hd, -1, -1, 0, scale, table=table, rel=rel)
    v = qkv[:, 2 * w:].double()
    compare(f"scores of 2^31 {hd} bias={bias}", out, v, v.abs())
    te.check()
