"""Finite values whose weighted sum passes f32 though their mean does not."""
import pytest

import transformer_encoder_forward_gb300 as te
from tests.attn_span_ref import attention
from tests.test_gpu_attn_span import _lib, call, compare, panel  # noqa: F401  (the library as a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_values_whose_sum_passes_the_type(hd, bias):
    """Values up to 3e38 (f32 ends at 3.4e38): a mean of them is no larger, their sum is."""
    import torch
    ln, nq = [200, 3, 70], 2
    w = nq * hd
    qkv = panel(sum(ln), 3 * w, 90)
    # the second head's values and a few of the first's
    qkv[:, 2 * w + hd:] = (qkv[:, 2 * w + hd:].float().clamp(-3, 3) * 1e38).to(torch.bfloat16)
    qkv[::7, 2 * w + 3] = 2.5e38
    rel = (32, 128, True) if bias else None
    table = torch.randn(32, nq, device="cuda") if bias else None
    ref, mag = attention(qkv, ln, nq, nq, hd, 60, -1, 2, hd ** -0.5, table=table, rel=rel)
    out = call(qkv, ln, nq, nq, hd, 60, -1, 2, hd ** -0.5, table=table, rel=rel)
    compare(f"large values {hd} bias={bias}", out, ref, mag)
    te.check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_tiny_values_beside_a_lost_one(hd, bias):
    """Rows that are computed again because a tile of theirs holds a NaN keep values near
    the type's smallest (a product of a weight and such a value may not be taken down by 2^29)."""
    import torch
    ln, nq, span = [400, 90], 2, (60, 20, 3)
    w = nq * hd
    qkv = panel(sum(ln), 3 * w, 93)
    qkv[:, 2 * w:] = (qkv[:, 2 * w:].float() * 2.0 ** -116).to(torch.bfloat16)
    rel = (32, 128, True) if bias else None
    table = torch.randn(32, nq, device="cuda") if bias else None
    ref, mag = attention(qkv, ln, nq, nq, hd, *span, hd ** -0.5, table=table, rel=rel)
    qkv[30, w:] = float("nan")                        # beside the sinks: in a tile of every row
    out = call(qkv, ln, nq, nq, hd, *span, hd ** -0.5, table=table, rel=rel)
    hidden = list(range(91, 490)) + list(range(0, 10))
    compare(f"tiny values {hd} bias={bias}", out[hidden], ref[hidden], mag[hidden])
    te.check()
