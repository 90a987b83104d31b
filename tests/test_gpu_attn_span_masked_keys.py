"""Keys that a bias of -inf masks have no influence, whatever they hold: not
even a key of infinities or NaN, whose score is no number before its bias."""
import pytest

import transformer_encoder_forward_gb300 as te
from tests.attn_span_ref import attention
from tests.test_gpu_attn_span import _lib, call, compare, panel  # noqa: F401  (the library as a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("far", [False, True])
def test_a_key_that_its_bias_masks(hd, bad, far):
    """far: a bucket beyond the reach (one bias for whole tiles), else one of near distances."""
    import torch
    ln, nq, rel = [300, 40], 2, (8, 30, True)
    w = nq * hd
    qkv = panel(sum(ln), 3 * w, 80)
    table = torch.randn(8, nq, device="cuda", generator=torch.Generator(device="cuda").manual_seed(81))
    # keys behind a row: buckets 5 (distance 1), 6 (2 to 7) and 7 (8 and more)
    if far:
        table[7, 0] = float("-inf")
    else:
        table[5:, 0] = float("-inf")
    ref, mag = attention(qkv, ln, nq, nq, hd, -1, -1, 0, hd ** -0.5, table=table, rel=rel)
    dirty = qkv.clone()
    dirty[250, w:2 * w] = bad                         # a key; its value stays
    out = call(dirty, ln, nq, nq, hd, -1, -1, 0, hd ** -0.5, table=table, rel=rel)
    rows = list(range(250 - (8 if far else 1), 300))  # rows of head 0 that see it
    blind = [i for i in range(340) if i not in rows]
    compare(f"key {bad} masked by its bias {hd} far={far}", out[blind, :hd], ref[blind, :hd], mag[blind, :hd])
    te.check()
