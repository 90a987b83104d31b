"""Blocks whose query tiles see different key tiles, or have no rows, one behind the
other in a CTA: random batches against 64 bits."""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.attn_span_ref import attention
from tests.test_gpu_attn_span import _lib, call, compare, panel  # noqa: F401  (the library as a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("reach", [0, 128, 2048])
@pytest.mark.parametrize("seed", range(6))
def test_random_batches(hd, reach, seed):
    import torch
    rng = np.random.default_rng(seed)
    pick = lambda *a: a[rng.integers(len(a))]
    span = (pick(-1, 0, 5, 64, 200, 500), pick(-1, 0, 10, 100, 300), pick(0, 0, 3, 70, 400))
    ln = [int(pick(1, 64, 100, 129, 300, 400, 500, 700, 1200)) for _ in range(40)]
    nq = 8                                            # some hundreds of blocks: several a CTA
    qkv = panel(sum(ln), 3 * nq * hd, 130 + seed)
    rel = (64, reach, True) if reach else None
    table = torch.randn(64, nq, device="cuda") if reach else None
    ref, mag = attention(qkv, ln, nq, nq, hd, *span, hd ** -0.5, table=table, rel=rel)
    first = call(qkv, ln, nq, nq, hd, *span, hd ** -0.5, table=table, rel=rel)
    compare(f"random batch {span} {hd} {reach}", first, ref, mag)
    for _ in range(5):
        assert torch.equal(call(qkv, ln, nq, nq, hd, *span, hd ** -0.5, table=table, rel=rel), first)
    te.check()
