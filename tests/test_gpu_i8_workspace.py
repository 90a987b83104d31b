"""8-bit products of short k, called without a workspace."""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [9, 40, 300, 3000])
@pytest.mark.parametrize("k", [64, 512])
def test_short_k_without_a_workspace(m, k):
    import torch
    rng = np.random.default_rng([m, k])
    x, w = (torch.from_numpy(rng.integers(-127, 128, s).astype(np.int8)).cuda() for s in ((m, k), (2, 96, k)))
    one = torch.ones(max(m, 96), device="cuda")
    qw = [te.q8w(w[i], one[:96]) for i in range(2)]
    y, o = torch.zeros(m, 96, device="cuda"), torch.zeros(m, 96, device="cuda", dtype=torch.bfloat16)
    te.i8_linear(x, one[:m], [dict(w=qw[0], y=y, ldy=96)], None)
    te.i8_gated_linear(x, one[:m], qw[0], qw[1], te.TE_ACT_SILU, o, None)
    te.check()
    g, u = (x.double() @ a.double().T for a in w)
    assert torch.equal(y.double(), g)                        # sums below 2^24: exact
    ref = g / (1 + torch.exp(-g)) * u
    # the product rounded once to bf16 (2^-8), behind the activation in f32:
    # three roundings of the exponent |g| and sixteen half steps; factors of
    # g u below 2^-125 may be flushed to zero
    lim = (2.0 ** -8 + (3 * g.abs() + 16) * 2.0 ** -24) * ref.abs() + 2.0 ** -125 * (g * u).abs()
    assert bool(((o.double() - ref).abs() <= lim).all())
