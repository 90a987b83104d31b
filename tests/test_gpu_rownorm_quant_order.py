"""te_rownorm_quant takes te_rownorm_mod's steps in their order: its integers and
scales are those of te_quant_rows on that norm's f32 output, to the bit."""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    torch.cuda.init()
    te.lib()
    yield
    te.check()


@pytest.mark.parametrize("kind", [te.TE_NORM_RMS, te.TE_NORM_LN])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,mod,bias,pre", [(8, False, True, 1.0), (264, True, True, 0.5), (512, False, False, 1.0),
                                            (768, True, False, 2.0), (1536, False, True, 1.0), (2048, True, True, 1.0),
                                            (3840, False, False, 1.0), (4096, True, True, 0.25)])
def test_rownorm_quant_is_the_norm_and_then_the_quantiser(d, mod, bias, pre, dt, kind):
    # Rows whose statistics no order of summation can round: quarters of small
    # integers, in pairs of either sign about 3/4 (LN: the mean is 3/4 exactly).
    # Sums of their squares stay below 2^24 sixteenths: exact in f32.
    import torch
    rng = np.random.default_rng([d, kind, mod])
    t, eps = 301, 1e-6
    half = rng.integers(0, 13, (t, d // 2))
    half[:, 0] += 1                                          # no row is constant
    x = np.concatenate([half, -half], 1)
    x = np.take_along_axis(x, rng.permuted(np.tile(np.arange(d), (t, 1)), axis=1), 1)
    x = torch.from_numpy(((x + 3) / 4).astype(np.float32)).to(torch.float32 if dt == "f32" else torch.bfloat16).cuda()
    vec = lambda m, s: torch.from_numpy((m + s * rng.standard_normal(d)).astype(np.float32)).cuda()
    w = vec(1.0, 0.2)
    b = vec(0.0, 0.3) if bias and kind == te.TE_NORM_LN else None
    ms = vec(0.0, 0.2) if mod else None
    y = torch.empty(t, d, device="cuda")
    te.rownorm_mod(x, w, b, ms, kind, eps, y, pre=pre)
    ldq = -(-d // 16) * 16
    want, got = (torch.zeros(t, ldq, dtype=torch.int8, device="cuda")[:, :d] for _ in range(2))
    ws, gs = torch.zeros(t, device="cuda"), torch.zeros(t, device="cuda")
    te.quant_rows(y, want, ws)
    te.rownorm_quant(x, w, b, kind, eps, got, gs, pre=pre, mod_scale=ms)
    te.check()
    assert torch.equal(gs, ws)
    assert torch.equal(got, want)
