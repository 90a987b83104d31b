"""Products of many tokens on every kernel that takes them: few output features
(k split over clusters), short k (resident weights) and long k (the widening
pass and the large pipeline), at widths that end inside their tiles."""
import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_gpu_i8 import (_lib, _torch, _ws, test_i8_gated_linear_matches_64_bits as gated,  # noqa: F401
                               test_i8_linear_matches_64_bits as linear)

pytestmark = pytest.mark.gpu

FEW = [(4000, 1024, [128], False, None, "bf16"), (8000, 2112, [64, 32], True, "sep", "f32"),
       (20000, 64, [32], True, "in", "f32"), (5001, 4096, [96], True, None, "bf16"), (1500, 768, [768], True, "in", "f32")]
SHORT = [(9000, 512, [512, 512, 96], True, "in", "f32"), (16000, 192, [512, 160], False, "sep", "bf16"),
         (30000, 64, [512], True, None, "f32"), (9001, 448, [640, 512], True, None, "bf16")]
LONG = [(3000, 1024, [1024, 160, 32], True, "in", "f32"), (2600, 576, [768, 288], False, "sep", "bf16"),
        (4100, 2048, [1024], True, None, "f32")]


@pytest.mark.parametrize("m,k,ns,bias,resid,ydt", FEW + SHORT + LONG)
def test_many_tokens_match_64_bits(m, k, ns, bias, resid, ydt):
    linear(m, k, ns, bias, resid, ydt)


@pytest.mark.parametrize("act", [te.TE_ACT_GELU_TANH, te.TE_ACT_SILU])
@pytest.mark.parametrize("m,k,f", [(1284, 832, 64), (5000, 192, 64), (9000, 2112, 32), (16000, 512, 480), (30000, 64, 512),
                                   (9001, 448, 992), (3000, 1024, 992), (5000, 576, 416), (2600, 2048, 1024)])
def test_many_tokens_gated_match_64_bits(m, k, f, act):
    gated(m, k, f, act)


@pytest.mark.parametrize("m", [1025, 4097, 20001])
@pytest.mark.parametrize("k,ns", [(64, [512, 96]), (512, [512, 160, 32]), (512, [1600]), (576, [1600]), (1024, [1024, 288]),
                                  (1024, [32]), (4096, [64])])
def test_many_tokens_are_exact_on_integers(m, k, ns):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(m + k)
    x = torch.randint(-60, 61, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    ones = torch.ones(m, device="cuda")
    w = [torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8) for n in ns]
    sw = torch.ones(4096, device="cuda")
    full = [torch.full((m + 1, n), float("nan"), device="cuda") for n in ns]
    te.i8_linear(x, ones, [dict(w=te.q8w(a, sw[:a.shape[0]]), y=y[:m], ldy=y.shape[1]) for a, y in zip(w, full)],
                 _ws(m, k, sum(ns)))
    for a, y in zip(w, full):
        ref = x.double() @ a.double().T
        assert float(ref.abs().max()) < 2 ** 24
        assert torch.equal(y[:m].double(), ref)
        assert bool(torch.isnan(y[m]).all())
    te.check()


@pytest.mark.parametrize("m,k", [(5, 512), (13, 1024), (30, 64), (60, 768), (700, 192), (9000, 512), (20000, 64), (3000, 1024)])
def test_items_of_one_call_of_every_kind_at_once(m, k):
    # f32 and bf16 outputs, bias, both residuals and both activations in one call,
    # against a call for each; sums below 2^24 are exact, so the bits are the same
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(m + k)
    x = torch.randint(-127, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    xs = torch.rand(m, generator=gen, device="cuda") * 1e-3
    ns = [512, 96, 288, 32]
    keep, qw = [], []
    for i, n in enumerate(ns):
        w = torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
        s, b = torch.rand(n, generator=gen, device="cuda"), torch.randn(n, generator=gen, device="cuda")
        keep.append((w, s, b))
        qw.append(te.q8w(w, s, b if i % 2 else None))
    start = torch.randn(m, 512, generator=gen, device="cuda")
    sep = torch.randn(m, 288, generator=gen, device="cuda")

    def outputs():
        return [start.clone(), torch.zeros(m, 96, device="cuda", dtype=torch.bfloat16), torch.zeros(m, 288, device="cuda"),
                torch.zeros(m, 32, device="cuda", dtype=torch.bfloat16)]

    def item(i, y):
        d = dict(w=qw[i], y=y, ldy=ns[i])
        d.update([dict(residual=y, ldr=512), dict(epilogue=te.TE_EPI_SILU), dict(residual=sep, ldr=288),
                  dict(epilogue=te.TE_EPI_GELU_TANH)][i])
        return d

    ws = _ws(m, k, sum(ns))
    together, apart = outputs(), outputs()
    te.i8_linear(x, xs, [item(i, y) for i, y in enumerate(together)], ws)
    for i, y in enumerate(apart):
        te.i8_linear(x, xs, [item(i, y)], ws)
    te.check()
    for a, b in zip(together, apart):
        assert torch.equal(a, b)
        assert bool((a != 0).any())
