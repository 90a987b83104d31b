"""Sums past 2^24 in the 8-bit products: every kernel, up to the longest k, stays
within the bound that the header states, one f32 step (2^-23 of the largest
partial sum) for every 16 products."""
import pytest

import transformer_encoder_forward_gb300 as te
from tests.gpu_util import record_margin
from tests.test_gpu_i8_choice import FEW, LARGE, MID, RES, _rule_again, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = [((FEW, 8, 2), 5), ((FEW, 8, 4), 8), ((FEW, 16, 1), 13), ((FEW, 16, 2), 9), ((FEW, 32, 1), 30),
           *(((MID, t, s), t + 3) for t in (16, 32, 64, 128) for s in (1, 2, 4, 8)),
           ((LARGE, 0, 0), 50), ((LARGE, 0, 0), 300), ((LARGE, 0, 0), 1300), ((LARGE, 0, 0), 4300)]


@pytest.mark.parametrize("k", [1088, 10240, 65536])
@pytest.mark.parametrize("choice,m", KERNELS)
def test_one_signed_sums(choice, m, k):
    import torch
    n = 96
    te.i8_choose(choice)
    x = torch.full((m, k), 127, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), 127, dtype=torch.int8, device="cuda")
    w[1::4] = -127                                           # sums of the other sign
    w[2::4, k // 2:] = -127                                  # up to half, and back to nothing
    w[3::4] = torch.randint(1, 128, (n // 4, k), dtype=torch.int8, device="cuda",
                            generator=torch.Generator("cuda").manual_seed(k))
    x[:, 1::3] = 126                                         # sums that are no multiple of a power of two
    one = torch.ones(max(m, n), device="cuda")
    y = torch.empty(m, n, device="cuda")
    te.i8_linear(x, one[:m], [dict(w=te.q8w(w, one[:n]), y=y, ldy=n)], workspace(m, k, n))
    te.check()
    ref = x.double() @ w.double().T
    lim = (k / 16) * 2.0 ** -23 * 127.0 * 127.0 * k
    err = float((y.double() - ref).abs().max())
    assert record_margin("i8 sums", f"{choice} m={m} k={k}: {err / (127.0 * 127.0 * k):.2e} of the largest sum", err / lim, 1.0) <= 1


@pytest.mark.parametrize("choice,m", [*KERNELS, ((RES, 128, 1), 300)])
def test_sums_to_1024_products_are_exact_whatever_their_values(choice, m):
    # 1024 products of -128 and -128 reach 2^24, which f32 still holds
    import torch
    n, k = 96, 512 if choice[0] == RES else 1024
    te.i8_choose(choice)
    x = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    w[1::3], w[2::3] = 127, torch.randint(-128, 0, (n // 3, k), dtype=torch.int8, device="cuda",
                                          generator=torch.Generator("cuda").manual_seed(1))
    one = torch.ones(max(m, n), device="cuda")
    y = torch.empty(m, n, device="cuda")
    te.i8_linear(x, one[:m], [dict(w=te.q8w(w, one[:n]), y=y, ldy=n)], workspace(m, k, n))
    te.check()
    assert torch.equal(y.double(), x.double() @ w.double().T)
