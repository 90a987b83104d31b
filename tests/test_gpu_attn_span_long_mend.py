"""Long sequences whose rows have to be computed again: the call takes longer,
and every other row, head and channel has the same bits as without them."""
import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_gpu_attn_span import _lib, call, compare, panel  # noqa: F401  (the library as a fixture)

pytestmark = pytest.mark.gpu

N, NQ = 30001, 6      # about 80 to 120 blocks of 6 heads: several a CTA


def rows_of(qkv, rows, h, hd, see, scale):
    """Some rows of head h in 64 bits: (o, sum_j p_j |v_j|); see [rows, keys]."""
    import torch
    w = NQ * hd
    q, k, v = (qkv[:, i * w + h * hd:i * w + (h + 1) * hd].double() for i in range(3))
    v = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    s = torch.where(see, q[rows] @ torch.nan_to_num(k).T * scale, torch.full((1, 1), float("-inf"), dtype=torch.float64, device="cuda"))
    p = torch.softmax(s, 1)
    return p @ v, p @ v.abs()


@pytest.mark.parametrize("hd", [64, 128])
def test_one_infinite_value(hd):
    """Every row of one head sees it: that channel is infinite, all others keep their bits."""
    import torch
    w = NQ * hd
    qkv = panel(N, 3 * w, 100)
    clean = call(qkv, [N], NQ, NQ, hd, -1, -1, 0, hd ** -0.5)
    qkv[N // 3, 2 * w + hd + 7] = float("-inf")       # head 1
    out = call(qkv, [N], NQ, NQ, hd, -1, -1, 0, hd ** -0.5)
    te.check()
    assert bool((out[:, hd + 7] == float("-inf")).all())
    clean[:, hd + 7] = out[:, hd + 7]
    other = [c for c in range(w) if not hd <= c < 2 * hd]
    assert torch.equal(out[:, other], clean[:, other])
    rows = torch.arange(0, N, 977, device="cuda")
    qkv[N // 3, 2 * w + hd + 7] = 0
    o, mag = rows_of(qkv, rows, 1, hd, torch.ones(len(rows), N, dtype=torch.bool, device="cuda"), hd ** -0.5)
    keep = [c for c in range(hd) if c != 7]
    compare(f"beside an infinite value {hd}", out[rows, hd:2 * hd][:, keep], o[:, keep], mag[:, keep])


@pytest.mark.parametrize("hd", [64, 128])
def test_a_key_that_later_rows_alone_see(hd):
    """Causal: rows before a NaN key keep their results, those of its own tiles too."""
    import torch
    w, j = NQ * hd, N - 30
    qkv = panel(N, 3 * w, 101)
    clean = call(qkv, [N], NQ, NQ, hd, -1, 0, 0, hd ** -0.5)
    dirty = qkv.clone()
    dirty[j, w:] = float("nan")
    out = call(dirty, [N], NQ, NQ, hd, -1, 0, 0, hd ** -0.5)
    te.check()
    assert torch.equal(out[:j - 256], clean[:j - 256])
    assert bool(torch.isnan(out[j:].float()).all())
    rows = torch.arange(j - 256, j, device="cuda")
    see = torch.arange(N, device="cuda")[None] <= rows[:, None]
    for h in (0, NQ - 1):
        o, mag = rows_of(dirty, rows, h, hd, see, hd ** -0.5)
        compare(f"before a key that is NaN {hd}", out[rows, h * hd:(h + 1) * hd], o, mag)


@pytest.mark.parametrize("hd", [64, 128])
def test_a_head_without_a_visible_key(hd):
    """A table column of -inf: that head's rows are 0, the others keep their bits."""
    import torch
    w = NQ * hd
    qkv = panel(N, 3 * w, 102)
    table = torch.randn(32, NQ, device="cuda", generator=torch.Generator(device="cuda").manual_seed(103))
    clean = call(qkv, [N], NQ, NQ, hd, -1, -1, 0, hd ** -0.5, table=table, rel=(32, 128, True))
    table[:, 2] = float("-inf")
    out = call(qkv, [N], NQ, NQ, hd, -1, -1, 0, hd ** -0.5, table=table, rel=(32, 128, True))
    te.check()
    assert bool((out[:, 2 * hd:3 * hd] == 0).all())
    clean[:, 2 * hd:3 * hd] = 0
    assert torch.equal(out, clean)
