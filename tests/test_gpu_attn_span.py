"""Attention with limits to either side, sinks and a bucketed relative position
bias (te.attn_sink_fwd, te.attn_relbias_fwd) against 64 bits."""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.attn_span_ref import attention, bound
from tests.gpu_util import record_margin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    torch.cuda.init()
    te.lib()
    yield
    te.check()


def offsets(lens):
    import torch
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


def panel(rows, width, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, width, generator=g, device="cuda").to(torch.bfloat16)


def call(qkv, lens, nq, nkv, hd, left, right, sinks, scale, table=None, rel=None, offs=None, out=None, stream=None):
    import torch
    cu, cu_dev = offsets(lens)
    q_off, k_off, v_off = offs or (0, nq * hd, (nq + nkv) * hd)
    if out is None:
        out = torch.full((sum(lens), nq * hd), float("nan"), dtype=torch.bfloat16, device="cuda")
    args = (qkv, qkv.stride(0), q_off, k_off, v_off, cu, cu_dev, nq, nkv, hd, left, right, sinks, scale)
    if table is None:
        te.attn_sink_fwd(*args, out, out.stride(0), stream=stream)
    else:
        te.attn_relbias_fwd(*args, te.relpos_plan(*rel), table, out, out.stride(0), stream=stream)
    return out


def compare(name, got, ref, mag):
    import torch
    err = (got.to(torch.float64) - ref).abs()
    worst = float((err / bound(ref, mag)).nan_to_num(nan=float("inf")).max())
    record_margin(name, "of the elementwise bound", worst, 1.0)
    assert worst <= 1.0, (name, worst)


LENS = {"one": [1], "two": [2], "short": [37, 64], "edges": [127, 128, 129], "blocks": [255, 256, 257, 1],
        "ones": [1, 1, 1, 600, 1], "long": [1201, 5]}
SPANS = [(-1, -1, 0), (0, 0, 0), (16, 16, 2), (0, -1, 0), (-1, 0, 0), (5, 0, 3), (128, 127, 130), (300, 2, 129),
         (64, 64, 1000), (1, 500, 64)]
HEADS = [(64, 3, 3), (64, 4, 2), (128, 2, 2), (128, 6, 2)]


@pytest.mark.parametrize("hd,nq,nkv", HEADS)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("span", SPANS, ids=lambda s: "l%d_r%d_s%d" % s)
def test_sinks(span, lens, hd, nq, nkv):
    ln = LENS[lens]
    qkv = panel(sum(ln), (nq + 2 * nkv) * hd, 1)
    ref, mag = attention(qkv, ln, nq, nkv, hd, *span, hd ** -0.5)
    out = call(qkv, ln, nq, nkv, hd, *span, hd ** -0.5)
    compare(f"sink {lens} {span} {hd}", out, ref, mag)


RELS = [(32, 128, True), (32, 128, False), (4, 2, True), (320, 800, True), (2, 2, False), (7, 40, False),
        (512, 2048, True), (16, 5, True)]


@pytest.mark.parametrize("hd,nq,nkv", HEADS)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("rel", RELS, ids=lambda r: "b%d_d%d_%d" % r)
def test_relative_bias(rel, lens, hd, nq, nkv):
    import torch
    ln = LENS[lens]
    qkv = panel(sum(ln), (nq + 2 * nkv) * hd, 2)
    table = 3 * torch.randn(rel[0], nq, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    span = (-1, -1, 0)
    ref, mag = attention(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    out = call(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    compare(f"bias {lens} {rel} {hd}", out, ref, mag)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("reach", [960, 970, 980, 990, 1000, 1024, 2048])
def test_bias_of_a_wide_reach(reach, hd):
    """Spread biases that leave shared memory for more, and for fewer, keys and values in flight."""
    import torch
    ln, nq, nkv = [2200, 1100, 700], 8, 4
    rel = (512, reach, True)
    qkv = panel(sum(ln), (nq + 2 * nkv) * hd, 20)
    table = 3 * torch.randn(rel[0], nq, device="cuda", generator=torch.Generator(device="cuda").manual_seed(21))
    span = (-1, -1, 0)
    ref, mag = attention(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    out = call(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    compare(f"bias of reach {reach} {hd}", out, ref, mag)


@pytest.mark.parametrize("hd,nq,nkv", HEADS)
@pytest.mark.parametrize("span", SPANS, ids=lambda s: "l%d_r%d_s%d" % s)
@pytest.mark.parametrize("rel", [(32, 128, True), (32, 128, False), (64, 300, True)], ids=lambda r: "b%d_d%d_%d" % r)
def test_relative_bias_in_a_window(rel, span, hd, nq, nkv):
    import torch
    ln = [700, 130, 3]
    qkv = panel(sum(ln), (nq + 2 * nkv) * hd, 4)
    table = 3 * torch.randn(rel[0], nq, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    ref, mag = attention(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    out = call(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    compare(f"bias in a window {span} {rel} {hd}", out, ref, mag)


def test_only_itself():
    """left = right = 0 without sinks: each row's output is its own value, to the bit."""
    import torch
    for hd in (64, 128):
        ln = [300, 1, 129]
        qkv = panel(sum(ln), 3 * 2 * hd, 6)
        out = call(qkv, ln, 2, 2, hd, 0, 0, 0, hd ** -0.5)
        assert torch.equal(out, qkv[:, 4 * hd:])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 100, 512, 5000])
def test_as_the_symmetric_window(hd, window):
    """Without sinks or bias: te.attn_varlen_fwd's results, each within its bound."""
    import torch
    ln = [900, 257, 64, 1]
    qkv = panel(sum(ln), 3 * 2 * hd, 7)
    side = window if window else -1
    out = call(qkv, ln, 2, 2, hd, side, side, 0, hd ** -0.5)
    want = torch.empty_like(out)
    cu, cu_dev = offsets(ln)
    te.attn_varlen_fwd(qkv, qkv.stride(0), 0, 2 * hd, 4 * hd, cu, cu_dev, 2, 2, hd, window, hd ** -0.5, want, want.stride(0))
    ref, mag = attention(qkv, ln, 2, 2, hd, side, side, 0, hd ** -0.5)
    compare(f"symmetric window {window} {hd}", out, ref, mag)
    err = (out.double() - want.double()).abs()
    assert bool((err <= 2 * bound(ref, mag)).all())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_many_blocks(hd, bias):
    """More query blocks than the launch carries in a list."""
    import torch
    rng = np.random.default_rng(8)
    ln = [int(n) for n in rng.integers(1, 60, 690)] + [1500] + [int(n) for n in rng.integers(1, 300, 30)]
    nq, nkv = 2, 1
    qkv = panel(sum(ln), (nq + 2 * nkv) * hd, 9)
    rel = (32, 128, True) if bias else None
    table = torch.randn(32, nq, device="cuda") if bias else None
    for span in ((-1, -1, 0), (40, 10, 3)):
        ref, mag = attention(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
        out = call(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
        compare(f"many blocks {span} {hd} bias={bias}", out, ref, mag)


@pytest.mark.parametrize("hd", [64, 128])
def test_panel_layout(hd):
    """v before q before k, wider rows, odd heads; columns and rows that are no output stay."""
    import torch
    ln, nq, nkv = [200, 33], 6, 3
    offs = (nkv * hd + 8, (nkv + nq) * hd + 16, 0)
    rows = sum(ln) + 7
    qkv = panel(rows, (nq + 2 * nkv) * hd + 24, 10)
    qkv[sum(ln):] = float("nan")                      # rows behind the last sequence
    out = torch.full((rows, nq * hd + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    ref, mag = attention(qkv[:sum(ln)], ln, nq, nkv, hd, 50, 20, 5, 0.1, offs=offs)
    call(qkv, ln, nq, nkv, hd, 50, 20, 5, 0.1, offs=offs, out=out)
    compare(f"layout {hd}", out[:sum(ln), :nq * hd], ref, mag)
    assert bool((out[sum(ln):] == 7).all()) and bool((out[:, nq * hd:] == 7).all())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_masked_values_have_no_influence(hd, bias, bad):
    """Keys and values that a row does not see may be anything."""
    import torch
    ln, nq, nkv = [260, 150, 31], 2, 2
    qkv = panel(sum(ln), (nq + 2 * nkv) * hd, 11)
    rel = (32, 128, True) if bias else None
    table = torch.randn(32, nq, device="cuda") if bias else None
    span = (20, 10, 3)
    clean = call(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    dirty = qkv.clone()
    # row 100 of the first sequence as key and value, and the whole last sequence
    dirty[100, nq * hd:] = bad
    dirty[410:] = bad
    out = call(dirty, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    sees = [i for i in range(260) if 90 <= i <= 120]  # i - 20 <= 100 <= i + 10
    hidden = [i for i in range(410) if i not in sees]
    ref, mag = attention(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=rel)
    compare(f"masked {bad} {hd} bias={bias}", out[hidden], ref[hidden], mag[hidden])
    compare(f"not masked {hd} bias={bias}", clean, ref, mag)
    assert not bool(torch.isfinite(out[sees].float()).all(1).any())
    # a neighbour in the packing changes no bit
    assert torch.equal(out[260:410], clean[260:410])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("low", [float("-inf"), -3.4028234663852886e38, -1e30])
def test_bias_that_masks(hd, low):
    """Buckets of -inf are masked (a row with nothing left is 0); of the type's
    lowest value they count only where a row has nothing else."""
    import torch
    ln, nq, nkv, rel = [400, 20, 1], 3, 3, (8, 30, True)
    qkv = panel(sum(ln), (nq + 2 * nkv) * hd, 12)
    table = torch.randn(8, nq, device="cuda")
    table[:, 0] = low                                 # head 0: everything
    table[5:, 1] = low                                # head 1: distances j - i > 1
    table[0, 2] = low                                 # head 2: itself
    ref, mag = attention(qkv, ln, nq, nkv, hd, -1, -1, 0, hd ** -0.5, table=table, rel=rel)
    out = call(qkv, ln, nq, nkv, hd, -1, -1, 0, hd ** -0.5, table=table, rel=rel)
    compare(f"bias {low} {hd}", out, ref, mag)
    if low == float("-inf"):
        assert bool((out[:, :hd] == 0).all())
        # and a value that only such a bucket holds may be anything
        dirty = qkv.clone()
        dirty[420, 5 * hd + nkv * hd:] = float("nan")  # the last sequence's one row, head 2's value
        again = call(dirty, ln, nq, nkv, hd, -1, -1, 0, hd ** -0.5, table=table, rel=rel)
        assert bool((again[420, 2 * hd:] == 0).all())
        assert torch.equal(again[:420], out[:420])


@pytest.mark.parametrize("hd", [64, 128])
def test_large_scores(hd):
    """Scores far apart, a maximum that moves from tile to tile, either sign."""
    import torch
    ln, nq = [900], 2
    qkv = panel(900, 3 * nq * hd, 13)
    qkv[:, :nq * hd] *= 6
    qkv[:, nq * hd:2 * nq * hd] *= torch.linspace(0.1, 6, 900, device="cuda")[:, None]
    qkv[450:, nq * hd:2 * nq * hd] = qkv[450:, nq * hd:2 * nq * hd].flip(0)
    # q and k so that sums are exact in f32: whole numbers
    qkv[:, :2 * nq * hd] = qkv[:, :2 * nq * hd].round()
    ref, mag = attention(qkv, ln, nq, nq, hd, 600, 300, 2, 0.25)
    out = call(qkv, ln, nq, nq, hd, 600, 300, 2, 0.25)
    compare(f"large scores {hd}", out, ref, mag)


def test_order_of_sequences_and_runs():
    """A sequence's rows do not depend on what it is packed with, nor on the run."""
    import torch
    for hd in (64, 128):
        nq = 2
        a, b = panel(333, 3 * nq * hd, 14), panel(200, 3 * nq * hd, 15)
        table, rel = torch.randn(32, nq, device="cuda"), (32, 128, True)
        f = lambda x, ln: call(x, ln, nq, nq, hd, 100, 50, 4, hd ** -0.5, table=table, rel=rel)
        ab, ba, alone = f(torch.cat([a, b]), [333, 200]), f(torch.cat([b, a]), [200, 333]), f(a, [333])
        assert torch.equal(ab[:333], alone) and torch.equal(ba[200:], alone) and torch.equal(ab[333:], ba[:200])


def test_no_limit_is_a_limit_past_the_end():
    import torch
    qkv = panel(500, 3 * 128, 16)
    big = 2 ** 31 - 1
    for hd, nq in ((64, 2), (128, 1)):
        x = call(qkv, [500], nq, nq, hd, -1, -1, 0, 0.1)
        assert torch.equal(x, call(qkv, [500], nq, nq, hd, big, big, big, 0.1))
        assert torch.equal(x, call(qkv, [500], nq, nq, hd, 0, -1, big, 0.1))
