"""Values and keys that are not finite: each output is what the keys that its row
sees make of it, in every window, with sinks and with buckets that mask."""
import pytest

import transformer_encoder_forward_gb300 as te
from tests.attn_span_ref import attention, bucket_table, visible
from tests.test_gpu_attn_span import _lib, call, compare, panel  # noqa: F401  (the library as a fixture)

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
REL = (8, 30, True)


def expected(qkv, ln, nq, nkv, hd, span, table):
    """o and mag in 64 bits; o is +-inf where a row sees infinite values of one sign in
    that channel, NaN where it sees both or a NaN."""
    import torch
    w, kw = nq * hd, nkv * hd
    o, mag = attention(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=REL if table is not None else None)
    at = 0
    for n in ln:
        see = visible(n, *span, device="cuda")
        if table is not None:
            b = torch.tensor(bucket_table(n, *REL), device="cuda")
            i = torch.arange(n, device="cuda")
            which = b[i[None] - i[:, None] + n - 1]
        for h in range(nq):
            g = h // (nq // nkv)
            own = see if table is None else see & (table[:, h] != -INF)[which]
            v = qkv[at:at + n, w + kw + g * hd:w + kw + (g + 1) * hd].double()
            count = lambda m: own.double() @ m.double() > 0
            up, down = count(~torch.isfinite(v) & ~(v < 0)), count(~torch.isfinite(v) & ~(v > 0))
            x = attention_of_finite(qkv[at:at + n], own, h, g, nq, nkv, hd, table, which if table is not None else None)
            y = o[at:at + n, h * hd:(h + 1) * hd]
            y.copy_(x[0])
            mag[at:at + n, h * hd:(h + 1) * hd] = x[1]
            y[up] = INF
            y[down] = -INF
            y[up & down] = NAN
        at += n
    return o, mag


def attention_of_finite(x, own, h, g, nq, nkv, hd, table, which):
    """One head with the values that are not finite left out."""
    import torch
    w, kw = nq * hd, nkv * hd
    q, k = x[:, h * hd:(h + 1) * hd].double(), x[:, w + g * hd:w + (g + 1) * hd].double()
    v = x[:, w + kw + g * hd:w + kw + (g + 1) * hd].double()
    v = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    s = q @ k.T * hd ** -0.5
    if table is not None:
        s = s + table[:, h].double()[which]
    s = torch.where(own, s, torch.full_like(s, -INF))
    m = s.amax(1, keepdim=True)
    p = torch.exp(s - torch.where(m == -INF, torch.zeros_like(m), m))
    den = p.sum(1, keepdim=True)
    p = torch.where(den > 0, p / den, torch.zeros_like(p))
    return p @ v, p @ v.abs()


def same(name, out, o, mag):
    import torch
    out = out.double()
    assert torch.equal(torch.isnan(out), torch.isnan(o)), name
    assert torch.equal(out == INF, o == INF) and torch.equal(out == -INF, o == -INF), name
    fin = torch.isfinite(o)
    compare(name, out[fin], o[fin], mag[fin])


SPANS = [(-1, -1, 0), (-1, 0, 0), (20, 10, 3), (70, 0, 130), (0, -1, 2), (33, 64, 70)]


@pytest.mark.parametrize("hd,nq,nkv", [(64, 4, 2), (128, 2, 2)])
@pytest.mark.parametrize("span", SPANS, ids=lambda s: "l%d_r%d_s%d" % s)
@pytest.mark.parametrize("bias", ["none", "finite", "masks"])
@pytest.mark.parametrize("many", [False, True])
def test_values_that_are_not_finite(hd, nq, nkv, span, bias, many):
    import torch
    ln = [500, 1, 161, 64]
    w, kw = nq * hd, nkv * hd
    g = torch.Generator(device="cuda").manual_seed(120)
    qkv = panel(sum(ln), w + 2 * kw, 121)
    table = None
    if bias != "none":
        table = torch.randn(REL[0], nq, device="cuda", generator=g)
    if bias == "masks":
        table[3, 0] = -INF                            # the far keys before a row
        table[5:, 1] = -INF                           # the keys behind it
    rows = torch.randint(0, sum(ln), (60 if many else 5,), device="cuda", generator=g)
    cols = torch.randint(0, kw, (len(rows),), device="cuda", generator=g)
    what = torch.tensor([INF, -INF, NAN], device="cuda")[torch.randint(0, 3, (len(rows),), device="cuda", generator=g)]
    qkv[rows, w + kw + cols] = what.to(torch.bfloat16)
    qkv[40, w + kw:w + kw + hd] = NAN                 # a whole value, beside the first sinks
    o, mag = expected(qkv, ln, nq, nkv, hd, span, table)
    out = call(qkv, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=REL if table is not None else None)
    te.check()
    same(f"values not finite {span} {hd} {bias} {many}", out, o, mag)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_a_score_of_minus_infinity_takes_nothing(hd, bias):
    """A key of -inf against positive queries has weight 0, and its value may be anything."""
    import torch
    ln, nq = [300, 130], 2
    w = nq * hd
    qkv = panel(sum(ln), 3 * w, 122)
    qkv[:, 0] = qkv[:, 0].abs() + 1
    table = torch.randn(REL[0], nq, device="cuda") if bias else None
    qkv[100, w] = -INF
    for value in (INF, NAN):
        qkv[100, 2 * w + 5] = value
        see = torch.ones(300, 300, dtype=torch.bool, device="cuda")
        see[:, 100] = False
        which = None
        if bias:
            b = torch.tensor(bucket_table(300, *REL), device="cuda")
            i = torch.arange(300, device="cuda")
            which = b[i[None] - i[:, None] + 299]
        x = qkv[:300].clone()
        x[100, w] = 0
        o, mag = attention_of_finite(x, see, 0, 0, nq, nq, hd, table, which)
        out = call(qkv, ln, nq, nq, hd, -1, -1, 0, hd ** -0.5, table=table, rel=REL if bias else None)
        compare(f"a score of -inf {hd} bias={bias}", out[:300, :hd], o, mag)


@pytest.mark.parametrize("hd", [64, 128])
def test_lost_queries_and_keys(hd):
    """A row of q that is not finite loses itself; one of k every row that sees it; at several rows at once."""
    import torch
    ln, nq, span = [700, 90], 2, (100, 50, 3)
    w = nq * hd
    qkv = panel(sum(ln), 3 * w, 123)
    clean = call(qkv, ln, nq, nq, hd, *span, hd ** -0.5)
    bad = qkv.clone()
    bad[[5, 130, 600], :hd] = NAN                     # queries of head 0
    bad[[77, 400, 430], w + hd:2 * w] = NAN           # keys of head 1
    out = call(bad, ln, nq, nq, hd, *span, hd ** -0.5)
    te.check()
    lost = torch.zeros(790, 2, dtype=torch.bool, device="cuda")
    lost[[5, 130, 600], 0] = True
    see = visible(700, *span, device="cuda")
    lost[:700, 1] = see[:, [77, 400, 430]].any(1)
    for h in range(nq):
        o = out[:, h * hd:(h + 1) * hd]
        assert bool(torch.isnan(o[lost[:, h]].float()).all())
        ref, mag = attention(qkv, ln, nq, nq, hd, *span, hd ** -0.5)
        keep = ~lost[:, h]
        compare(f"beside lost rows {hd}", o[keep], ref[keep, h * hd:(h + 1) * hd], mag[keep, h * hd:(h + 1) * hd])
    assert torch.equal(out[700:], clean[700:])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_among_many_sequences(hd, bias):
    """More blocks than travel with the launch; a wide panel with its heads in another order."""
    import torch
    rng = torch.Generator().manual_seed(124)
    ln = [int(n) for n in torch.randint(1, 40, (690,), generator=rng)] + [600, 1, 257]
    nq, nkv = 4, 2
    w, kw = nq * hd, nkv * hd
    plain = panel(sum(ln), w + 2 * kw, 125)
    rows = torch.randint(0, sum(ln), (200,), generator=rng).cuda()
    plain[rows, w + kw + (rows * 7) % kw] = INF
    plain[rows[:20] // 2 * 2, w + kw + 3] = NAN
    table = torch.randn(REL[0], nq, device="cuda") if bias else None
    if bias:
        table[2:4, 0] = -INF
    span = (20, 5, 2)
    o, mag = expected(plain, ln, nq, nkv, hd, span, table)
    wide = torch.full((sum(ln), w + 2 * kw + 72), NAN, dtype=torch.bfloat16, device="cuda")
    offs = (kw + 8, kw + w + 24, 0)
    for at, (a, b) in zip(offs, ((0, w), (w, w + kw), (w + kw, w + 2 * kw))):
        wide[:, at:at + b - a] = plain[:, a:b]
    out = torch.full((sum(ln) + 3, w + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    call(wide, ln, nq, nkv, hd, *span, hd ** -0.5, table=table, rel=REL if bias else None, offs=offs, out=out)
    te.check()
    same(f"many sequences {hd} bias={bias}", out[:sum(ln), :w], o, mag)
    assert bool((out[sum(ln):] == 7).all()) and bool((out[:, w:] == 7).all())


def test_offsets_past_32_bits():
    """Panels of more than 2^31 values: rows at their end."""
    import torch
    hd, nq, ld = 64, 2, 8200
    rows = (1 << 31) // ld + 3000
    w = nq * hd
    tail = [700, 300, 5]
    lens, start = [rows - 1005] + tail, rows - 1005
    off = ld - 3 * w - 8
    qkv = torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    small = panel(1005, 3 * w, 126)
    small[[100, 130, 800], [2 * w + 5, 2 * w + 70, 2 * w + 9]] = INF
    small[40, 2 * w:] = NAN
    qkv[start:, off:off + 3 * w] = small
    qkv[start - 50, off + 2 * w:off + 3 * w] = NAN    # of the long sequence
    span = (64, 64, 2)
    call(qkv, lens, nq, nq, hd, *span, hd ** -0.5, offs=(off, off + w, off + 2 * w), out=out)
    te.check()
    o, mag = expected(small, tail, nq, nq, hd, span, None)
    same("rows past 2^31 values", out[start:, :w], o, mag)
    seen = torch.isnan(out[:start, :w].float()).all(1).nonzero()[:, 0]
    assert seen.tolist() == list(range(start - 114, start))
