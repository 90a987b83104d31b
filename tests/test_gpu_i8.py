"""The 8-bit activation operators against plain 64-bit arithmetic: te_quant_rows,
te_rownorm_quant, te_i8_linear, te_i8_gated_linear.

Tolerances are bounds on the rounding the operators' definitions allow, per
value: U32 = 2^-24 (half a step of f32), UB = 2^-8 (half a step of bf16).
"""
import math

import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.gpu_util import record_margin, to_np

pytestmark = pytest.mark.gpu

U32, UB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    torch.cuda.init()
    te.lib()
    yield
    te.check()


def _torch():
    import torch
    return torch


def _ratio(got, ref, lim):
    """The largest error over its bound; a value bounded by nothing (a sum that
    is exactly zero) must be met exactly."""
    off = np.abs(got - ref)
    return float(np.where(lim > 0, off / np.where(lim > 0, lim, 1.0), np.where(off == 0, 0.0, np.inf)).max())


# ------------------------------------------------------------------ quantiser

def _quant_ref(v):
    """q and scale of the f32 rows v, step by step in f32 as defined."""
    v = np.asarray(v, dtype=np.float32)
    a = np.abs(v).max(axis=1)
    zero = a < np.float32(2.0 ** -120)
    safe = np.where(zero, np.float32(1), a)
    up = np.float32(127) / safe
    q = np.rint(v * up[:, None])
    return np.where(zero[:, None], 0, q).astype(np.int8), np.where(zero, np.float32(0), safe / np.float32(127))


QUANT_D = [8, 24, 64, 256, 264, 512, 768, 1032, 2048, 3840, 4104, 8200, 10240, 16384]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", QUANT_D)
def test_quant_rows_is_bit_exact(d, dt):
    torch = _torch()
    rng = np.random.default_rng([d, 1])
    t = 1 if d == 64 else 37
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    x = torch.from_numpy((rng.standard_normal((t, d + 8)) * 10.0 ** rng.integers(-3, 4, (t, 1))).astype(np.float32))
    x = x.to(dtype).cuda()[:, :d]                            # rows wider than d
    if t > 5:
        x[1] = 0                                             # a row of nothing
        x[2] = 2.0 ** -125                                   # a row below the smallest scale
        x[3, 0] = -1e30                                      # one value far above the rest
        x[4] = x[4, 0]                                       # all on the same step
    ldq = -(-d // 16) * 16 + 16
    qf = torch.full((t, ldq), 99, dtype=torch.int8, device="cuda")
    s = torch.full((t,), -1.0, device="cuda")
    te.quant_rows(x, qf[:, :d], s)
    te.check()
    q_ref, s_ref = _quant_ref(x.float().cpu().numpy())
    assert np.array_equal(qf[:, :d].cpu().numpy(), q_ref)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), s_ref.astype(np.float32).view(np.uint32))
    assert bool((qf[:, d:] == 99).all())                     # the rows' padding is left alone


def test_quant_rows_confines_values_that_are_not_finite_to_their_row():
    torch = _torch()
    x = torch.randn(9, 520, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[1, 7], x[3, 519], x[5, 0] = math.inf, math.nan, -math.inf
    q = torch.empty(9, 528, dtype=torch.int8, device="cuda")[:, :520]
    s = torch.empty(9, device="cuda")
    te.quant_rows(x, q, s)
    te.check()
    bad = [1, 3, 5]
    good = [r for r in range(9) if r not in bad]
    assert bool(torch.isnan(s[bad]).all()) and not bool(q[bad].any())
    q_ref, s_ref = _quant_ref(x[good].cpu().numpy())
    assert np.array_equal(q[good].cpu().numpy(), q_ref) and np.array_equal(s[good].cpu().numpy(), s_ref)


@pytest.mark.parametrize("kind", [te.TE_NORM_RMS, te.TE_NORM_LN])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,mod,pre", [(8, False, 1.0), (264, True, 1.0), (512, False, 0.5), (768, True, 1.0),
                                       (1536, False, 1.0), (3840, True, 1.0), (5000, False, 1.0),
                                       (16384, False, 1.0)])
def test_rownorm_quant_matches_64_bits(d, mod, pre, dt, kind):
    torch = _torch()
    rng = np.random.default_rng([d, kind])
    t, eps = 19, 1e-6
    x = torch.from_numpy((rng.standard_normal((t, d)) * 3 + 0.5).astype(np.float32))
    x = x.to(torch.float32 if dt == "f32" else torch.bfloat16).cuda()
    w = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    b = (0.1 * rng.standard_normal(d)).astype(np.float32) if kind == te.TE_NORM_LN else None
    m = (0.1 * rng.standard_normal(d)).astype(np.float32) if mod else None
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()
    q = torch.empty(t, -(-d // 16) * 16, dtype=torch.int8, device="cuda")[:, :d]
    s = torch.empty(t, device="cuda")
    te.rownorm_quant(x, dev(w), dev(b), kind, eps, q, s, pre=pre, mod_scale=dev(m))
    te.check()
    v = to_np(x) * pre
    size = np.abs(v).max(axis=1, keepdims=True)
    if kind == te.TE_NORM_LN:
        v = v - v.mean(axis=1, keepdims=True)
    inv = 1 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    v = v * inv * w.astype(np.float64)
    big = size * inv * np.abs(w).max()                       # the size that the f32 steps round at
    if b is not None:
        v = v + b
        big = big + np.abs(b).max()
    if m is not None:
        v = v * (1 + m.astype(np.float64))
        big = big * (1 + np.abs(m).max())
    # A value's relative error: the sum of d squares and the mean, each in a
    # tree of at most 64 + 5 + 8 additions (77 U32), halved by the root for
    # the squares, then rsqrt (2 steps), the products and sums (8 U32): under
    # 200 U32 at the size of the row's largest terms.
    dv = 200 * U32 * big
    a = np.abs(v).max(axis=1, keepdims=True)
    s64 = to_np(s)[:, None]
    assert np.all(np.abs(s64 - a / 127) <= dv / 127 + 2 * U32 * a / 127)
    # half a step of rounding, and what the value and the scale may be off
    off = np.abs(to_np(q) * s64 - v)
    lim = s64 * 0.5 * (1 + 1e-6) + dv + 127 * np.abs(s64 - a / 127) + 4 * U32 * a
    record_margin("rownorm_quant", f"d={d} {dt} kind {kind}", float((off / lim).max()), 1.0)
    assert np.all(off <= lim)
    assert np.all(np.abs(to_np(q)).max(axis=1) == 127)


def test_quant_rows_reads_rows_past_32_bit_offsets():
    torch = _torch()
    t, ld, d = 1100, 1 << 21, 512                            # the last row starts past 2^31 values
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 6 GB")
    x = torch.empty(t * ld, dtype=torch.bfloat16, device="cuda").view(t, ld)[:, :d]
    x.copy_(torch.randn(t, d, device="cuda", generator=torch.Generator("cuda").manual_seed(2)))
    q = torch.empty(t, d, dtype=torch.int8, device="cuda")
    s = torch.empty(t, device="cuda")
    te.quant_rows(x, q, s)
    te.check()
    q_ref, s_ref = _quant_ref(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), q_ref) and np.array_equal(s.cpu().numpy(), s_ref)


# ------------------------------------------------------------------- products

def _tokens(rng, m, k, full=False):
    q = rng.integers(-127, 128, (m, k)).astype(np.int8) if full else \
        np.clip(np.rint(rng.standard_normal((m, k)) * 32), -127, 127).astype(np.int8)
    return q, rng.uniform(0.01, 0.1, m).astype(np.float32)


def _weight(rng, n, k, bias):
    q = rng.integers(-127, 128, (n, k)).astype(np.int8)
    s = (rng.uniform(0.75, 1.25, n) / (127 * math.sqrt(k))).astype(np.float32)
    b = (rng.standard_normal(n) * 0.1).astype(np.float32) if bias else None
    return q, s, b


def _dev(a):
    return None if a is None else _torch().from_numpy(np.ascontiguousarray(a)).cuda()


def _dev_w(w):
    t = tuple(_dev(a) for a in w)
    return te.q8w(*t), t


def _ws(m, k, n):
    torch = _torch()
    return torch.full((max(1, te.i8_workspace(m, k, n)),), 0xA5, dtype=torch.uint8, device="cuda")


def _product(x, xs, w):
    """The exact integer sums, and the product's value in 64 bits without bias."""
    acc = x.astype(np.float64) @ w[0].astype(np.float64).T   # integers below 2^53: exact
    return acc, acc * xs.astype(np.float64)[:, None] * w[1].astype(np.float64)


def _act(g, act):
    if act == te.TE_ACT_SILU:
        return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def _act_slack(g, act):
    """Error of act(g) in f32 over its own value: the exponent t of e^t is off
    by two roundings of |t| (3 U32 |t|), the exponential and reciprocal by two
    steps each (8 U32), the products by 3 U32."""
    t = np.abs(g) if act == te.TE_ACT_SILU else 1.6 * np.abs(g) * (1 + 0.045 * g * g)
    return (3 * t + 11) * U32


LINEAR = [
    # m, k, widths, bias, residual (None, "in", "sep"), out
    (1, 64, [32], False, None, "f32"),
    (1, 512, [512, 512, 512], True, None, "bf16"),
    (2, 3840, [96], True, "in", "f32"),
    (3, 1024, [160, 32], False, "sep", "bf16"),
    (5, 10240, [64], False, None, "f32"),
    (7, 3840, [384, 96, 32, 128], True, None, "bf16"),
    (8, 576, [2048], False, "sep", "f32"),
    (9, 64, [32, 64], True, None, "f32"),
    (15, 1600, [320], False, "in", "f32"),
    (16, 768, [768, 768, 768], True, None, "bf16"),
    (17, 2048, [512], True, "sep", "f32"),
    (31, 256, [1024], False, None, "bf16"),
    (33, 10240, [480], False, None, "f32"),
    (37, 512, [2048, 2048], False, None, "f32"),
    (64, 768, [2304], True, None, "bf16"),
    (65, 1152, [128, 288], True, "in", "f32"),
    (101, 768, [768, 768, 768], True, None, "f32"),
    (128, 4096, [512], False, "sep", "bf16"),
    (129, 128, [96, 160], True, None, "f32"),
    (200, 3840, [3840], False, None, "f32"),
    (257, 320, [640], True, "sep", "f32"),
    (300, 2048, [1024, 1024], False, None, "bf16"),
    (513, 1024, [1536], True, "in", "f32"),
    (777, 768, [768, 768, 768], True, None, "bf16"),
    (1000, 192, [64, 128, 192, 288], True, "in", "f32"),
    (1025, 512, [512], False, None, "f32"),
    (2111, 2048, [3840], False, "in", "f32"),
    (2112, 3840, [3840, 3840, 3840], False, None, "bf16"),
    (3000, 256, [3840, 3840], True, "sep", "f32"),
    (4100, 320, [640], False, None, "bf16"),
    (5000, 512, [512, 512, 512], False, None, "f32"),
    (6001, 448, [1536], False, None, "bf16"),
    (8448, 3840, [3840], False, "in", "f32"),
    # short k, many tokens: weights that stay, runs that cross into the next features
    (3000, 448, [96, 160, 512], True, "in", "f32"),
    (2000, 64, [32], False, "sep", "bf16"),
    (2500, 128, [640], True, None, "bf16"),
    (1100, 320, [96, 32], True, "sep", "f32"),
    (20000, 512, [224], True, None, "f32"),
    (12345, 192, [96, 416], False, None, "bf16"),
]


@pytest.mark.parametrize("m,k,ns,bias,resid,ydt", LINEAR)
def test_i8_linear_matches_64_bits(m, k, ns, bias, resid, ydt):
    torch = _torch()
    rng = np.random.default_rng([m, k, len(ns)])
    x, xs = _tokens(rng, m, k)
    ldx = k + 16 if m % 2 else k
    xd = torch.full((m, ldx), 77, dtype=torch.int8, device="cuda")[:, :k]
    xd.copy_(_dev(x))
    dt = torch.float32 if ydt == "f32" else torch.bfloat16
    items, keep, want = [], [], []
    for n in ns:
        w = _weight(rng, n, k, bias)
        qw, t = _dev_w(w)
        full = torch.full((m + 1, n + 16), float("nan"), dtype=dt, device="cuda")
        y = full[:m, :n]
        it = dict(w=qw, y=y, ldy=n + 16)
        r = rng.standard_normal((m, n)).astype(np.float32) if resid else None
        if resid == "in":
            y.copy_(_dev(r))
            it.update(residual=y, ldr=n + 16)
        elif resid == "sep":
            rd = torch.full((m, n + 8), 3.0, device="cuda")
            rd[:, :n] = _dev(r)
            it.update(residual=rd, ldr=n + 8)
            t += (rd,)
        items.append(it)
        keep.append((t, full))
        want.append((w, r))
    te.i8_linear(xd, _dev(xs), items, _ws(m, k, sum(ns)))
    te.check()
    for i, ((w, r), (_, full)) in enumerate(zip(want, keep)):
        acc, p = _product(x, xs, w)
        assert np.abs(acc).max() < 2 ** 24                   # the f32 sums are exact for these draws
        ref, size = p, np.abs(p)
        if bias:
            ref, size = ref + w[2], size + np.abs(w[2])
        if r is not None:
            ref, size = ref + r, size + np.abs(r)
        # two products, the bias and the residual: one rounding each
        lim = 4 * U32 * size + (UB * np.abs(ref) if ydt == "bf16" else 0)
        got = to_np(full[:m, :w[0].shape[0]])
        assert np.all(np.isfinite(got))
        worst = record_margin("i8_linear", f"m={m} k={k} item {i} {ydt}", _ratio(got, ref, lim), 1.0)
        assert worst <= 1.0
        # the padding of y's rows and the row behind the last token
        assert bool(torch.isnan(full[:m, w[0].shape[0]:]).all()) and bool(torch.isnan(full[m:]).all())


@pytest.mark.parametrize("act", [te.TE_EPI_GELU_TANH, te.TE_EPI_SILU])
@pytest.mark.parametrize("m,k,n,ydt", [(1, 512, 2048, "bf16"), (6, 768, 320, "f32"), (45, 768, 256, "bf16"),
                                       (300, 512, 1024, "f32"), (2500, 768, 768, "bf16"), (2500, 2304, 3840, "f32"),
                                       (2500, 512, 224, "f32"), (1500, 128, 96, "bf16")])
def test_i8_linear_epilogue_activation(m, k, n, ydt, act):
    torch = _torch()
    rng = np.random.default_rng([m, k, n, act])
    x, xs = _tokens(rng, m, k)
    w = _weight(rng, n, k, True)
    qw, keep = _dev_w(w)
    y = torch.full((m, n), float("nan"), dtype=torch.float32 if ydt == "f32" else torch.bfloat16, device="cuda")
    te.i8_linear(_dev(x), _dev(xs), [dict(w=qw, y=y, ldy=n, epilogue=act)], _ws(m, k, n))
    te.check()
    _, p = _product(x, xs, w)
    g = p + w[2]
    ref = _act(g, act - 1)
    dg = 3 * U32 * (np.abs(p) + np.abs(w[2]))                # the value under the activation (slope below 1.13)
    lim = 1.13 * dg + _act_slack(g, act - 1) * np.abs(ref) + 1e-30 + (UB * np.abs(ref) if ydt == "bf16" else 0)
    worst = record_margin("i8_linear act", f"m={m} n={n} {ydt}", _ratio(to_np(y), ref, lim), 1.0)
    assert worst <= 1.0


GATED = [(1, 64, 32), (1, 3840, 160), (4, 512, 2048), (8, 1024, 96), (13, 768, 480), (37, 512, 2048), (64, 256, 64),
         (70, 3840, 1024), (101, 768, 3840), (257, 192, 96), (600, 512, 2048), (1100, 512, 2048), (2112, 1024, 1440),
         (2112, 3840, 2560), (5000, 512, 320), (1500, 64, 32), (3333, 320, 992), (20000, 192, 96)]


@pytest.mark.parametrize("act", [te.TE_ACT_GELU_TANH, te.TE_ACT_SILU])
@pytest.mark.parametrize("m,k,f", GATED)
def test_i8_gated_linear_matches_64_bits(m, k, f, act):
    torch = _torch()
    rng = np.random.default_rng([m, k, f])
    x, xs = _tokens(rng, m, k)
    xs *= 4                                                  # gates on both sides of the activation's bend
    bias = bool(m % 2)
    wg, wu = _weight(rng, f, k, bias), _weight(rng, f, k, bias)
    (qg, kg), (qu, ku) = _dev_w(wg), _dev_w(wu)
    full = torch.full((m + 1, f + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    te.i8_gated_linear(_dev(x), _dev(xs), qg, qu, act, full[:m, :f], _ws(m, k, 2 * f))
    te.check()
    gu, err = [], []
    for w in (wg, wu):
        _, p = _product(x, xs, w)
        gu.append(p + w[2] if bias else p)
        err.append(3 * U32 * (np.abs(p) + (np.abs(w[2]) if bias else 0)))
    g, u = gu
    a = _act(g, act)
    ref = a * u
    da = 1.13 * err[0] + _act_slack(g, act) * np.abs(a)
    lim = da * np.abs(u) + np.abs(a) * err[1] + U32 * np.abs(ref) + UB * np.abs(ref) + 1e-30
    got = to_np(full[:m, :f])
    assert np.all(np.isfinite(got))
    worst = record_margin("i8_gated", f"m={m} k={k} f={f}", _ratio(got, ref, lim), 1.0)
    assert worst <= 1.0
    assert bool(torch.isnan(full[:m, f:]).all()) and bool(torch.isnan(full[m:]).all())


@pytest.mark.parametrize("m", [1, 8, 9, 16, 17, 32, 33, 64, 65, 100, 128, 129, 200, 333, 512, 1000, 1024, 1025, 1999])
@pytest.mark.parametrize("k", [64, 192, 512, 576, 4096])
def test_every_kernel_choice_is_exact_on_integers(m, k):
    # unit scales and an f32 output: the sums themselves, for item widths that
    # end inside a tile, one item and several, plain and gated
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(m * 7 + k)
    x = torch.randint(-60, 61, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    ones = torch.ones(max(m, 4096), device="cuda")
    for ns in ([32], [96, 160, 32], [1600]):
        w = [torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8) for n in ns]
        full = [torch.full((m + 1, n), float("nan"), device="cuda") for n in ns]
        te.i8_linear(x, ones[:m], [dict(w=te.q8w(a, ones[:a.shape[0]]), y=y[:m], ldy=y.shape[1])
                                   for a, y in zip(w, full)], _ws(m, k, sum(ns)))
        for a, y in zip(w, full):
            ref = x.double() @ a.double().T
            assert float(ref.abs().max()) < 2 ** 24
            assert torch.equal(y[:m].double(), ref), (m, k, ns)
            assert bool(torch.isnan(y[m]).all())
    te.check()


@pytest.mark.parametrize("m,k,ns,gated", [(7, 3840, [384, 96], False), (25, 1024, [512], False), (40, 512, [640], True),
                                          (101, 768, [768, 768], False), (200, 2048, [1024], True),
                                          (700, 4096, [256], False), (3000, 512, [512, 96], False),
                                          (2500, 448, [320], True), (2112, 1152, [1024], True)])
def test_repeated_calls_give_the_same_bits(m, k, ns, gated):
    # back to back on one workspace and one set of outputs, other work between
    torch = _torch()
    rng = np.random.default_rng([m, k])
    x, xs = _tokens(rng, m, k, full=True)
    xd, sd, ws = _dev(x), _dev(xs), _ws(m, k, 2 * sum(ns))
    ws_tensors = [_dev_w(_weight(rng, n, k, True)) for n in ns + ns]
    qw = [t[0] for t in ws_tensors]
    dt = torch.bfloat16 if gated else torch.float32
    outs = [torch.empty(m, n, device="cuda", dtype=dt) for n in ns]

    def call():
        if gated:
            te.i8_gated_linear(xd, sd, qw[0], qw[1], te.TE_ACT_GELU_TANH, outs[0], ws)
        else:
            te.i8_linear(xd, sd, [dict(w=w, y=y, ldy=y.shape[1]) for w, y in zip(qw, outs)], ws)

    call()
    first = [y.clone() for y in outs]
    differ = torch.zeros((), device="cuda", dtype=torch.int64)
    for _ in range(60):
        for y in outs:
            y.zero_()
        call()
        for y, f in zip(outs, first):
            differ += (y != f).sum()
    te.check()
    assert int(differ) == 0


def test_calls_on_two_streams_with_workspaces_of_their_own():
    torch = _torch()
    rng = np.random.default_rng(77)
    jobs = []
    for m, k, n in ((3000, 1024, 768), (90, 768, 768), (2500, 512, 512), (5, 2048, 1024)):
        x, xs = _tokens(rng, m, k)
        w = _weight(rng, n, k, True)
        qw, keep = _dev_w(w)
        xd, sd = _dev(x), _dev(xs)
        ref, y = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
        te.i8_linear(xd, sd, [dict(w=qw, y=ref, ldy=n)], _ws(m, k, n))
        jobs.append((xd, sd, qw, keep, ref, y, _ws(m, k, n), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for xd, sd, qw, _, ref, y, ws, s in jobs:
            te.i8_linear(xd, sd, [dict(w=qw, y=y, ldy=y.shape[1])], ws, stream=s)
    torch.cuda.synchronize()
    te.check()
    for *_, ref, y, ws, s in jobs:
        assert torch.equal(y, ref)


@pytest.mark.parametrize("m", [1, 6, 40, 300, 2200])
def test_i8_linear_indexes_every_weight_and_token(m):
    # one-hot tokens pick single weights: any wrong row, column or scale shows, to the bit
    torch = _torch()
    k, n = 448, 352
    rng = np.random.default_rng(m)
    x = np.zeros((m, k), dtype=np.int8)
    hot = rng.integers(0, k, m)
    x[np.arange(m), hot] = rng.integers(1, 128, m)
    x[0, hot[0]] = -128                                      # the one int8 that the quantiser never makes
    q = rng.integers(-128, 128, (n, k)).astype(np.int8)
    ones = torch.ones(max(m, n), device="cuda")
    y = torch.empty(m, n, device="cuda")
    qd = _dev(q)
    te.i8_linear(_dev(x), ones[:m], [dict(w=te.q8w(qd, ones[:n]), y=y, ldy=n)], _ws(m, k, n))
    te.check()
    ref = x[np.arange(m), hot].astype(np.float64)[:, None] * q[:, hot].T
    assert np.array_equal(to_np(y), ref)


@pytest.mark.parametrize("m", [2, 50, 1200])
def test_i8_linear_largest_sums_stay_within_f32_rounding(m):
    # every product at its largest: 16129 k, far past 2^24; an f32 sum in steps
    # of 16 products is off by at most a step (2 U32) of its value each
    torch = _torch()
    k, n = 10240, 96
    x = np.full((m, k), 127, dtype=np.int8)
    q = np.full((n, k), 127, dtype=np.int8)
    q[1::2] = -127
    ones = torch.ones(max(m, n), device="cuda")
    y = torch.empty(m, n, device="cuda")
    qd = _dev(q)                                             # the descriptor holds its address only
    te.i8_linear(_dev(x), ones[:m], [dict(w=te.q8w(qd, ones[:n]), y=y, ldy=n)], _ws(m, k, n))
    te.check()
    ref = x.astype(np.float64) @ q.astype(np.float64).T
    assert np.abs(to_np(y) - ref).max() <= (k / 16) * 2 * U32 * 16129.0 * k


@pytest.mark.parametrize("m", [1, 30, 1500])
def test_i8_linear_of_a_row_that_is_not_finite_or_empty(m):
    # scale NaN (a row the quantiser found not finite) and scale 0 (an empty row)
    torch = _torch()
    k, n = 256, 64
    rng = np.random.default_rng(3)
    x, xs = _tokens(rng, m + 2, k)
    x[0], xs[0] = 0, math.nan
    x[1], xs[1] = 0, 0.0
    w = _weight(rng, n, k, True)
    qw, keep = _dev_w(w)
    y = torch.empty(m + 2, n, device="cuda")
    te.i8_linear(_dev(x), _dev(xs), [dict(w=qw, y=y, ldy=n)], _ws(m + 2, k, n))
    te.check()
    assert bool(torch.isnan(y[0]).all()) and bool(torch.isfinite(y[1:]).all())
    assert np.array_equal(to_np(y[1]), w[2].astype(np.float64))


def test_i8_linear_repeats_to_the_bit_and_per_row():
    # the same bits on every call, and a token's outputs do not depend on the
    # other tokens where the sums are exact
    torch = _torch()
    rng = np.random.default_rng(11)
    k, n = 1024, 512
    x, xs = _tokens(rng, 1300, k)
    w = _weight(rng, n, k, True)
    qw, keep = _dev_w(w)
    xd, sd = _dev(x), _dev(xs)
    out = []
    for m in (1300, 1300, 700, 90, 20, 4, 1):
        y = torch.empty(m, n, device="cuda")
        te.i8_linear(xd[:m], sd[:m], [dict(w=qw, y=y, ldy=n)], _ws(m, k, n))
        out.append(y)
    te.check()
    for y in out[1:]:
        assert torch.equal(y, out[0][:y.shape[0]]), y.shape


@pytest.mark.parametrize("m", [3, 60, 1400])
def test_i8_linear_on_another_stream_and_in_a_graph(m):
    torch = _torch()
    rng = np.random.default_rng(m)
    k, n = 768, 256
    x, xs = _tokens(rng, m, k)
    w = _weight(rng, n, k, False)
    (qw, keep), xd, sd = _dev_w(w), _dev(x), _dev(xs)
    ref = torch.empty(m, n, device="cuda")
    gref = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    ws = _ws(m, k, 2 * n)
    te.i8_linear(xd, sd, [dict(w=qw, y=ref, ldy=n)], ws)
    te.i8_gated_linear(xd, sd, qw, qw, te.TE_ACT_SILU, gref, ws)
    te.check()
    y, g, q, s = torch.zeros_like(ref), torch.zeros_like(gref), torch.zeros_like(xd), torch.zeros_like(sd)
    src = xd.float() * sd[:, None]
    ws2 = _ws(m, k, 2 * n)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        te.i8_linear(xd, sd, [dict(w=qw, y=y, ldy=n)], ws2)
    stream.synchronize()
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        te.i8_linear(xd, sd, [dict(w=qw, y=y, ldy=n)], ws2)
        te.i8_gated_linear(xd, sd, qw, qw, te.TE_ACT_SILU, g, ws2)
        te.quant_rows(src, q, s)
    for _ in range(3):
        for t in (y, g, q, s):
            t.zero_()
        ws2.fill_(0x5A)
        graph.replay()
    te.check()
    assert torch.equal(y, ref) and torch.equal(g, gref)
    assert np.array_equal(q.cpu().numpy(), _quant_ref(src.cpu().numpy())[0])


def test_i8_linear_writes_rows_past_32_bit_offsets():
    torch = _torch()
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 9 GB")
    rng = np.random.default_rng(8)
    k, n, ld = 128, 64, 1 << 21
    for m in (7, 1100):
        x, xs = _tokens(rng, m, k)
        w = _weight(rng, n, k, False)
        qw, keep = _dev_w(w)
        ldy = ld if m > 100 else 1 << 29
        y = torch.empty((m - 1) * ldy + n, dtype=torch.bfloat16, device="cuda")
        y = torch.as_strided(y, (m, n), (ldy, 1))
        te.i8_linear(_dev(x), _dev(xs), [dict(w=qw, y=y, ldy=ldy)], _ws(m, k, n))
        te.check()
        _, ref = _product(x, xs, w)
        assert np.all(np.abs(to_np(y) - ref) <= (UB + 4 * U32) * np.abs(ref))


def test_binding_refuses_tensors_it_would_misread():
    torch = _torch()
    x = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(4, device="cuda")
    qw, keep = _dev_w(_weight(np.random.default_rng(0), 32, 64, False))
    y = torch.zeros(4, 32, device="cuda")
    item = [dict(w=qw, y=y, ldy=32)]
    ws = _ws(4, 64, 32)
    with pytest.raises(TypeError):
        te.i8_linear(x.to(torch.uint8), s, item, ws)
    with pytest.raises(TypeError):
        te.i8_linear(x, s.half(), item, ws)
    with pytest.raises(TypeError):
        te.i8_linear(x, s, [dict(w=qw, y=y.half(), ldy=32)], ws)
    with pytest.raises(ValueError):
        te.i8_linear(x, s[:3], item, ws)
    with pytest.raises(ValueError):
        te.i8_linear(x.t().contiguous().t(), s, item, ws)
    with pytest.raises(ValueError):
        te.i8_linear(x.cpu(), s, item, ws)
    with pytest.raises(TypeError):
        te.quant_rows(y.half(), x[:, :32], s)
    with pytest.raises(ValueError):
        te.quant_rows(torch.zeros(4, 128, device="cuda")[:, ::2], x, s)
