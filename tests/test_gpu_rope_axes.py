"""te_qk_rope_axes against plain 64-bit arithmetic, and the block's way through
the 8-bit activation operators (norm + quantise, products, rotation, attention)."""
import math

import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.gpu_util import record_margin, to_np
from tests.test_gpu_i8 import _act, _dev, _dev_w, _product, _ratio, _weight, _ws

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


def pair_layout(hd, sections, pairing, whole, theta=10000.0):
    """(first channel, second channel, axis, frequency) of each pair."""
    rot, p, start, out = sum(sections), 0, 0, []
    for a, sec in enumerate(sections):
        for i in range(sec // 2):
            if pairing == te.TE_ROPE_SECTION_HALVES:
                c = (start + i, start + i + sec // 2)
            elif pairing == te.TE_ROPE_HEAD_HALVES:
                c = (p, p + rot // 2)
            else:
                c = (2 * p, 2 * p + 1)
            out.append((*c, a, theta ** (-2.0 * p / rot if whole else -2.0 * i / sec)))
            p += 1
        start += sec
    return out


def rope_ref(x, hd, nq, layout, pos, qn, kn, eps, q_mul):
    """x [rows, heads, hd] in f64 -> (result, bound on an f32 evaluation's error).

    The bound, at the size (|x1| + |x2|) mul of a pair: the angle's fraction
    is one f32 rounding of a half turn (U32 pi), sine and cosine two steps
    (4 U32), the two products and the sum 3 U32, the multiplication by q_mul
    one, and with a norm the f32 sum of hd squares (hd/8 + 5 additions, halved
    by the root), rsqrt (two steps) and two products: 16 U32 in all without,
    16 + hd/16 + 10 with a norm."""
    x = x.copy()
    slack = 16.0
    if qn is not None:
        x = x / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps)
        x[:, :nq] *= qn
        x[:, nq:] *= kn
        slack += hd / 16 + 10
    y, size = x.copy(), np.abs(x)
    for c1, c2, a, f in layout:
        # the angle in 64 bits: positions here stay below 2^31, off by 2^-53 of the angle
        ang = pos[:, a].astype(np.float64) * f
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y[:, :, c1] = x[:, :, c1] * c - x[:, :, c2] * s
        y[:, :, c2] = x[:, :, c2] * c + x[:, :, c1] * s
        both = np.abs(x[:, :, c1]) + np.abs(x[:, :, c2])
        size[:, :, c1] = size[:, :, c2] = both
    y[:, :nq] *= q_mul
    size[:, :nq] *= abs(q_mul)
    return y, slack * U32 * size


CASES = [
    # rows, nq, nkv, hd, sections, pairing, whole, norm, dtype, furthest position
    (1, 8, 8, 64, (16, 24, 24), 1, True, True, "bf16", 50),
    (1, 1, 0, 8, (2,), 0, False, False, "f32", 3),
    (3, 2, 1, 16, (2, 4, 6), 2, False, True, "bf16", 100),
    (33, 12, 4, 72, (24, 24, 16), 1, True, False, "f32", 900),
    (33, 12, 4, 72, (18, 26, 28), 0, False, True, "bf16", 900),
    (50, 3, 3, 80, (10, 6, 22, 42), 2, True, True, "f32", 5000),
    (64, 30, 30, 128, (32, 48, 48), 0, False, True, "bf16", 64),
    (65, 30, 30, 128, (44, 42, 42), 2, False, True, "bf16", 40000),
    (65, 30, 30, 128, (44, 42, 42), 1, False, False, "f32", 40000),
    (129, 5, 1, 96, (32, 32, 32), 2, True, False, "bf16", 100000),
    (40, 4, 2, 256, (64, 96, 96), 0, False, True, "f32", 2000),
    (40, 4, 2, 256, (62, 98, 90), 1, True, True, "bf16", 2000),
    (40, 4, 2, 256, (128, 128), 2, True, False, "bf16", 2000),
    (300, 8, 8, 64, (64,), 0, False, True, "bf16", 300),
    (77, 7, 1, 40, (8, 16, 16), 0, False, True, "f32", 10),
    (77, 7, 1, 136, (40, 48, 48), 0, False, True, "bf16", 10),
    (77, 7, 1, 136, (40, 48, 48), 2, False, False, "f32", 10),
    (1000, 64, 8, 128, (16, 24, 24), 1, True, True, "bf16", 1 << 20),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows,nq,nkv,hd,sections,pairing,whole,norm,dt,far", CASES)
def test_qk_rope_axes_matches_64_bits(rows, nq, nkv, hd, sections, pairing, whole, norm, dt, far, in_place):
    torch = _torch()
    rng = np.random.default_rng([rows, hd, pairing, in_place])
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    # k heads in front of the q heads, a gap between, rows wider than the heads
    k_off, q_off = 16, 16 + nkv * hd + 8
    width = q_off + nq * hd + 24
    x = torch.from_numpy(rng.standard_normal((rows, width)).astype(np.float32)).to(dtype)
    pos = rng.integers(-far, far + 1, (rows, len(sections))).astype(np.int32)
    qn = (1 + 0.1 * rng.standard_normal(hd)).astype(np.float32) if norm else None
    kn = (1 + 0.1 * rng.standard_normal(hd)).astype(np.float32) if norm else None
    q_mul = 0.3
    src = x.cuda()
    ldd = width if in_place else width + 8
    dst = src if in_place else torch.full((rows + 1, ldd), 7.0, dtype=dtype, device="cuda")
    plan = te.rope_axes_plan(hd, sections, pairing=pairing, whole=whole)
    posd = torch.full((rows, len(sections) + 1), 1 << 30, dtype=torch.int32, device="cuda")[:, :len(sections)]
    posd.copy_(torch.from_numpy(pos))
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()
    te.qk_rope_axes(src, width, dst[:rows], ldd, q_off, k_off, nq, nkv, hd, dev(qn), dev(kn), 1e-6, plan, posd,
                    q_mul, rows)
    te.check()
    x64 = x.double().numpy()
    heads = np.concatenate([x64[:, q_off:q_off + nq * hd].reshape(rows, nq, hd),
                            x64[:, k_off:k_off + nkv * hd].reshape(rows, nkv, hd)], axis=1)
    layout = pair_layout(hd, sections, pairing, whole)
    ref, lim = rope_ref(heads, hd, nq, layout, pos, qn, kn, 1e-6, q_mul)
    # far positions: the frequency word is within 4 steps of an f64, far * 2^-51 radians
    lim = lim + 2.0 ** -51 * far * 8 + (UB * np.abs(ref) if dt == "bf16" else 0)
    out = to_np(dst)
    got = np.concatenate([out[:rows, q_off:q_off + nq * hd].reshape(rows, nq, hd),
                          out[:rows, k_off:k_off + nkv * hd].reshape(rows, nkv, hd)], axis=1)
    worst = record_margin("qk_rope_axes", f"rows={rows} hd={hd} {dt}", _ratio(got, ref, lim), 1.0)
    assert worst <= 1.0
    # columns without a head, and rows behind the last
    other = np.ones(out.shape[1], dtype=bool)
    other[q_off:q_off + nq * hd] = other[k_off:k_off + nkv * hd] = False
    if in_place:
        assert np.array_equal(out[:, other], x64[:, other])
    else:
        assert np.all(out[:rows, other] == 7.0) and np.all(out[rows:] == 7.0)


@pytest.mark.parametrize("hd,sections", [(64, (64,)), (64, (32, 32)), (128, (64, 64))])
def test_equal_sections_agree_with_the_table_form(hd, sections):
    # te_qk_prep_rope's 1-D and 2-D rotation from its tables, on the same positions
    torch = _torch()
    rng = np.random.default_rng(hd)
    rows, nq, nkv = 90, 4, 4
    width = 3 * nq * hd
    x = torch.from_numpy(rng.standard_normal((rows, width)).astype(np.float32)).bfloat16().cuda()
    pos = rng.integers(0, 200, (rows, len(sections))).astype(np.int32)
    half = sections[0] // 2
    ang = np.concatenate([pos[:, a:a + 1] * 10000.0 ** (-2.0 * np.arange(half) / sections[0])
                          for a in range(len(sections))], axis=1)
    cos, sin = (torch.from_numpy(f(ang).astype(np.float32)).cuda() for f in (np.cos, np.sin))
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal((2, hd))).astype(np.float32)).cuda()
    a, b = x.clone(), x.clone()
    te.qk_prep_rope(a, width, 0, nq * hd, nq, nkv, hd, w[0], w[1], 1e-6, cos, sin, None, sections[0], 0.5, rows)
    te.qk_rope_axes(b, width, b, width, 0, nq * hd, nq, nkv, hd, w[0], w[1], 1e-6, te.rope_axes_plan(hd, sections),
                    torch.from_numpy(pos).cuda(), 0.5, rows)
    te.check()
    # both within half a bf16 step (and f32 roundings, 64 U32 of the pair) of the same value
    a64, b64 = to_np(a), to_np(b)
    assert np.all(np.abs(a64 - b64) <= 2 * UB * np.maximum(np.abs(a64), np.abs(b64)) + 128 * U32 * 8)


def test_far_and_negative_positions_keep_the_angle():
    # the last int32 positions: the 64-bit angle is the definition's, exactly reduced
    torch = _torch()
    hd = 64
    freq = [1.0 / (i + 1) for i in range(32)]
    pos = np.array([[2 ** 31 - 1], [-2 ** 31], [2 ** 30 + 12345], [0]], dtype=np.int32)
    x = torch.zeros(4, hd, device="cuda")
    x[:, :32] = 1.0
    y = torch.empty_like(x)
    plan = te.rope_axes_plan(hd, (64,), freq=freq)
    te.qk_rope_axes(x, hd, y, hd, 0, 0, 1, 0, hd, None, None, 1e-6, plan, torch.from_numpy(pos).cuda(), 1.0, 4)
    te.check()
    got = to_np(y)
    for r, p in enumerate(pos[:, 0]):
        for i, f in enumerate(freq):
            turns = f / (2 * math.pi)
            word = int(math.ldexp(turns - math.floor(turns), 64))
            assert abs(word - plan.turn[i]) <= 2 ** 13
            frac = ((int(p) * int(plan.turn[i])) % 2 ** 64) / 2.0 ** 64
            assert abs(got[r, i] - math.cos(2 * math.pi * frac)) <= 16 * U32
            assert abs(got[r, 32 + i] - math.sin(2 * math.pi * frac)) <= 16 * U32


def test_infinities_and_nans_stay_in_their_head():
    torch = _torch()
    rows, nq, hd = 6, 3, 64
    plan = te.rope_axes_plan(hd, (16, 24, 24))
    pos = torch.arange(18, dtype=torch.int32, device="cuda").view(rows, 3)
    x = torch.randn(rows, 2 * nq * hd, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    w = torch.ones(hd, device="cuda")
    bad = x.clone()
    bad[2, 70], bad[4, 3 * hd + 5] = math.nan, math.inf
    y, z = torch.empty_like(x), torch.empty_like(x)
    args = (0, nq * hd, nq, nq, hd, w, w, 1e-6, plan, pos, 1.0, rows)
    te.qk_rope_axes(x, 2 * nq * hd, y, 2 * nq * hd, *args)
    te.qk_rope_axes(bad, 2 * nq * hd, z, 2 * nq * hd, *args)
    te.check()
    same = (y == z).view(rows, 2 * nq, hd).all(2).cpu().numpy()
    want = np.ones((rows, 2 * nq), dtype=bool)
    want[2, 1] = want[4, 3] = False
    assert np.array_equal(same, want)


def test_rows_past_32_bit_offsets():
    torch = _torch()
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 5 GB")
    rows, ld, hd = 1100, 1 << 21, 64
    x = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)
    x[:, :2 * hd] = torch.randn(rows, 2 * hd, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    small = x[:, :2 * hd].clone()
    pos = torch.arange(3 * rows, dtype=torch.int32, device="cuda").view(rows, 3)
    plan = te.rope_axes_plan(hd, (16, 24, 24))
    te.qk_rope_axes(x, ld, x, ld, 0, hd, 1, 1, hd, None, None, 1e-6, plan, pos, 1.0, rows)
    te.qk_rope_axes(small, 2 * hd, small, 2 * hd, 0, hd, 1, 1, hd, None, None, 1e-6, plan, pos, 1.0, rows)
    te.check()
    assert torch.equal(x[:, :2 * hd], small)


def test_graph_replay_and_another_stream():
    torch = _torch()
    rows, nq, hd = 200, 8, 128
    width = 2 * nq * hd
    plan = te.rope_axes_plan(hd, (32, 48, 48))
    pos = torch.arange(3 * rows, dtype=torch.int32, device="cuda").view(rows, 3)
    x = torch.randn(rows, width, device="cuda", generator=torch.Generator("cuda").manual_seed(6)).bfloat16()
    ref, y = torch.empty_like(x), torch.zeros_like(x)
    args = (0, nq * hd, nq, nq, hd, None, None, 1e-6, plan, pos, 1.0, rows)
    te.qk_rope_axes(x, width, ref, width, *args)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        te.qk_rope_axes(x, width, y, width, *args)
    graph.replay()
    te.check()
    assert torch.equal(y, ref)


def test_binding_refuses_tensors_it_would_misread():
    torch = _torch()
    plan = te.rope_axes_plan(64, (16, 24, 24))
    x = torch.zeros(4, 128, device="cuda")
    pos = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    call = lambda s=x, d=x, p=pos: te.qk_rope_axes(s, 128, d, 128, 0, 64, 1, 1, 64, None, None, 1e-6, plan, p, 1.0, 4)
    call()
    with pytest.raises(TypeError):
        call(s=x.half(), d=x.half())
    with pytest.raises(TypeError):
        call(d=x.bfloat16())
    with pytest.raises(TypeError):
        call(p=pos.long())
    with pytest.raises(ValueError):
        call(p=pos[:, :2])
    with pytest.raises(ValueError):
        call(s=x.cpu())
    te.check()


# ------------------------------------------------------------ a run of them all

def test_the_block_with_8_bit_activations_on_a_video_grid():
    """Pre-norm + quantise -> q|k|v -> norm + 3-axis rotation -> attention ->
    quantise -> out projection into the residual -> norm + quantise -> gate|up
    -> quantise -> down into the residual: each step against 64 bits on the
    inputs it got, as the other block tests teacher-force theirs."""
    torch = _torch()
    rng = np.random.default_rng(21)
    d, H, hd, F, eps = 512, 4, 128, 1024, 1e-6
    grid, sections = (3, 6, 8), (32, 48, 48)
    lens = [int(np.prod(grid)), 45]                          # a clip and a caption
    T = sum(lens)
    cu = np.array([0, lens[0], T], dtype=np.int32)
    t, h, w_ = np.meshgrid(*(np.arange(n) for n in grid), indexing="ij")
    pos = np.stack([t.ravel(), h.ravel(), w_.ravel()], 1)
    cap = np.repeat(np.arange(lens[1])[:, None], 3, 1)
    pos = torch.from_numpy(np.concatenate([pos, cap]).astype(np.int32)).cuda()
    norm = [(1 + 0.1 * rng.standard_normal(n)).astype(np.float32) for n in (d, d, hd, hd)]
    ws = {n: _weight(rng, o, i, False) for n, o, i in (("q", d, d), ("k", d, d), ("v", d, d), ("o", d, d),
                                                       ("g", F, d), ("u", F, d), ("d", d, F))}
    dev = {n: _dev_w(w) for n, w in ws.items()}
    qw = {n: p[0] for n, p in dev.items()}
    x = _dev(rng.standard_normal((T, d)).astype(np.float32))
    a8, as_ = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    m8 = torch.empty(T, F, dtype=torch.int8, device="cuda")
    scratch = _ws(T, max(d, F), 2 * F + 3 * d)
    qkv = torch.empty(T, 3 * d, dtype=torch.bfloat16, device="cuda")
    items = [dict(w=qw[n], y=qkv[:, i * d:(i + 1) * d], ldy=3 * d) for i, n in enumerate("qkv")]
    plan = te.rope_axes_plan(hd, sections, theta=256.0)
    o = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    m = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    cu_dev = torch.from_numpy(cu).cuda()

    def q64(q, s):
        return q.cpu().numpy().astype(np.int8), s.cpu().numpy()

    x0 = to_np(x)
    te.rownorm_quant(x, _dev(norm[0]), None, te.TE_NORM_RMS, eps, a8, as_)
    te.i8_linear(a8, as_, items, scratch)
    pre = qkv.clone()
    te.qk_rope_axes(qkv, 3 * d, qkv, 3 * d, 0, d, H, H, hd, _dev(norm[2]), _dev(norm[3]), eps, plan, pos, 1.0, T)
    te.attn_varlen_fwd(qkv, 3 * d, 0, d, 2 * d, cu, cu_dev, H, H, hd, 0, hd ** -0.5, o, d)
    a_in = q64(a8, as_)
    te.quant_rows(o, a8, as_)
    te.i8_linear(a8, as_, [dict(w=qw["o"], y=x, ldy=d, residual=x, ldr=d)], scratch)
    o_in, x1 = q64(a8, as_), to_np(x)
    te.rownorm_quant(x, _dev(norm[1]), None, te.TE_NORM_RMS, eps, a8, as_)
    te.i8_gated_linear(a8, as_, qw["g"], qw["u"], te.TE_ACT_SILU, m, scratch)
    f_in, m64 = q64(a8, as_), to_np(m)
    te.quant_rows(m, m8, as_)
    te.i8_linear(m8, as_, [dict(w=qw["d"], y=x, ldy=d, residual=x, ldr=d)], scratch)
    te.check()

    def rel(got, ref):
        return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))

    v = x0 / np.sqrt((x0 * x0).mean(1, keepdims=True) + eps) * norm[0]
    step = np.abs(v).max(1, keepdims=True) / 127
    assert np.all(np.abs(a_in[0] * a_in[1][:, None].astype(np.float64) - v) <= 0.5001 * step)
    for i, n in enumerate("qkv"):
        assert rel(to_np(pre[:, i * d:(i + 1) * d]), _product(*a_in, ws[n])[1]) <= UB
    heads = to_np(pre)[:, :2 * d].reshape(T, 2 * H, hd)
    layout = pair_layout(hd, sections, te.TE_ROPE_SECTION_HALVES, False, theta=256.0)
    ref, lim = rope_ref(heads, hd, H, layout, pos.cpu().numpy(), norm[2], norm[3], eps, 1.0)
    got = to_np(qkv)[:, :2 * d].reshape(T, 2 * H, hd)
    assert np.all(np.abs(got - ref) <= lim + UB * np.abs(ref))
    p64 = to_np(qkv).reshape(T, 3, H, hd)
    for s in range(2):
        rows = slice(cu[s], cu[s + 1])
        qq, kk, vv = (p64[rows, i].transpose(1, 0, 2) for i in range(3))
        sc = qq @ kk.transpose(0, 2, 1) * hd ** -0.5
        e = np.exp(sc - sc.max(2, keepdims=True))
        ref = ((e / e.sum(2, keepdims=True)) @ vv).transpose(1, 0, 2).reshape(-1, d)
        # P and the output are each rounded to bf16
        assert rel(to_np(o[rows]), ref) <= 2 * UB
    assert rel(x1, x0 + _product(*o_in, ws["o"])[1]) <= 16 * U32
    g, u = _product(*f_in, ws["g"])[1], _product(*f_in, ws["u"])[1]
    assert rel(m64, _act(g, te.TE_ACT_SILU) * u) <= UB
    d_in = q64(m8, as_)
    assert rel(to_np(x), x1 + _product(*d_in, ws["d"])[1]) <= 16 * U32


@pytest.mark.parametrize("rows,nq,nkv,hd,dt", [(2600, 20, 10, 256, "bf16"), (5000, 16, 14, 128, "bf16"),
                                               (5003, 13, 13, 104, "bf16"), (3700, 17, 12, 256, "f32"),
                                               (9001, 16, 15, 128, "bf16")])
def test_rows_are_turned_alike_however_many_there_are(rows, nq, nkv, hd, dt):
    # many rows, whose last ones are cut finer, against a few at a time: the same bits
    torch = _torch()
    t = torch.float32 if dt == "f32" else torch.bfloat16
    gen = torch.Generator("cuda").manual_seed(rows)
    w = (nq + nkv) * hd
    x = torch.randn(rows, w, device="cuda", generator=gen).to(t)
    qn, kn = torch.rand(hd, device="cuda", generator=gen), torch.rand(hd, device="cuda", generator=gen)
    pos = torch.randint(-500, 500, (rows, 2), dtype=torch.int32, device="cuda", generator=gen)
    plan = te.rope_axes_plan(hd, (hd // 2, hd // 2))
    a, b = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    te.qk_rope_axes(x, w, a, w, 0, nq * hd, nq, nkv, hd, qn, kn, 1e-6, plan, pos, 0.5, rows)
    for r in range(0, rows, 400):
        n = min(400, rows - r)
        te.qk_rope_axes(x[r:r + n], w, b[r:r + n], w, 0, nq * hd, nq, nkv, hd, qn, kn, 1e-6, plan, pos[r:r + n], 0.5, n)
    assert not bool(torch.isnan(a.float()).any())
    assert torch.equal(a, b)
    te.check()
