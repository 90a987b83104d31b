"""Host validation of the 8-bit activation and multi-axis rotation entry points
(no GPU needed: every call here must fail validation), and the rotation plan,
which is host work."""
import ctypes
import math

import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_abi import FAKE, L, _call  # noqa: F401  (the built library as a fixture)


def _item(n=64, k=128, **over):
    f = dict(q=FAKE, scale=FAKE, bias=None, block_scale=None, col=None, y=FAKE, ldy=n, ydt=te.TE_F32,
             epi=0, resid=None, ldr=0)
    f.update(over)
    w = te.te_q8w(f["q"], f["scale"], f["bias"], n, k, f["block_scale"], f["col"])
    return te.te_q8_item(w, f["y"], f["ldy"], f["ydt"], f["epi"], f["resid"], f["ldr"])


def _linear(L, item=None, x=FAKE, ldx=128, xs=FAKE, m=16, k=128, z=1, ws=FAKE * 16, nb=1 << 30):
    arr = (te.te_q8_item * 1)(item if item is not None else _item())
    return _call(L, "te_i8_linear", x, ldx, xs, m, k, arr, z, ws, nb, None)


def test_i8_linear_rejects_bad_arguments(L):
    assert _linear(L, x=None)[0] == te.TE_EINVAL
    assert _linear(L, xs=None)[0] == te.TE_EINVAL
    assert _linear(L, z=0)[0] == te.TE_ESHAPE
    assert _linear(L, z=5)[0] == te.TE_ESHAPE
    assert _linear(L, m=-1)[0] == te.TE_ESHAPE
    st, msg = _linear(L, k=100)
    assert st == te.TE_ESHAPE and "k=100" in msg
    assert _linear(L, k=65600, ldx=65600)[0] == te.TE_ESHAPE
    assert _linear(L, ldx=64)[0] == te.TE_ESHAPE
    assert _linear(L, ldx=136)[0] == te.TE_ESHAPE            # 8-bit rows off the 16-byte grid
    assert _linear(L, x=FAKE + 8)[0] == te.TE_EALIGN
    assert _linear(L, xs=FAKE + 2)[0] == te.TE_EALIGN
    for bad, st in ((dict(q=None), te.TE_EINVAL), (dict(scale=None), te.TE_EINVAL),
                    (dict(block_scale=FAKE), te.TE_EINVAL), (dict(col=FAKE), te.TE_EINVAL),
                    (dict(k=64), te.TE_ESHAPE), (dict(n=40), te.TE_ESHAPE), (dict(y=None), te.TE_EINVAL),
                    (dict(ydt=7), te.TE_EINVAL), (dict(ldy=32), te.TE_ESHAPE), (dict(ldy=66), te.TE_EALIGN),
                    (dict(y=FAKE + 4), te.TE_EALIGN), (dict(q=FAKE + 4), te.TE_EALIGN),
                    (dict(bias=FAKE + 1), te.TE_EALIGN), (dict(epi=9), te.TE_EINVAL),
                    (dict(epi=te.TE_EPI_SILU, resid=FAKE, ldr=64), te.TE_EINVAL),
                    (dict(resid=FAKE * 2, ldr=32), te.TE_ESHAPE), (dict(resid=FAKE * 2, ldr=66), te.TE_EALIGN),
                    (dict(resid=FAKE, ldr=68), te.TE_EINVAL),
                    (dict(resid=FAKE, ldr=64, ydt=te.TE_BF16), te.TE_EINVAL)):
        assert _linear(L, item=_item(**bad))[0] == st, bad
    need = te.i8_workspace(1000, 128, 64)
    if need:
        assert _linear(L, m=1000, nb=need - 1)[0] == te.TE_EWORKSPACE
        assert _linear(L, m=1000, ws=None, nb=need)[0] == te.TE_EWORKSPACE
        assert _linear(L, m=1000, ws=FAKE * 16 + 16)[0] == te.TE_EALIGN
    # no rows: nothing to do, but the arguments are still looked at
    assert _linear(L, m=0)[0] == te.TE_OK
    assert _linear(L, m=0, item=_item(n=40))[0] == te.TE_ESHAPE


def test_i8_gated_linear_rejects_bad_arguments(L):
    def call(g=None, u=None, act=te.TE_ACT_SILU, out=FAKE, ldm=256, k=128, m=16):
        wg = g or te.te_q8w(FAKE, FAKE, None, 256, 128)
        wu = u or te.te_q8w(FAKE, FAKE, None, 256, 128)
        return _call(L, "te_i8_gated_linear", FAKE, 128, FAKE, m, k, ctypes.byref(wg), ctypes.byref(wu),
                     act, out, ldm, FAKE * 16, 1 << 30, None)
    assert call(act=7)[0] == te.TE_EINVAL
    assert call(out=None)[0] == te.TE_EINVAL
    assert call(out=FAKE + 8)[0] == te.TE_EALIGN
    assert call(ldm=248)[0] == te.TE_ESHAPE
    assert call(k=64)[0] == te.TE_ESHAPE
    assert call(u=te.te_q8w(FAKE, FAKE, None, 192, 128))[0] == te.TE_ESHAPE
    assert call(u=te.te_q8w(FAKE, None, None, 256, 128))[0] == te.TE_EINVAL
    assert call(g=te.te_q8w(FAKE, FAKE, None, 256, 128, None, FAKE))[0] == te.TE_EINVAL
    assert call(m=0)[0] == te.TE_OK


def test_i8_workspace_of_sizes_outside_the_range(L):
    assert te.i8_workspace(-1, 128, 64) == 0 and te.i8_workspace(0, 128, 64) == 0
    assert te.i8_workspace(16, 100, 64) == 0 and te.i8_workspace(16, 128, 0) == 0


def test_quant_rejects_bad_arguments(L):
    def q(x=FAKE, xdt=te.TE_F32, ldx=64, o=FAKE, ldq=64, s=FAKE, t=4, d=64):
        return _call(L, "te_quant_rows", x, xdt, ldx, o, ldq, s, t, d, None)
    assert q(x=None)[0] == q(o=None)[0] == q(s=None)[0] == q(xdt=3)[0] == te.TE_EINVAL
    assert q(t=-1)[0] == q(d=0)[0] == q(d=12)[0] == q(d=16392, ldx=16392, ldq=16400)[0] == te.TE_ESHAPE
    assert q(ldx=32)[0] == q(ldq=48)[0] == te.TE_ESHAPE
    assert q(x=FAKE + 4)[0] == q(o=FAKE + 8)[0] == q(s=FAKE + 2)[0] == te.TE_EALIGN
    assert q(ldx=66)[0] == q(ldq=72)[0] == te.TE_EALIGN
    assert q(t=0)[0] == te.TE_OK

    def n(w=FAKE, b=None, ms=None, kind=te.TE_NORM_RMS, t=4):
        return _call(L, "te_rownorm_quant", FAKE, te.TE_F32, 64, w, b, ms, kind, 1e-6, 1.0, FAKE, 64, FAKE,
                     t, 64, None)
    assert n(w=None)[0] == n(kind=2)[0] == te.TE_EINVAL
    assert n(w=FAKE + 4)[0] == n(b=FAKE + 4)[0] == n(ms=FAKE + 4)[0] == te.TE_EALIGN
    assert n(t=0)[0] == te.TE_OK


def test_rope_axes_plan_is_checked(L):
    assert L.te_rope_axes_size() == ctypes.sizeof(te.te_rope_axes)
    for hd, sec, kw in ((12, (4, 4), {}), (0, (2,), {}), (264, (8,), {}), (64, (), {}), (64, (8,) * 5, {}),
                        (64, (3, 5), {}), (64, (0, 8), {}), (64, (32, 34), {}), (64, (8, 8), {"pairing": 3}),
                        (64, (8, 8), {"theta": 0.0}), (64, (8, 8), {"theta": math.inf}),
                        (64, (8, 8), {"theta": math.nan}), (64, (2, 2), {"freq": [1.0, -1.0]}),
                        (64, (2, 2), {"freq": [1.0, math.nan]})):
        with pytest.raises(te.TEError):
            te.rope_axes_plan(hd, sec, **kw)
    with pytest.raises(ValueError):
        te.rope_axes_plan(64, (4, 4), freq=[1.0])


@pytest.mark.parametrize("whole", [False, True])
def test_rope_axes_plan_holds_the_frequencies_in_turns(whole):
    hd, sec = 72, (24, 6, 30)
    plan = te.rope_axes_plan(hd, sec, theta=10000.0, pairing=te.TE_ROPE_ADJACENT, whole=whole)
    rot, p = sum(sec), 0
    assert (plan.hd, plan.axes, plan.pairs, tuple(plan.sections[:3])) == (hd, 3, rot // 2, sec)
    for a, s in enumerate(sec):
        for i in range(s // 2):
            f = 10000.0 ** (-2.0 * p / rot if whole else -2.0 * i / s)
            # pow, the product and its own rounding: four half steps of an f64, and the truncated word
            assert abs(plan.turn[p] / 2.0 ** 64 - f / (2 * math.pi)) <= 4 * 2.0 ** -53 * f + 2.0 ** -64
            assert plan.axis[p] == a
            p += 1
    own = te.rope_axes_plan(16, (4, 4), freq=[0.5, 0.0, 7.0, 1.0])
    turns = np.array([0.5, 0.0, 7.0, 1.0]) / (2 * math.pi)
    assert np.allclose([t / 2.0 ** 64 for t in own.turn[:4]], turns - np.floor(turns), rtol=0, atol=1e-15)


def test_qk_rope_axes_rejects_bad_arguments(L):
    plan = te.rope_axes_plan(64, (16, 24, 24))

    def call(src=FAKE, lds=256, dst=FAKE * 2, ldd=256, dt=te.TE_BF16, q=0, k=128, nq=2, nkv=2, hd=64,
             qn=None, kn=None, pl=plan, pos=FAKE, ldp=3, rows=4):
        return _call(L, "te_qk_rope_axes", src, lds, dst, ldd, dt, q, k, nq, nkv, hd, qn, kn, 1e-6,
                     ctypes.byref(pl) if pl is not None else None, pos, ldp, 1.0, rows, None)
    assert call(src=None)[0] == call(dst=None)[0] == call(pl=None)[0] == call(pos=None)[0] == te.TE_EINVAL
    assert call(dt=5)[0] == te.TE_EINVAL
    assert call(hd=128)[0] == te.TE_ESHAPE                    # the plan is for another width
    assert call(nq=-1)[0] == call(rows=-1)[0] == call(k=-64)[0] == te.TE_ESHAPE
    assert call(k=192)[0] == call(ldd=248)[0] == call(lds=248)[0] == te.TE_ESHAPE
    assert call(k=64)[0] == te.TE_ESHAPE                      # heads on top of one another
    assert call(ldp=2)[0] == te.TE_ESHAPE
    assert call(dst=FAKE, ldd=512)[0] == te.TE_EINVAL         # in place, other rows
    assert call(qn=FAKE)[0] == te.TE_EINVAL
    assert call(src=FAKE + 8)[0] == call(dst=FAKE * 2 + 8)[0] == te.TE_EALIGN
    assert call(lds=260)[0] == call(q=4, k=136, lds=264, ldd=264)[0] == te.TE_EALIGN
    assert call(qn=FAKE + 4, kn=FAKE)[0] == call(pos=FAKE + 2)[0] == te.TE_EALIGN
    # a plan that nothing has filled, or with an axis it does not have
    assert call(pl=te.te_rope_axes())[0] == te.TE_ESHAPE
    empty = te.te_rope_axes()
    empty.hd = 64
    assert call(pl=empty)[0] == te.TE_EINVAL
    bad = te.rope_axes_plan(64, (16, 24, 24))
    bad.axis[5] = 3
    assert call(pl=bad)[0] == te.TE_EINVAL
    assert call(rows=0)[0] == call(nq=0, nkv=0)[0] == te.TE_OK


def test_the_binding_refuses_what_is_not_a_tensor_on_the_device(L):
    # the marshalling module's own checks, before any CUDA call
    import torch
    x, s, q = torch.zeros(2, 64), torch.zeros(2), torch.zeros(2, 64, dtype=torch.int8)
    with pytest.raises(ValueError, match="current CUDA device"):
        te.quant_rows(x, q, s)
    with pytest.raises(TypeError, match="dtype"):
        te.quant_rows(x.double(), q, s)
    with pytest.raises(TypeError, match="not a tensor"):
        te.quant_rows(3, q, s)
    with pytest.raises(ValueError, match="current CUDA device"):
        te.i8_linear(q, s, [], None)
    plan = te.rope_axes_plan(64, (16, 24, 24))
    with pytest.raises(ValueError, match="current CUDA device"):
        te.qk_rope_axes(x, 64, x, 64, 0, 0, 1, 0, 64, None, None, 1e-6, plan, q, 1.0, 2)
    with pytest.raises(OverflowError):
        te.qk_rope_axes(x, 64, x, 64, 0, 0, 1, 0, 64, None, None, 1e-6, plan, q, 1.0, 1 << 40)


def test_qk_rope_axes_rejects_a_plan_of_heads_out_of_range(L):
    # fields that hold together, of a head wider than the kernels index
    plan = te.te_rope_axes()
    plan.hd, plan.axes, plan.pairs, plan.pairing = 512, 1, 256, te.TE_ROPE_ADJACENT
    plan.sections[0] = 512
    args = [FAKE, 512, FAKE * 16, 512, te.TE_F32, 0, 0, 1, 0, 512, None, None, 1e-6, ctypes.byref(plan), FAKE, 1, 1.0, 1,
            None]
    assert _call(L, "te_qk_rope_axes", *args)[0] == te.TE_EINVAL
    plan.hd, plan.pairs, plan.sections[0] = 12, 6, 12         # not a multiple of 8
    args[1] = args[3] = args[9] = 12
    assert _call(L, "te_qk_rope_axes", *args)[0] == te.TE_EINVAL


def test_no_rows_need_no_memory(L):
    assert _linear(L, x=None, xs=None, m=0, item=_item(y=None))[0] == te.TE_OK
    assert _linear(L, x=None, m=1)[0] == te.TE_EINVAL
    w = te.te_q8w(FAKE, FAKE, None, 64, 128, None, None)
    assert _call(L, "te_i8_gated_linear", None, 128, None, 0, 128, ctypes.byref(w), ctypes.byref(w), te.TE_ACT_SILU, None, 64,
                 None, 0, None)[0] == te.TE_OK
    assert _call(L, "te_quant_rows", None, te.TE_F32, 64, None, 64, None, 0, 64, None)[0] == te.TE_OK
    assert _call(L, "te_rownorm_quant", None, te.TE_F32, 64, FAKE, None, None, te.TE_NORM_RMS, 1e-6, 1.0, None, 64, None, 0,
                 64, None)[0] == te.TE_OK
    plan = te.rope_axes_plan(64, (16, 24, 24))
    assert _call(L, "te_qk_rope_axes", None, 128, None, 128, te.TE_BF16, 0, 64, 1, 1, 64, None, None, 1e-6,
                 ctypes.byref(plan), None, 3, 1.0, 0, None)[0] == te.TE_OK


def test_i8_products_reject_rows_whose_tiles_pass_an_int(L):
    assert _linear(L, m=0x7FFFFFFF)[0] == te.TE_ESHAPE
    assert te.i8_workspace(0x7FFFFFFF, 128, 64) == 0
