"""Host validation of attention with sinks and relative position bias (no GPU
needed: every call here must fail validation), and the buckets, which are host
work."""
import ctypes
import math

import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.attn_span_ref import bucket_of, visible
from tests.test_abi import FAKE, L, _call  # noqa: F401  (the built library as a fixture)

OUT = 1 << 40       # far from FAKE, so that nothing overlaps


def _args(bias, **over):
    cu = np.asarray(over.pop("cu", [0, 10, 30]), dtype=np.int32)
    a = dict(qkv=FAKE, ld=768, q_off=0, k_off=256, v_off=512, cu=cu.ctypes.data, cu_dev=FAKE, nseq=len(cu) - 1, nq=4,
             nkv=4, hd=64, left=5, right=5, sinks=2, scale=0.125, plan=te.relpos_plan(32, 128), table=FAKE, ldt=4,
             out=OUT, ldo=256)
    a.update(over)
    if isinstance(a["plan"], te.te_relpos):
        a["plan"] = ctypes.byref(a["plan"])
    names = ["qkv", "ld", "q_off", "k_off", "v_off", "cu", "cu_dev", "nseq", "nq", "nkv", "hd", "left", "right", "sinks",
             "scale"] + (["plan", "table", "ldt"] if bias else []) + ["out", "ldo"]
    return [a[n] for n in names] + [None], cu


def _fwd(L, bias, **over):
    args, keep = _args(bias, **over)
    return _call(L, "te_attn_relbias_fwd" if bias else "te_attn_sink_fwd", *args)


@pytest.mark.parametrize("bias", [False, True])
def test_refusals(L, bias):
    for over, want in (
            (dict(qkv=None), te.TE_EINVAL), (dict(out=None), te.TE_EINVAL), (dict(hd=96), te.TE_ESHAPE),
            (dict(hd=32), te.TE_ESHAPE), (dict(nq=0), te.TE_ESHAPE), (dict(nkv=0), te.TE_ESHAPE),
            (dict(nq=4, nkv=3), te.TE_ESHAPE), (dict(nq=65536, nkv=1, ld=1 << 30), te.TE_ESHAPE),
            (dict(left=-2), te.TE_EINVAL), (dict(right=-2), te.TE_EINVAL), (dict(sinks=-1), te.TE_EINVAL),
            (dict(scale=0.0), te.TE_EINVAL), (dict(scale=-0.1), te.TE_EINVAL), (dict(scale=math.nan), te.TE_EINVAL),
            (dict(scale=math.inf), te.TE_EINVAL), (dict(scale=1e-38), te.TE_EINVAL), (dict(scale=1e38), te.TE_EINVAL),
            (dict(ld=760), te.TE_ESHAPE), (dict(q_off=-8), te.TE_ESHAPE), (dict(k_off=520), te.TE_ESHAPE),
            (dict(v_off=-8), te.TE_ESHAPE), (dict(ld=1 << 31), te.TE_ESHAPE), (dict(ldo=248), te.TE_ESHAPE),
            (dict(ldo=1 << 31), te.TE_ESHAPE), (dict(ld=772), te.TE_EALIGN), (dict(ldo=260), te.TE_EALIGN),
            (dict(k_off=260, ld=1024), te.TE_EALIGN), (dict(qkv=FAKE + 8), te.TE_EALIGN),
            (dict(out=OUT + 8), te.TE_EALIGN), (dict(cu=[0, 10, 10]), te.TE_EINVAL), (dict(cu=[1, 10]), te.TE_EINVAL),
            (dict(cu=[0, 10, 5]), te.TE_EINVAL), (dict(cu=[0], nseq=0), te.TE_EINVAL), (dict(cu_dev=None), te.TE_EINVAL),
            (dict(cu_dev=FAKE + 2), te.TE_EALIGN), (dict(cu=[0, (1 << 29) + 1]), te.TE_ESHAPE),
            (dict(out=FAKE + 30 * 768 * 2 - 16), te.TE_EINVAL), (dict(out=FAKE), te.TE_EINVAL)):
        st, msg = _fwd(L, bias, **over)
        assert st == want, (over, st, msg)
        assert msg


def test_refusals_of_the_bias(L):
    for over, want in ((dict(plan=None), te.TE_EINVAL), (dict(table=None), te.TE_EINVAL), (dict(ldt=3), te.TE_ESHAPE),
                       (dict(table=FAKE + 2), te.TE_EALIGN)):
        assert _fwd(L, True, **over)[0] == want, over
    # plans that no te_relpos_init filled
    for field, value in (("buckets", 0), ("buckets", 31), ("buckets", 514), ("two_sided", 2), ("reach", 5000),
                         ("reach", 90), ("buckets", -2)):
        p = te.relpos_plan(32, 128)
        setattr(p, field, value)
        assert _fwd(L, True, plan=p)[0] == te.TE_EINVAL, (field, value)
    p = te.relpos_plan(32, 128)
    p.first[9] = 3
    assert _fwd(L, True, plan=p)[0] == te.TE_EINVAL
    assert _fwd(L, True, plan=te.te_relpos())[0] == te.TE_EINVAL


def test_relpos_init_refusals(L):
    p = te.te_relpos()
    for b, far, two, want in ((3, 10, 1, te.TE_ESHAPE), (2, 10, 1, te.TE_ESHAPE), (5, 10, 1, te.TE_ESHAPE),
                              (1, 10, 0, te.TE_ESHAPE), (514, 2000, 1, te.TE_ESHAPE), (513, 2000, 0, te.TE_ESHAPE),
                              (32, 8, 1, te.TE_ESHAPE), (32, 16, 0, te.TE_ESHAPE), (32, 2049, 1, te.TE_ESHAPE),
                              (32, 0, 1, te.TE_ESHAPE), (32, -1, 1, te.TE_ESHAPE), (32, 128, 2, te.TE_EINVAL),
                              (32, 128, -1, te.TE_EINVAL)):
        p.buckets = 77
        assert _call(L, "te_relpos_init", ctypes.byref(p), b, far, two)[0] == want, (b, far, two)
        assert p.buckets == 77          # left alone
    assert _call(L, "te_relpos_init", None, 32, 128, 1)[0] == te.TE_EINVAL
    assert L.te_relpos_size() == ctypes.sizeof(te.te_relpos)


@pytest.mark.parametrize("buckets,far,two", [(32, 128, True), (32, 128, False), (4, 2, True), (2, 2, False), (3, 2048, False),
                                             (7, 40, False), (320, 800, True), (512, 2048, True), (512, 2048, False),
                                             (512, 257, False), (16, 5, True), (64, 256, True), (36, 2000, True)])
def test_buckets(L, buckets, far, two):
    """Each distance's bucket against the definition, in whole numbers at the borders."""
    p = te.relpos_plan(buckets, far, two)
    side = buckets // 2 if two else buckets
    first = list(p.first)[:side]
    assert p.reach == first[-1] <= far
    for d in range(0, far + 3):
        b = max(i for i in range(side) if first[i] <= d)
        assert b == bucket_of(-d, buckets, far, two), d
    assert bucket_of(5, buckets, far, two) == ((side if two else 0) + (bucket_of(-5, buckets, far, two) if two else 0))


def test_borders_that_are_whole():
    """8 2^(k/2) for 32 two-sided buckets to 128: powers of two are the first of their bucket."""
    assert [bucket_of(-d, 32, 128, True) for d in (7, 8, 11, 12, 15, 16, 31, 32, 63, 64, 127, 128, 10 ** 6)] == \
        [7, 8, 8, 9, 9, 10, 11, 12, 13, 14, 15, 15, 15]
    assert list(te.relpos_plan(32, 128).first)[:16] == [0, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 23, 32, 46, 64, 91]


def test_the_mask_of_the_reference():
    see = visible(6, 1, 0, 2)
    assert see.int().tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0],
                                  [1, 1, 0, 1, 1, 0], [1, 1, 0, 0, 1, 1]]
    assert bool(visible(5, -1, -1, 0).all()) and visible(4, 0, 0, 0).int().sum() == 4


def test_block_attention_refusals(L):
    """What is no descriptor's fault is refused too, before anything is launched."""
    st, msg = _call(L, "te_encoder_block_attn_fwd", None, None, FAKE, FAKE, None, FAKE, 1, FAKE, 0, None)
    assert st == te.TE_EINVAL and "attention" in msg
    a = te.block_attn()
    assert _call(L, "te_encoder_block_attn_fwd", None, ctypes.byref(a), FAKE, FAKE, None, FAKE, 1, FAKE, 0, None)[0] == te.TE_EINVAL


def test_block_attn_checks_its_table():
    torch = pytest.importorskip("torch")
    plan = te.relpos_plan(32, 128)
    for table, err in ((torch.zeros(32, 4), ValueError),                    # not on the device
                       (torch.zeros(32, 4, dtype=torch.float64), TypeError), (torch.zeros(31, 4), ValueError),
                       (torch.zeros(32), ValueError), (torch.zeros(4, 32).T, ValueError)):
        with pytest.raises(err):
            te.block_attn(plan=plan, table=table)
    with pytest.raises(TypeError):
        te.block_attn(plan=object(), table=torch.zeros(32, 4))
    with pytest.raises(ValueError):
        te.block_attn(table=torch.zeros(32, 4))
