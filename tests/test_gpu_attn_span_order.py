"""te.attn_sink_fwd and te.attn_relbias_fwd among other calls: the work before and
behind them in a stream, other streams, threads, captured graphs, far offsets,
and device tables that are not the host's."""
import threading

import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.attn_span_ref import attention, bound
from tests.test_gpu_attn_span import call, compare, offsets, panel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    torch.cuda.init()
    te.lib()
    yield
    te.check()


class Chain:
    """A panel that a rotation fills, the attention, and a quantisation of its
    output: each may start while the one before it ends."""

    def __init__(self, hd, lens, seed, stream=None):
        import torch
        self.hd, self.lens, self.stream = hd, lens, stream
        self.nq = 128 // hd * 2
        t = sum(lens)
        self.src = [panel(t, 3 * self.nq * hd, seed + i) for i in range(3)]
        self.qkv = torch.zeros_like(self.src[0])
        self.out = torch.zeros(t, self.nq * hd, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(t, self.nq * hd, dtype=torch.int8, device="cuda")
        self.s = torch.zeros(t, device="cuda")
        self.cu, self.cu_dev = offsets(lens)
        self.plan = te.rope_axes_plan(hd, (hd,))
        self.pos = torch.arange(t, dtype=torch.int32, device="cuda").reshape(t, 1)
        self.rel = te.relpos_plan(32, 128)
        self.table = torch.randn(32, self.nq, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))

    def attend(self, bias):
        n = self.nq * self.hd
        args = (self.qkv, 3 * n, 0, n, 2 * n, self.cu, self.cu_dev, self.nq, self.nq, self.hd, 50, 50, 3, self.hd ** -0.5)
        if bias:
            te.attn_relbias_fwd(*args, self.rel, self.table, self.out, n, stream=self.stream)
        else:
            te.attn_sink_fwd(*args, self.out, n, stream=self.stream)

    def run(self, i, apart=False):
        import torch
        n = self.nq * self.hd
        t = sum(self.lens)
        steps = [lambda: self.qkv[:, 2 * n:].copy_(self.src[i][:, 2 * n:]),
                 lambda: te.qk_rope_axes(self.src[i], 3 * n, self.qkv, 3 * n, 0, n, self.nq, self.nq, self.hd, None, None,
                                         1e-6, self.plan, self.pos, 1.0, t, stream=self.stream),
                 lambda: self.attend(i % 2 == 0),
                 lambda: te.quant_rows(self.out, self.q, self.s, stream=self.stream)]
        for f in steps:
            f()
            if apart:
                torch.cuda.synchronize()

    def outputs(self):
        return self.out.clone(), self.q.clone(), self.s.clone()

    def expected(self):
        got = []
        for i in range(3):
            self.run(i, apart=True)
            got.append(self.outputs())
        return got


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("lens", [[37, 64], [900, 300, 1, 500] * 3])
def test_order_in_a_stream(hd, lens):
    import torch
    c = Chain(hd, lens, 21)
    want = c.expected()
    for _ in range(10):
        got = []
        for i in range(3):
            c.run(i)
            got.append(c.outputs())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("hd", [64, 128])
def test_captured_and_replayed(hd):
    """A graph of the chain, replayed with other inputs; an eager call between two replays."""
    import torch
    c = Chain(hd, [300, 64, 129], 22)
    want = c.expected()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(0)
    for i in (0, 2, 0):
        if i == 2:
            c.run(1)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(c.outputs(), want[1]))
        keep = c.src[0].clone()
        c.src[0].copy_(c.src[i])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.outputs(), want[i]))
        c.src[0].copy_(keep)


def test_other_streams():
    """Work of another stream joined by an event, and two streams at once."""
    import torch
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        ca = Chain(64, [700, 33, 250], 23, a)
    with torch.cuda.stream(b):
        cb = Chain(128, [500, 300], 24, b)
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        wa = ca.expected()
    with torch.cuda.stream(b):
        wb = cb.expected()
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(3):
            with torch.cuda.stream(a):
                ca.run(i)
                ga = ca.outputs()
            with torch.cuda.stream(b):
                cb.run(i)
                gb = cb.outputs()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(ga, wa[i])) and all(torch.equal(x, y) for x, y in zip(gb, wb[i]))


def test_beside_products():
    """Beside products whose clusters hold TMEM while they wait for one another."""
    import torch
    s = torch.cuda.Stream()
    c = Chain(64, [1500, 700, 200], 25)
    want = c.expected()
    m, k, n = 101, 768, 768
    x = torch.randint(-127, 128, (m, k), dtype=torch.int8, device="cuda")
    xs = torch.rand(m, device="cuda")
    w, ws = torch.randint(-127, 128, (3, n, k), dtype=torch.int8, device="cuda"), torch.rand(3, n, device="cuda")
    y = torch.zeros(3, m, n, device="cuda")
    items = [dict(w=te.q8w(w[i], ws[i]), y=y[i], ldy=n) for i in range(3)]
    room = torch.empty(max(256, te.i8_workspace(m, k, 3 * n)), dtype=torch.uint8, device="cuda")
    te.i8_linear(x, xs, items, room)
    torch.cuda.synchronize()
    first = y.clone()
    for i in range(60):
        with torch.cuda.stream(s):
            te.i8_linear(x, xs, items, room)
        c.attend(True)
        c.attend(False)
    torch.cuda.synchronize()
    te.check()
    assert torch.equal(y, first)
    c.run(0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(c.outputs(), want[0]))


def test_threads():
    import torch
    chains = [Chain(hd, lens, 30 + i) for i, (hd, lens) in enumerate([(64, [300, 5]), (128, [200, 77]), (64, [64] * 9)])]
    want = [c.expected() for c in chains]
    torch.cuda.synchronize()
    bad = []

    def work(c, w):
        st = torch.cuda.Stream()
        c.stream = st
        with torch.cuda.stream(st):
            for r in range(20):
                c.run(r % 3)
                got = c.outputs()
                st.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, w[r % 3])):
                    bad.append((c.hd, r))
    ts = [threading.Thread(target=work, args=cw) for cw in zip(chains, want)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_offsets_past_32_bits():
    """Panels of more than 2^31 values: the last sequences' rows."""
    import torch
    hd, nq, ld = 64, 2, 8200
    rows = (1 << 31) // ld + 3000
    qkv = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    w = 3 * nq * hd
    off = ld - w - 8                                  # the heads at the rows' ends
    tail = [700, 300, 5]
    lens = [rows - sum(tail)] + tail
    qkv[:, off:off + w] = panel(rows, w, 41)
    qkv[-300:, :off] = float("nan")                   # columns that hold no head
    cu, cu_dev = offsets(lens)
    offs = (off, off + nq * hd, off + 2 * nq * hd)
    te.attn_sink_fwd(qkv, ld, *offs, cu, cu_dev, nq, nq, hd, 64, 64, 2, 0.125, out, ld)
    got = out[rows - sum(tail):, :nq * hd]
    ref, mag = attention(qkv[rows - sum(tail):], tail, nq, nq, hd, 64, 64, 2, 0.125, offs=offs)
    compare("offsets past 32 bits", got, ref, mag)
    # and a row in the middle of the long sequence that sees its first two keys
    i = lens[0] - 100
    sub = torch.cat([qkv[:2], qkv[i - 64:i + 65]])
    sr, sm = attention(sub, [131], nq, nq, hd, -1, -1, 0, 0.125, offs=offs)
    compare("a row of the long sequence", out[i:i + 1, :nq * hd], sr[66:67], sm[66:67])


@pytest.mark.parametrize("hd", [64, 128])
def test_device_offsets_that_are_not_the_hosts(hd):
    """The kernel's own bounds: rows outside the panel are neither read nor written."""
    import torch
    nq, lens = 2, [100, 200]
    cu, good = offsets(lens)
    qkv = panel(300, 3 * nq * hd, 51)
    for bad in ([0, 100, 10 ** 9], [-5, 100, 300], [0, 300, 100], [2 ** 31 - 1, -2 ** 31, 7], [0, 100, 301]):
        guard = torch.full((900, nq * hd), 7.0, dtype=torch.bfloat16, device="cuda")
        dev = torch.tensor(bad, dtype=torch.int32, device="cuda")
        te.attn_sink_fwd(qkv, 3 * nq * hd, 0, nq * hd, 2 * nq * hd, cu, dev, nq, nq, hd, 9, 9, 1, 0.1, guard[300:600], nq * hd)
        torch.cuda.synchronize()
        assert bool((guard[:300] == 7).all()) and bool((guard[600:] == 7).all()), bad
    # more sequences than the launch lists
    many = [1] * 700 + [50]
    cu, _ = offsets(many)
    qkv = panel(750, 3 * nq * hd, 52)
    rng = np.random.default_rng(1)
    for bad in (rng.integers(-2 ** 31, 2 ** 31, 702), np.full(702, 2 ** 31 - 1), np.full(702, -2 ** 31), np.arange(702)[::-1]):
        guard = torch.full((2250, nq * hd), 7.0, dtype=torch.bfloat16, device="cuda")
        dev = torch.from_numpy(bad.astype(np.int32)).cuda()
        te.attn_sink_fwd(qkv, 3 * nq * hd, 0, nq * hd, 2 * nq * hd, cu, dev, nq, nq, hd, 9, 9, 1, 0.1, guard[750:1500], nq * hd)
        torch.cuda.synchronize()
        assert bool((guard[:750] == 7).all()) and bool((guard[1500:] == 7).all())
    te.check()


def test_table_rows_apart_and_values_that_are_not_finite():
    import torch
    ln, nq, hd, rel = [200, 70], 3, 64, (8, 30, True)
    qkv = panel(sum(ln), 3 * nq * hd, 61)
    wide = torch.randn(8, nq + 5, device="cuda")
    table = wide[:, 2:2 + nq]
    ref, mag = attention(qkv, ln, nq, nq, hd, -1, -1, 0, 0.125, table=table, rel=rel)
    compare("table rows apart", call(qkv, ln, nq, nq, hd, -1, -1, 0, 0.125, table=table, rel=rel), ref, mag)
    bad = table.contiguous().clone()
    bad[3, 1] = float("nan")                          # the far keys before a row, of head 1
    out = call(qkv, ln, nq, nq, hd, -1, -1, 0, 0.125, table=bad, rel=rel)
    # bucket 3 holds every distance from some of at most 30 on
    assert bool(torch.isnan(out[30:200, hd:2 * hd].float()).all())
    ref, mag = attention(qkv, ln, nq, nq, hd, -1, -1, 0, 0.125, table=table, rel=rel)
    keep = [c for c in range(nq * hd) if not hd <= c < 2 * hd]
    compare("heads beside one that is lost", out[:, keep], ref[:, keep], mag[:, keep])
    assert bool((out[:1, hd:2 * hd].float().isfinite()).all())


def test_python_checks():
    import torch
    ln, nq, hd = [30], 2, 64
    qkv = panel(30, 3 * nq * hd, 71)
    cu, cu_dev = offsets(ln)
    out = torch.empty(30, nq * hd, dtype=torch.bfloat16, device="cuda")
    good = dict(qkv=qkv, ld=384, q=0, k=128, v=256, cu=cu, cu_dev=cu_dev, nq=nq, nkv=nq, hd=hd, left=-1, right=-1, sinks=0,
                scale=0.1, out=out, ldo=128)
    f = lambda **o: te.attn_sink_fwd(*{**good, **o}.values())
    f()
    f(cu=[0, 30])
    f(cu=torch.tensor([0, 30]))
    for over, err in ((dict(qkv=qkv.float()), TypeError), (dict(qkv=qkv.cpu()), ValueError), (dict(out=out.float()), TypeError),
                      (dict(ld=392), ValueError), (dict(ldo=136), ValueError), (dict(cu_dev=cu_dev.long()), TypeError),
                      (dict(cu_dev=cu_dev.cpu()), ValueError), (dict(cu=[0, 20, 30]), ValueError), (dict(cu=[0]), ValueError),
                      (dict(cu=[0, 31]), ValueError), (dict(v=264), ValueError), (dict(left=2 ** 40), OverflowError),
                      (dict(out=out[:20]), ValueError), (dict(cu=[0, 30, 40], cu_dev=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError)):
        with pytest.raises(err):
            f(**over)
    with pytest.raises(te.TEError):
        f(left=-3)
    plan = te.relpos_plan(32, 128)
    tab = torch.zeros(32, nq, device="cuda")
    b = lambda plan=plan, tab=tab: te.attn_relbias_fwd(qkv, 384, 0, 128, 256, cu, cu_dev, nq, nq, hd, -1, -1, 0, 0.1, plan, tab, out, 128)
    b()
    for args, err in (((plan, tab[:31]), ValueError), ((plan, tab[:, :1]), ValueError), ((plan, tab.double()), TypeError),
                      ((te.te_q8w(), tab), TypeError)):
        with pytest.raises(err):
            b(*args)
