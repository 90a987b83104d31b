"""Order between calls: the 8-bit and rotation kernels may start while the one
before them ends, and have to see everything that came before all the same -
the buffers that the last call wrote or still reads, other libraries' kernels,
work of another stream that was joined by an event, and all of it in a replayed
graph.  Every result is compared to the bit with one whose calls ran apart."""
import pytest

import transformer_encoder_forward_gb300 as te

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    torch.cuda.init()
    te.lib()
    yield
    te.check()


class Chain:
    """One set of buffers that every pass reuses: norm + quantise, q | k product,
    rotation in place, quantise, gated product, quantise, product."""

    def __init__(self, m, k, heads, hd, f, seed):
        import torch
        self.torch = torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = heads * hd
        i8 = lambda *s: torch.randint(-127, 128, s, dtype=torch.int8, device="cuda", generator=g)
        f32 = lambda *s: torch.rand(*s, device="cuda", generator=g) * 0.01 + 0.001
        self.m, self.k, self.n, self.f, self.heads, self.hd = m, k, n, f, heads, hd
        self.raw = [i8(2, n, k), i8(2, f, n), i8(k, f)]
        self.sc = [f32(2, n), f32(2, f), f32(k)]
        self.wq = [te.q8w(self.raw[0][i], self.sc[0][i]) for i in range(2)]
        self.wg, self.wu = (te.q8w(self.raw[1][i], self.sc[1][i]) for i in range(2))
        self.wd = te.q8w(self.raw[2], self.sc[2])
        self.norm = torch.rand(k, device="cuda", generator=g) + 0.5
        self.x = torch.zeros(m, k, device="cuda")
        self.q = torch.zeros(m, max(k, n, f), dtype=torch.int8, device="cuda")
        self.s = torch.zeros(m, device="cuda")
        self.qk = torch.zeros(m, 2 * n, device="cuda")
        self.gate = torch.zeros(m, f, dtype=torch.bfloat16, device="cuda")
        self.y = torch.zeros(m, k, device="cuda")
        self.pos = torch.arange(3 * m, dtype=torch.int32, device="cuda").reshape(m, 3) % 97
        self.plan = te.rope_axes_plan(hd, (hd // 2, hd // 4, hd // 4))
        self.ws = torch.empty(max(te.i8_workspace(m, k, 2 * n), te.i8_workspace(m, n, 2 * f), te.i8_workspace(m, f, k)) + 256,
                              dtype=torch.uint8, device="cuda")
        self.inputs = [torch.randn(m, k, device="cuda", generator=g) for _ in range(3)]

    def rotate(self):
        te.qk_rope_axes(self.qk, 2 * self.n, self.qk, 2 * self.n, 0, self.n, self.heads, self.heads, self.hd, None, None,
                        1e-6, self.plan, self.pos, 1.0, self.m)

    def calls(self):
        m, k, n, f = self.m, self.k, self.n, self.f
        yield lambda: te.rownorm_quant(self.x, self.norm, None, 0, 1e-6, self.q[:, :k], self.s)
        items = [dict(w=self.wq[i], y=self.qk[:, i * n:(i + 1) * n], ldy=2 * n) for i in range(2)]
        yield lambda: te.i8_linear(self.q[:, :k], self.s, items, self.ws)
        yield lambda: self.rotate()
        yield lambda: te.quant_rows(self.qk[:, :n], self.q[:, :n], self.s)
        yield lambda: te.i8_gated_linear(self.q[:, :n], self.s, self.wg, self.wu, 1, self.gate, self.ws)
        yield lambda: te.quant_rows(self.gate, self.q[:, :f], self.s)
        yield lambda: te.i8_linear(self.q[:, :f], self.s, [dict(w=self.wd, y=self.y, ldy=k, residual=self.x, ldr=k)], self.ws)

    def run(self, apart=False):
        for c in self.calls():
            c()
            if apart:
                self.torch.cuda.synchronize()

    def outputs(self):
        return [t.clone() for t in (self.q, self.s, self.qk, self.gate, self.y)]

    def expect(self, x):
        self.x.copy_(x)
        self.torch.cuda.synchronize()
        self.run(apart=True)
        out = self.outputs()
        self.torch.cuda.synchronize()
        return out


SIZES = [(1, 256, 4, 64, 512), (13, 512, 6, 64, 256), (40, 768, 4, 128, 1024), (300, 512, 4, 64, 512),
         (1500, 512, 4, 96, 320), (2100, 1024, 8, 64, 704)]


def same(a, b):
    return all(bool((x == y).all()) for x, y in zip(a, b))


@pytest.mark.parametrize("m,k,heads,hd,f", SIZES)
def test_calls_in_a_row_on_the_same_buffers(m, k, heads, hd, f):
    c = Chain(m, k, heads, hd, f, 1)
    want = [c.expect(x) for x in c.inputs]
    for r in range(12):
        got = []
        for x in c.inputs:                      # nothing between the passes but torch's copies
            c.x.copy_(x)
            c.run()
            got.append(c.outputs())
        assert all(same(g, w) for g, w in zip(got, want)), r


@pytest.mark.parametrize("m,k,heads,hd,f", SIZES)
def test_rotations_in_place_one_after_another(m, k, heads, hd, f):
    c = Chain(m, k, heads, hd, f, 2)
    torch = c.torch
    x = torch.randn(m, 2 * c.n, device="cuda")
    def go(apart):
        c.qk.copy_(x)
        for _ in range(30):
            c.rotate()
            if apart:
                torch.cuda.synchronize()
        return c.qk.clone()
    want = go(True)
    assert all(bool((go(False) == want).all()) for _ in range(5))


@pytest.mark.parametrize("m,k,heads,hd,f", SIZES)
def test_an_event_of_another_stream_between_two_calls(m, k, heads, hd, f):
    c = Chain(m, k, heads, hd, f, 3)
    torch = c.torch
    side, big = torch.cuda.Stream(), torch.ones(64 << 20, device="cuda")
    want = [c.expect(x) for x in c.inputs]
    q0, s0 = torch.empty_like(c.q[:, :k]), torch.empty_like(c.s)
    for r in range(6):
        for x, w in zip(c.inputs, want):
            te.quant_rows(c.inputs[0], q0, s0)  # a call of ours right before the join
            back = torch.cuda.Event()
            back.record()
            with torch.cuda.stream(side):
                side.wait_event(back)
                big.mul_(1.0)                   # a while, before the input arrives
                c.x.copy_(x)
                done = torch.cuda.Event()
                done.record()
            torch.cuda.current_stream().wait_event(done)
            c.run()
            assert same(c.outputs(), w), r


@pytest.mark.parametrize("m,k,heads,hd,f", SIZES)
def test_a_replayed_graph_with_a_joined_branch(m, k, heads, hd, f):
    c = Chain(m, k, heads, hd, f, 4)
    torch = c.torch
    want = [c.expect(x) for x in c.inputs]
    src = c.inputs[0].clone()
    big = torch.ones(16 << 20, device="cuda")
    q0, s0 = torch.empty_like(c.q[:, :k]), torch.empty_like(c.s)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        te.quant_rows(src, q0, s0)
        with torch.cuda.stream(side):
            big.mul_(1.0)
            c.x.copy_(src)
        main.wait_stream(side)
        c.run()
        c.run()                                 # the same buffers again at once
    for r in range(4):
        for x, w in zip(c.inputs, want):
            src.copy_(x)
            graph.replay()
            assert same(c.outputs(), w), r
