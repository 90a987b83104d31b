"""The 8-bit products' clusters beside other kernels that hold TMEM on streams of
their own: all end, with the results of calls alone."""
import threading

import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te

pytestmark = pytest.mark.gpu


def jobs():
    import torch
    gen = torch.Generator("cuda").manual_seed(9)
    i8 = lambda *s: torch.randint(-127, 128, s, dtype=torch.int8, device="cuda", generator=gen)
    out = []
    for m, k, n in ((12, 4096, 4096), (60, 2048, 8192), (101, 768, 2304), (300, 4096, 1024), (40, 512, 4096)):
        x, xs, w, sw = i8(m, k), torch.rand(m, device="cuda"), i8(n, k), torch.rand(n, device="cuda")
        y, ws = torch.empty(m, n, device="cuda"), torch.empty(te.i8_workspace(m, k, n), device="cuda", dtype=torch.uint8)
        args = (x, xs, [dict(w=te.q8w(w, sw), y=y, ldy=n)], ws)
        te.i8_linear(*args)
        out.append((args, y, y.clone(), w, sw))
    torch.cuda.synchronize()
    return out


def beside(other, rounds):
    """Runs `other` in a thread while this one makes its products; both to the end."""
    import torch
    todo, stream, fails = jobs(), torch.cuda.Stream(), []

    def run():
        try:
            other()
        except Exception as e:
            fails.append(e)
    t = threading.Thread(target=run)
    t.start()
    for _ in range(rounds):
        for args, y, _, _, _ in todo:
            te.i8_linear(*args, stream=stream)
    t.join()
    stream.synchronize()
    te.check()
    assert not fails, fails
    for _, y, want, _, _ in todo:
        assert torch.equal(y, want)


@pytest.mark.parametrize("bn", [64, 256])
def test_beside_the_tensor_ceilings_pairs(bn):
    import torch
    stream = torch.cuda.Stream()
    beside(lambda: [te.mma_peak(bn, 400, stream=stream) for _ in range(40)], 150)


def test_beside_attention_and_the_q8_products():
    import torch
    gen = torch.Generator("cuda").manual_seed(4)
    T, d = 2000, 512
    qkv = torch.randn(T, 3 * d, device="cuda", generator=gen).bfloat16()
    w = torch.randint(-127, 128, (d, d), dtype=torch.int8, device="cuda", generator=gen)
    sw = torch.rand(d, device="cuda", generator=gen) / 2000
    o, y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, d, device="cuda")
    cu = np.array([0, 700, 1100, T], dtype=np.int32)
    cud, stream = torch.from_numpy(cu).cuda(), torch.cuda.Stream()

    def pair():
        te.attn_varlen_fwd(qkv, 3 * d, 0, d, 2 * d, cu, cud, 8, 8, 64, 0, 0.125, o, d, stream=stream)
        te.q8_linear(o, [dict(w=te.q8w(w, sw), y=y, ldy=d)], stream=stream)
    torch.cuda.synchronize()
    pair()
    stream.synchronize()
    want = o.clone(), y.clone()
    torch.cuda.synchronize()
    beside(lambda: [pair() for _ in range(400)], 300)
    assert torch.equal(o, want[0]) and torch.equal(y, want[1])
