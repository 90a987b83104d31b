"""Every kernel of the 8-bit products, each chosen by hand and seen to run, at
sizes that end inside its tiles; and which one the rule takes."""
import pytest

import transformer_encoder_forward_gb300 as te

pytestmark = pytest.mark.gpu

FEW, MID, RES, LARGE = te.TE_I8_FEW, te.TE_I8_MIDDLING, te.TE_I8_RESIDENT, te.TE_I8_LARGE
U32, UB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(autouse=True)
def _rule_again():
    import torch
    torch.cuda.init()
    te.lib()
    yield
    te.i8_choose(None)
    te.check()


def few(gated):
    return [(FEW, 8, 1), (FEW, 8, 2), (FEW, 16, 1), (FEW, 32, 1)] if gated else \
           [(FEW, 8, 2), (FEW, 8, 4), (FEW, 16, 1), (FEW, 16, 2), (FEW, 32, 1)]


MIDS = [(MID, t, s) for t in (16, 32, 64, 128) for s in (1, 2, 4, 8)]
PLAIN, GATED = ([*few(g), *MIDS, (RES, 128, 1), (LARGE, 0, 0)] for g in (False, True))
# the large pipeline's own tiles (tokens, tiles a unit)
TILES = [(64, 1), (128, 1), (192, 1), (128, 2), (192, 2)]


def size_of(tile, gated):
    """The smallest of some sizes, ragged against every tile, that the large pipeline cuts so."""
    sizes = [(m, k, n) for m in (50, 300, 1101, 1300, 2601, 4300, 6163, 7731) for k in (576, 832, 2048, 4096)
             for n in (160, 352, 768, 2080, 4128)]
    for m, k, n in sorted(sizes, key=lambda s: s[0] * s[1] * s[2]):
        if te.i8_choice_of(m, k, [n], gated) == (LARGE, *tile):
            return m, k, n
    raise AssertionError(f"no size takes {tile}")


def tokens(choice):
    kernel, tile, _ = choice
    if kernel == FEW:
        return [1, tile - 3, tile]
    if kernel == MID:
        return [1, tile - 1, tile, 3 * tile + 5]
    return [9, 127, 128, 1000, 20001] if kernel == RES else [9, 61, 200, 1300]


def depths(choice):
    kernel, _, split = choice
    if kernel == FEW:
        return [64, 192, 1088, 4160]
    if kernel == MID:                                        # at least one stage for each CTA; ragged and uneven shares
        return [k for k in (64, 192, 512, 1024, 1088, 2240) if (k + 127) // 128 >= split]
    return [64, 128, 320, 512] if kernel == RES else [576, 1024, 2112]


def draw(m, k, ns, seed):
    import torch
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randint(-60, 61, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    return x, [torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8) for n in ns]


def workspace(m, k, n):
    import torch
    return torch.full((te.i8_workspace(m, k, n) + 256,), 0xA5, dtype=torch.uint8, device="cuda")


def check_plain(m, k, ns):
    import torch
    x, w = draw(m, k, ns, m * 31 + k)
    one = torch.ones(max(m, max(ns)), device="cuda")
    full = [torch.full((m + 1, n + 8), float("nan"), device="cuda") for n in ns]
    te.i8_linear(x, one[:m], [dict(w=te.q8w(a, one[:a.shape[0]]), y=y[:m, :n], ldy=n + 8) for a, y, n in zip(w, full, ns)],
                 workspace(m, k, sum(ns)))
    for a, y, n in zip(w, full, ns):
        ref = x.double() @ a.double().T
        assert float(ref.abs().max()) < 2 ** 24              # sums that f32 holds exactly
        assert torch.equal(y[:m, :n].double(), ref), (m, k, ns)
        assert bool(torch.isnan(y[m]).all()) and bool(torch.isnan(y[:, n:]).all())


def check_gated(m, k, f):
    import torch
    x, (wg, wu) = draw(m, k, [f, f], m * 37 + k)
    xs = torch.full((m,), 2.0 ** -7, device="cuda")          # powers of two: g and u are exact
    ws = torch.full((f,), 2.0 ** -8, device="cuda")
    full = torch.full((m + 1, f + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
    te.i8_gated_linear(x, xs, te.q8w(wg, ws), te.q8w(wu, ws), te.TE_ACT_SILU, full[:m, :f], workspace(m, k, 2 * f))
    g, u = (x.double() @ a.double().T * 2.0 ** -15 for a in (wg, wu))
    ref = g * torch.sigmoid(g) * u
    # one rounding to bf16 behind f32: three roundings of the exponent |g|, two
    # steps each of the exponential and the reciprocal, three products
    lim = (UB + (3 * g.abs() + 12) * U32) * ref.abs() + 1e-30
    assert bool(((full[:m, :f].double() - ref).abs() <= lim).all()), (m, k, f)
    assert bool(torch.isnan(full[m]).all()) and bool(torch.isnan(full[:, f:]).all())


@pytest.mark.parametrize("choice", PLAIN)
def test_every_kernel_is_exact_on_integers(choice):
    te.i8_choose(choice)
    for m in tokens(choice):
        for k in depths(choice):
            for ns in ([32], [96, 160, 32], [416]):
                c = te.i8_choice_of(m, k, ns)
                assert c == choice or c[0] == choice[0] == LARGE
                check_plain(m, k, ns)


@pytest.mark.parametrize("choice", GATED)
def test_every_kernel_gated(choice):
    te.i8_choose(choice)
    for m in tokens(choice):
        for k in depths(choice):
            for f in (32, 224):
                c = te.i8_choice_of(m, k, [f], gated=True)
                assert c == choice or c[0] == choice[0] == LARGE
                check_gated(m, k, f)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tile", TILES)
def test_every_tile_of_the_large_pipeline(tile, gated):
    te.i8_choose((LARGE, 0, 0))
    m, k, n = size_of(tile, gated)
    if gated:
        check_gated(m, k, n)
    else:
        check_plain(m, k, [n])


@pytest.mark.parametrize("m,k,ns,gated,want", [
    (1, 512, [512] * 3, False, (FEW, 8, 2)), (7, 3840, [3840] * 3, False, (FEW, 8, 2)), (7, 10240, [3840], False, (FEW, 8, 4)),
    (1, 10240, [1024], False, (FEW, 8, 4)), (16, 768, [768] * 3, False, (FEW, 16, 1)), (32, 256, [512], False, (FEW, 32, 1)),
    (101, 768, [768] * 3, False, MID), (128, 3840, [3840], False, MID), (4000, 1024, [128], False, MID),
    (37, 512, [2048], True, MID), (16238, 512, [512], False, (RES, 128, 1)), (1100, 512, [2048], True, (RES, 128, 1)),
    (8448, 10240, [3840], False, LARGE), (2112, 3840, [3840] * 3, False, LARGE), (8448, 3840, [10240], True, LARGE)])
def test_the_rules_choice(m, k, ns, gated, want):
    c = te.i8_choice_of(m, k, ns, gated)
    assert (c if isinstance(want, tuple) else c[0]) == want


def test_the_rule_reaches_every_kernel():
    # no instantiation is there for nobody: sizes of the documented range that take it
    seen = {False: set(), True: set()}
    for gated in seen:
        for m in [1, 8, 12, 16, 24, 32, 33, 50, 64, 100, 128, 230, 300, 509, 570, 700, 1000, 1261, 1412, 1772, 2489, 2788, 4913,
                  5503, 9698, 10861, 16238, 21438]:
            for k in [64, 192, 320, 448, 512, 576, 768, 1024, 1536, 2048, 2560, 3840, 4096, 10240, 16384, 65536]:
                for n in [32, 64, 96, 128, 256, 352, 512, 1024, 2048, 3840, 5120, 7680, 11520, 20480]:
                    seen[gated].add(te.i8_choice_of(m, k, [n], gated))
    large = {(LARGE, *t) for t in TILES}
    assert seen[False] == {*few(False), *MIDS, (RES, 128, 1), *large}
    assert seen[True] == {*few(True), *MIDS, (RES, 128, 1), *large}
