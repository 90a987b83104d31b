"""te_qk_rope_axes at far positions and with frequencies above 1, against the
angle pos * f reduced in 2400-bit integers."""
import math

import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.gpu_util import to_np
from tests.test_rope_turns import turns64

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.mark.parametrize("pairing", [te.TE_ROPE_SECTION_HALVES, te.TE_ROPE_ADJACENT])
@pytest.mark.parametrize("hd", [64, 72])                 # 64: aligned pieces; 72 with 70 turning: single channels
def test_far_positions_of_any_frequency(hd, pairing):
    import torch
    te.check()
    rot = 64 if hd == 64 else 70
    freq = [1.0, 0.1, 3.7, 1000.0, 1e6 + 0.1, 1e19, 6e200] + [1.618 ** (i - 10) for i in range(rot // 2 - 7)]
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 1 << 20, 1, 0, -77], dtype=np.int32)
    rows = len(pos)
    x = torch.zeros(rows, hd, device="cuda")
    first = list(range(rot // 2)) if pairing == te.TE_ROPE_SECTION_HALVES else list(range(0, rot, 2))
    second = [c + rot // 2 for c in first] if pairing == te.TE_ROPE_SECTION_HALVES else [c + 1 for c in first]
    x[:, first] = 1.0
    y = torch.empty_like(x)
    plan = te.rope_axes_plan(hd, (rot,), freq=freq, pairing=pairing)
    te.qk_rope_axes(x, hd, y, hd, 0, 0, 1, 0, hd, None, None, 1e-6, plan, torch.from_numpy(pos[:, None].copy()).cuda(), 1.0,
                    rows)
    te.check()
    got = to_np(y)
    # the word's half unit times the position: 2^-34 turns; the product's top 32
    # bits: 2^-32 turns; the f32 fraction of a half turn: U32 pi; sine and
    # cosine two steps: 4 U32 (the other products are by 0 and 1)
    lim = 2 * math.pi * (2.0 ** -34 * (1 + 2.0 ** -9) + 2.0 ** -32) + (math.pi + 4) * U32
    for r, p in enumerate(pos):
        for i, f in enumerate(freq):
            a = 2 * math.pi * float(turns64(f, int(p)) / 2 ** 64)
            assert abs(got[r, first[i]] - math.cos(a)) <= lim, (p, f)
            assert abs(got[r, second[i]] - math.sin(a)) <= lim, (p, f)
