"""The stack's attention steps with a scale of their own, as encoders with a learned
relative position bias have it (unscaled scores)."""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from oracle import encoder as O
from transformer_encoder_forward_gb300 import synth
from tests.attn_span_ref import attention
from tests.gpu_util import record_margin, rel_frob, to_np
from tests.test_gpu_block_attn import TOL, biased, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1.0, 0.03])
@pytest.mark.parametrize("kind", ["sink", "bias"])
def test_block(monkeypatch, scale, kind):
    import torch
    lens = (100, 1, 300, 37)
    cfg = synth.small_config("c1", layers=2, lens=lens)
    at = dict(left=30, right=20, sinks=4, scale=scale) if kind == "sink" else biased(cfg, scale=scale)
    cfg, ps, tables, st = make("c1", 2, lens, [at, None])
    assert st.descs[0].attn_scale == pytest.approx(scale) and st.descs[1].attn_scale == pytest.approx(cfg.scale)

    def step(qkv, cu_, nq, nkv, hd, q_off, k_off, v_off, window, scale_, rows=None):
        table = torch.from_numpy(at["table"]) if "table" in at else None
        o, _ = attention(torch.from_numpy(np.ascontiguousarray(qkv)), list(np.diff(cu_)), nq, nkv, hd, at.get("left", -1),
                         at.get("right", -1), at.get("sinks", 0), scale, table=table, rel=at.get("relpos"))
        return o.numpy()
    x, a, _ = st.buffers()
    x.copy_(torch.from_numpy(synth.draw_x(st.T, cfg.d, 3)))
    st.input_norm(x, a)
    x_in, a_in = to_np(x), to_np(a)
    te.encoder_block_attn_fwd(st.descs[0], st.attn[0], x, a, st.cu_host, st.cu_dev, st.workspace)
    te.check()
    with monkeypatch.context() as m:
        m.setattr(O, "attention_varlen", step)
        r = O.block_forward(cfg, ps[0], x_in, a_in, st.cu_host, 0, tables, (ps[1]["norm1_w"], ps[1]["norm1_b"]))
    e = record_margin("block attn scale", f"{kind} {scale} x_out - x_in", rel_frob(to_np(x) - x_in, r["x_out"] - x_in), 2 * TOL)
    assert e < 2 * TOL, e


def test_refusals():
    import torch
    for bad in (0.0, -1.0, float("nan")):
        _, _, _, st = make("c1", 1, (37, 64), dict(left=8, right=8, scale=bad))
        x, a, _ = st.buffers()
        x.fill_(3.0)
        with pytest.raises(te.TEError, match="scale"):
            te.encoder_block_attn_fwd(st.descs[0], st.attn[0], x, a, st.cu_host, st.cu_dev, st.workspace)
        torch.cuda.synchronize()
        assert bool((x == 3).all())
