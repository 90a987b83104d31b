"""The encoder block and the stack with windowed, causal, sink and relative
position attention (te_encoder_block_attn_fwd, EncoderStack(attn=...)) against
the oracle's block with its attention step replaced by the plain 64-bit one."""
import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from oracle import encoder as O
from transformer_encoder_forward_gb300 import synth
from transformer_encoder_forward_gb300.model import EncoderStack
from tests.attn_span_ref import attention
from tests.gpu_util import record_margin, rel_frob, to_np

pytestmark = pytest.mark.gpu

TOL = 5e-3      # the block's gate, as in test_gpu_block.py


def oracle_block(monkeypatch, cfg, p, x, a, cu, i, tables, nxt, at):
    import torch

    def step(qkv, cu_, nq, nkv, hd, q_off, k_off, v_off, window, scale, rows=None):
        table = torch.from_numpy(at["table"]) if "table" in at else None
        o, _ = attention(torch.from_numpy(np.ascontiguousarray(qkv)), list(np.diff(cu_)), nq, nkv, hd, at.get("left", -1),
                         at.get("right", -1), at.get("sinks", 0), scale, table=table, rel=at.get("relpos"))
        return o.numpy()
    with monkeypatch.context() as m:
        m.setattr(O, "attention_varlen", step)
        return O.block_forward(cfg, p, x, a, cu, i, tables, nxt)


def make(name, layers, lens, attn, **over):
    cfg = synth.small_config(name, layers=layers, lens=lens, **over)
    ps = [synth.draw_layer(cfg, i, 31) for i in range(cfg.layers)]
    tables = synth.rope_tables(cfg, lens)
    fin = synth.draw_final_norm(cfg, 31) if cfg.pool else None
    return cfg, ps, tables, EncoderStack(cfg, ps, lens, tables, fin, attn=attn)


def biased(cfg, **more):
    rng = np.random.default_rng(7)
    return dict(relpos=(32, 128, True), table=rng.standard_normal((32, cfg.heads)).astype(np.float32), **more)


@pytest.mark.parametrize("name,over", [("c1", {}), ("c2", {}), ("c4", dict(d=512, heads=4, kv_heads=4, ffn=1024))])
@pytest.mark.parametrize("kind", ["sink", "causal", "bias", "bias_window"])
def test_block(monkeypatch, name, over, kind):
    import torch
    lens = (100, 1, 300, 37)
    cfg = synth.small_config(name, layers=2, lens=lens, **over)
    at = {"sink": dict(left=30, right=20, sinks=4), "causal": dict(right=0), "bias": biased(cfg),
          "bias_window": biased(cfg, left=64, right=0, sinks=1)}[kind]
    cfg, ps, tables, st = make(name, 2, lens, at, **over)
    x0 = synth.draw_x(st.T, cfg.d, 3)
    x, a, _ = st.buffers()
    x.copy_(torch.from_numpy(x0))
    st.input_norm(x, a)
    for i in range(cfg.layers):
        x_in, a_in = to_np(x), to_np(a)
        te.encoder_block_attn_fwd(st.descs[i], st.attn[i], x, a, st.cu_host, st.cu_dev, st.workspace)
        te.check()
        nxt = (ps[i + 1]["norm1_w"], ps[i + 1]["norm1_b"]) if i + 1 < cfg.layers else None
        r = oracle_block(monkeypatch, cfg, ps[i], x_in, a_in, st.cu_host, i, tables, nxt, at)
        e = record_margin("block attn", f"{name} {kind} x_out", rel_frob(to_np(x), r["x_out"]), TOL)
        d = record_margin("block attn", f"{name} {kind} x_out - x_in", rel_frob(to_np(x) - x_in, r["x_out"] - x_in), 2 * TOL)
        assert e < TOL and d < 2 * TOL, (i, e, d)


def test_stack_with_a_list_of_steps():
    """One entry a layer: plain layers give the plain stack's results to the bit,
    and a captured forward the eager one's."""
    import torch
    lens = (200, 64, 5)
    cfg, ps, tables, plain = make("c1", 3, lens, None)
    _, _, _, same = make("c1", 3, lens, [None, None, None])
    shared = biased(cfg)
    _, _, _, mixed = make("c1", 3, lens, [shared, None, shared])
    assert mixed.attn[0] is mixed.attn[2] and mixed.attn[1] is None
    x0 = torch.from_numpy(synth.draw_x(plain.T, cfg.d, 4)).cuda()
    outs = []
    for st in (plain, same, mixed):
        x, a, _ = st.buffers()
        x.copy_(x0)
        st.forward_device(x, a)
        te.check()
        outs.append(x.clone())
    assert torch.equal(outs[0], outs[1]) and not torch.equal(outs[0], outs[2])
    x, a, _ = mixed.buffers()
    x.copy_(x0)
    mixed.forward_device(x, a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mixed.forward_device(x, a, stream=torch.cuda.current_stream())
    for _ in range(2):
        x.copy_(x0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, outs[2])


def test_refusals_touch_nothing():
    import torch
    cfg, ps, tables, st = make("c1", 1, (37, 64), dict(left=8, right=8))
    x, a, _ = st.buffers()
    x.fill_(3.0)
    a.fill_(2.0)
    desc, ok = st.descs[0], st.attn[0]
    plan = te.relpos_plan(32, 128)
    table = torch.zeros(32, cfg.heads, device="cuda")
    bad_plan = te.te_relpos()
    for at in (te.block_attn(left=-2), te.block_attn(sinks=-1), te.block_attn(plan=bad_plan, table=table)):
        with pytest.raises(te.TEError):
            te.encoder_block_attn_fwd(desc, at, x, a, st.cu_host, st.cu_dev, st.workspace)
    desc.window = 8
    with pytest.raises(te.TEError, match="window"):
        te.encoder_block_attn_fwd(desc, ok, x, a, st.cu_host, st.cu_dev, st.workspace)
    desc.window = 0
    desc.attn_scale = -1.0
    with pytest.raises(te.TEError, match="scale"):
        te.encoder_block_attn_fwd(desc, ok, x, a, st.cu_host, st.cu_dev, st.workspace)
    with pytest.raises(ValueError):
        te.block_attn(plan=plan)
    torch.cuda.synchronize()
    assert bool((x == 3).all()) and bool((a == 2).all())
    for wrong in (dict(lft=3), dict(relpos=(32, 128, True)), dict(relpos=(32, 128, True), table=np.zeros((32, 1)))):
        with pytest.raises(ValueError):
            make("c1", 1, (37, 64), wrong)
    with pytest.raises(ValueError):
        make("c1", 2, (37, 64), [None])


def test_a_table_of_too_few_heads_is_refused():
    import torch
    cfg, ps, tables, st = make("c1", 1, (37, 64), dict(left=8, right=8))
    x, a, _ = st.buffers()
    at = te.block_attn(plan=te.relpos_plan(32, 128), table=torch.zeros(32, cfg.heads, device="cuda")[:, :cfg.heads - 1])
    with pytest.raises(ValueError, match="heads"):
        te.encoder_block_attn_fwd(st.descs[0], at, x, a, st.cu_host, st.cu_dev, st.workspace)
