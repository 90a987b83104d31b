"""Measured cases of the operators for 8-bit activations and multi-axis rotary positions.

Four operators of an encoder block whose activations are held in 8 bits and whose tokens sit on a
grid (image patches, video patches) or on a line (text):

* ``rope``        q/k norm + rotary positions with several axes (te.qk_rope_axes)
* ``linear``      product of 8-bit integers with a scale for each token and each output channel,
                  several weights sharing the activation (te.i8_linear)
* ``gated``       the gate and up products and the gate, from the same integers (te.i8_gated_linear)
* ``norm_linear`` the block's way into a product: (pre-norm and) quantisation of each token, then
                  the product (te.rownorm_quant or te.quant_rows, then te.i8_linear):
                  q = round(v * (127 / max |v|)), ties to even, each step rounded to 32 bits

With ``own`` false each is computed in its plain form from elementary torch operations.
"""
import math

import torch

own = False

GELU, SILU = 0, 1                # te_act_kind
NORMS = {"rms": 0, "ln": 1}      # te_norm_kind
PAIRINGS = {"section_halves": 0, "head_halves": 1, "adjacent": 2}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # an image's tokens through a DiT block: 2 x 4224 rows, 30 heads of 128, axes 32 | 48 | 48
        rope("rope_dit_image", 8448, 30, 30, 128, (32, 48, 48), "section_halves", "axis", True, "bf16", 0),
        # a long clip: 32760 patches of a 21 x 30 x 52 grid, every row far from the start
        rope("rope_video_clip", 32760, 30, 30, 128, (44, 42, 42), "adjacent", "axis", True, "bf16", 40000),
        # one new row, as a caption or query of a single token: latency
        rope("rope_one_row", 1, 8, 8, 64, (16, 24, 24), "head_halves", "whole", True, "bf16", 0),
        # grouped k heads of an odd width, part of each head unrotated, f32 panel, no norm
        rope("rope_vit_ragged", 1023, 12, 4, 72, (24, 24, 16), "head_halves", "whole", False, "f32", 3),
        # one token against the text stack's q|k|v: the smallest call
        linear("linear_one_token", 1, 512, 512, 3, "bf16", False),
        # a short query at the DiT's width: 7 tokens, bound by the weights' bytes
        linear("linear_short_query", 7, 3840, 3840, 3, "bf16", True),
        # a packed pair of short texts, odd row count, biased projections of the ViT width
        linear("linear_two_texts", 101, 768, 768, 3, "f32", True),
        # the DiT block's down projection over a whole image
        linear("linear_dit_down", 8448, 10240, 3840, 1, "f32", False),
        # the text stack's gate|up for one short sequence
        gated("gated_short_text", 37, 512, 2048, GELU, False),
        # the DiT block's gate|up over a whole image: the largest
        gated("gated_dit", 8448, 3840, 10240, SILU, False),
        # the DiT block's pre-norm, quantisation and q|k|v at one image's rows
        norm_linear("norm_qkv_dit", 2112, 3840, 3840, 3, "rms", "f32", "bf16"),
        # attention's output, quantised, through the text stack's out projection
        norm_linear("quant_out_text", 16238, 512, 512, 1, "none", "bf16", "f32"),
    ]


def rope(name, rows, nq, nkv, hd, sections, pairing, freqs, norm, dtype, start):
    return {"name": name, "op": "rope", "rows": rows, "nq": nq, "nkv": nkv, "hd": hd,
            "sections": "|".join(map(str, sections)), "pairing": pairing, "freqs": freqs,
            "norm": norm, "dtype": dtype, "start": start}


def linear(name, m, k, n, z, ydt, bias):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "z": z, "ydt": ydt, "bias": bias}


def gated(name, m, k, f, act, bias):
    return {"name": name, "op": "gated", "m": m, "k": k, "f": f, "act": act, "bias": bias}


def norm_linear(name, m, k, n, z, norm, xdt, ydt):
    return {"name": name, "op": "norm_linear", "m": m, "k": k, "n": n, "z": z, "norm": norm,
            "xdt": xdt, "ydt": ydt}


MOST_FLOPS = 2.0 * 8448 * 3840 * 20480
MOST_ROPE = 32760 * 60 * 128


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "linear", "gated", "norm_linear"])
    if op == "rope":
        hd = rng.choice([32, 64, 72, 80, 96, 128, 128])
        axes = rng.choice([2, 3, 3, 4])
        # even widths that leave at most a part of the head unrotated
        width = 2 * rng.randint(hd // 4, hd // 2)
        sections = [2] * axes
        for _ in range(width // 2 - axes):
            sections[rng.randrange(axes)] += 2
        if rng.random() < 0.5:   # widths a multiple of 8, as models choose them
            sections = [8] * axes
            for _ in range(hd // 8 - axes):
                sections[rng.randrange(axes)] += 8
        nkv = rng.randint(1, 16)
        nq = nkv * rng.choice([1, 1, 2, 4])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = min(32760, MOST_ROPE // ((nq + nkv) * hd) // (2 if dtype == "f32" else 1))
        case = rope("", _log(rng, 1, most), nq, nkv, hd, sections, rng.choice(sorted(PAIRINGS)),
                    rng.choice(["axis", "whole"]), rng.random() < 0.6, dtype,
                    rng.choice([0, 0, _log(rng, 1, 100000)]))
    else:
        k = 64 * _log(rng, 1, 160)
        if op == "gated":
            n, z = 32 * _log(rng, 1, 320), 2
        else:
            n, z = 32 * _log(rng, 1, 160), rng.choice([1, 2, 3])
        m = _log(rng, 1, min(16384, max(1, int(MOST_FLOPS / (2.0 * k * n * z)))))
        if op == "linear":
            case = linear("", m, k, n, z, rng.choice(["bf16", "f32"]), rng.random() < 0.5)
        elif op == "gated":
            case = gated("", m, k, n, rng.choice([GELU, SILU]), rng.random() < 0.5)
        else:
            norm = rng.choice(["rms", "ln", "none"])
            case = norm_linear("", m, k, n, z, norm, "bf16" if norm == "none" else rng.choice(["f32", "bf16"]),
                               rng.choice(["bf16", "f32"]) if norm == "none" else "bf16")
    del case["name"]
    return case


# ------------------------------------------------------------------------ inputs

def _sections(case):
    return [int(s) for s in case["sections"].split("|")]


def _weights(gen, n, k, count, bias):
    """int8 weights with a row scale that keeps outputs near the inputs' size."""
    q = torch.randint(-127, 128, (count, n, k), generator=gen, device="cuda", dtype=torch.int8)
    s = (0.75 + 0.5 * torch.rand(count, n, generator=gen, device="cuda")) / (73.0 * math.sqrt(k))
    b = 0.02 * torch.randn(count, n, generator=gen, device="cuda") if bias else None
    return q, s, b


def _tokens8(gen, m, k):
    """Quantised tokens as a quantiser leaves them: near-normal rows that reach +-127 once, each
    with the scale of its own size."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    a = x.abs().amax(1, keepdim=True)
    q = torch.round(x * (127.0 / a)).to(torch.int8)
    return q, (a[:, 0] / 127.0) * (0.5 + torch.rand(m, generator=gen, device="cuda"))


def _positions(gen, rows, axes, start):
    """Patches of a grid, frame by frame (time slowest); axes past the third count as text does.
    The last eighth is a caption whose tokens count the same on every axis."""
    side = max(1, int(round(rows ** (1.0 / 3))))
    i = torch.arange(rows, device="cuda")
    w, h = i % (2 * side), (i // (2 * side)) % side
    t = i // (2 * side * side)
    cols = ([t, h, w] + [i] * max(0, axes - 3))[:axes] if axes != 2 else [i // (2 * side), w]
    pos = torch.stack(cols, 1) + start + int(torch.randint(0, 8, (1,), generator=gen, device="cuda"))
    cap = rows - rows // 8
    pos[cap:] = (int(pos.max()) + 1 + i[cap:] - cap)[:, None]
    return pos.to(torch.int32).contiguous()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    d = {}
    if case["op"] == "rope":
        rows, nq, nkv, hd = case["rows"], case["nq"], case["nkv"], case["hd"]
        d["qkv"] = torch.randn(rows, (nq + 2 * nkv) * hd, generator=gen, device="cuda",
                               dtype=torch.float32).to(DTYPES[case["dtype"]])
        d["pos"] = _positions(gen, rows, len(_sections(case)), case["start"])
        if case["norm"]:
            d["qn"] = 1 + 0.1 * torch.randn(hd, generator=gen, device="cuda")
            d["kn"] = 1 + 0.1 * torch.randn(hd, generator=gen, device="cuda")
        return d
    m, k = case["m"], case["k"]
    if case["op"] == "norm_linear":
        x = torch.randn(m, k, generator=gen, device="cuda")
        x *= 0.25 + 4 * torch.rand(k, generator=gen, device="cuda") ** 4   # a few wide channels
        d["x"] = x.to(DTYPES[case["xdt"]])
        if case["norm"] != "none":
            d["nw"] = 1 + 0.1 * torch.randn(k, generator=gen, device="cuda")
        if case["norm"] == "ln":
            d["nb"] = 0.1 * torch.randn(k, generator=gen, device="cuda")
        d["w"] = _weights(gen, case["n"], k, case["z"], False)
        return d
    d["xq"], d["xs"] = _tokens8(gen, m, k)
    if case["op"] == "linear":
        d["w"] = _weights(gen, case["n"], k, case["z"], case["bias"])
    else:
        d["w"] = _weights(gen, case["f"], k, 2, case["bias"])
    return d


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if case["op"] == "rope":
        # the rotation's layout, which a program works out once
        first, second, axis, power = _pair_channels(case)
        state["first"], state["second"], state["axis"] = (torch.tensor(v, device="cuda") for v in (first, second, axis))
        state["freq"] = 10000.0 ** torch.tensor(power, dtype=torch.float64, device="cuda")
    if own:
        import transformer_encoder_forward_gb300 as te
        state["te"] = te
        if case["op"] == "rope":
            rows, width = case["rows"], (case["nq"] + case["nkv"]) * case["hd"]
            state["out"] = torch.empty(rows, width, device="cuda", dtype=DTYPES[case["dtype"]])
            state["plan"] = te.rope_axes_plan(case["hd"], _sections(case), theta=10000.0,
                                              pairing=PAIRINGS[case["pairing"]],
                                              whole=case["freqs"] == "whole")
            return state
        m, k = case["m"], case["k"]
        # what such a program holds: room for the quantised tokens, the weights' descriptors, a workspace
        if case["op"] == "norm_linear":
            state["xq"] = torch.empty(m, k, device="cuda", dtype=torch.int8)
            state["xs"] = torch.empty(m, device="cuda")
        q, s, b = state["w"]
        state["qw"] = [te.q8w(q[i], s[i], None if b is None else b[i]) for i in range(q.shape[0])]
        n = q.shape[1]
        state["ws"] = torch.empty(te.i8_workspace(m, k, n * q.shape[0]), device="cuda", dtype=torch.uint8)
        if case["op"] == "gated":
            state["out"] = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
        else:
            state["y"] = [torch.empty(m, n, device="cuda", dtype=DTYPES[case["ydt"]]) for _ in state["qw"]]
            state["items"] = [dict(w=w, y=y, ldy=n) for w, y in zip(state["qw"], state["y"])]
    return state


# --------------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    te, case = st["te"], st["case"]
    if case["op"] == "rope":
        nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
        te.qk_rope_axes(st["qkv"], (nq + 2 * nkv) * hd, st["out"], (nq + nkv) * hd, 0, nq * hd, nq, nkv,
                        hd, st.get("qn"), st.get("kn"), EPS, st["plan"], st["pos"], hd ** -0.5,
                        case["rows"])
        return st["out"]
    if case["op"] == "gated":
        te.i8_gated_linear(st["xq"], st["xs"], st["qw"][0], st["qw"][1], case["act"], st["out"], st["ws"])
        return st["out"]
    if case["op"] == "norm_linear":
        if case["norm"] == "none":
            te.quant_rows(st["x"], st["xq"], st["xs"])
        else:
            te.rownorm_quant(st["x"], st["nw"], st.get("nb"), NORMS[case["norm"]], EPS, st["xq"], st["xs"])
    te.i8_linear(st["xq"], st["xs"], st["items"], st["ws"])
    return st["y"]


def _pair_channels(case):
    """First and second channel and axis of each rotated pair, and its frequency's exponent."""
    sections = _sections(case)
    rot = sum(sections)
    first, second, axis, power = [], [], [], []
    start = 0
    for a, sec in enumerate(sections):
        for i in range(sec // 2):
            p = start // 2 + i
            if case["pairing"] == "section_halves":
                first.append(start + i)
                second.append(start + i + sec // 2)
            elif case["pairing"] == "head_halves":
                first.append(p)
                second.append(p + rot // 2)
            else:
                first.append(2 * p)
                second.append(2 * p + 1)
            axis.append(a)
            power.append(-2.0 * i / sec if case["freqs"] == "axis" else -2.0 * p / rot)
        start += sec
    return first, second, axis, power


def _plain(st):
    case = st["case"]
    if case["op"] == "rope":
        return _plain_rope(st)
    if case["op"] == "norm_linear":
        x = st["x"].float()
        if case["norm"] == "rms":
            x = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * st["nw"]
        elif case["norm"] == "ln":
            x = x - x.mean(1, keepdim=True)
            x = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * st["nw"] + st["nb"]
        a = x.abs().amax(1, keepdim=True)
        m127 = torch.full_like(a, 127.0)
        xq, xs = torch.round(x * (m127 / a)), (a / m127)[:, 0]
    else:
        xq, xs = st["xq"].float(), st["xs"]
    q, s, b = st["w"]
    y = torch.matmul(xq, q.float().transpose(1, 2)) * xs[:, None] * s[:, None]
    if b is not None:
        y = y + b[:, None]
    if case["op"] == "gated":
        g, u = y[0], y[1]
        if case["act"] == GELU:
            g = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
        else:
            g = g / (1 + torch.exp(-g))
        return (g * u).to(torch.bfloat16)
    return list(y.to(DTYPES[case["ydt"]]).unbind(0))


def _plain_rope(st):
    case = st["case"]
    rows, nq, nkv, hd = case["rows"], case["nq"], case["nkv"], case["hd"]
    x = st["qkv"][:, :(nq + nkv) * hd].float().view(rows, nq + nkv, hd)
    if case["norm"]:
        x = x / torch.sqrt((x * x).mean(2, keepdim=True) + EPS)
        x = torch.cat([x[:, :nq] * st["qn"], x[:, nq:] * st["kn"]], 1)
    # the angles of far positions need 64 bits
    angle = st["pos"].double()[:, st["axis"]] * st["freq"]
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    i1, i2 = st["first"], st["second"]
    x1, x2 = x[:, :, i1], x[:, :, i2]
    y = x.clone()
    y[:, :, i1] = x1 * c - x2 * s
    y[:, :, i2] = x2 * c + x1 * s
    y[:, :nq] *= hd ** -0.5
    return y.reshape(rows, -1).to(DTYPES[case["dtype"]])


# ----------------------------------------------------------------------- exact

def exact(case, seed):
    st = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] == "rope":
        rows, nq, nkv, hd = case["rows"], case["nq"], case["nkv"], case["hd"]
        sections = _sections(case)
        rot, half = sum(sections), sum(sections) // 2
        pos = st["pos"].to(f64)
        out = torch.empty(rows, nq + nkv, hd, dtype=f64, device="cuda")
        for h in range(nq + nkv):
            x = st["qkv"][:, h * hd:(h + 1) * hd].to(f64)
            if case["norm"]:
                inv = (x.square().sum(1) / hd + EPS).rsqrt()
                x = x * inv[:, None] * st["qn" if h < nq else "kn"].to(f64)
            o = x.clone()
            at = 0
            for a, sec in enumerate(sections):
                n = sec // 2
                i = torch.arange(n, dtype=f64, device="cuda")
                e = i / n if case["freqs"] == "axis" else (i + at // 2) / half
                turn = torch.polar(torch.ones(rows, n, dtype=f64, device="cuda"),
                                   pos[:, a:a + 1] * torch.exp(-math.log(10000.0) * e))
                if case["pairing"] == "section_halves":
                    re, im = slice(at, at + n), slice(at + n, at + sec)
                elif case["pairing"] == "head_halves":
                    re, im = slice(at // 2, at // 2 + n), slice(half + at // 2, half + at // 2 + n)
                else:
                    re, im = slice(at, at + sec, 2), slice(at + 1, at + sec, 2)
                v = torch.complex(x[:, re], x[:, im]) * turn
                o[:, re], o[:, im] = v.real, v.imag
                at += sec
            out[:, h] = o * hd ** -0.5 if h < nq else o
        return out.view(rows, -1)
    if case["op"] == "norm_linear":
        v = st["x"].to(f64)
        if case["norm"] == "ln":
            v = v - v.sum(1, keepdim=True) / case["k"]
        if case["norm"] != "none":
            v = v * (v.square().sum(1, keepdim=True) / case["k"] + EPS).rsqrt() * st["nw"].to(f64)
        if case["norm"] == "ln":
            v = v + st["nb"].to(f64)
        top = v.abs().max(1).values
        # the integers are defined by 32-bit steps: half the largest value lies on a border between
        # two of them (63.5), in any number of bits
        step = (127 / top.float().to(f64)).float()
        xq, xs = torch.round((v.float() * step[:, None]).to(f64)), top / 127
    else:
        xq, xs = st["xq"].to(f64), st["xs"].to(f64)
    ys = []
    for i, (q, s) in enumerate(zip(st["w"][0], st["w"][1])):
        y = torch.matmul(xq, q.to(f64).T) * torch.outer(xs, s.to(f64))
        ys.append(y if st["w"][2] is None else y + st["w"][2][i].to(f64))
    if case["op"] != "gated":
        return ys
    g, u = ys
    if case["act"] == GELU:      # 0.5 (1 + tanh z) is the logistic function of 2 z
        return g * torch.sigmoid(math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)) * u
    return g * torch.sigmoid(g) * u


# ------------------------------------------------------------------------ work

def work(case):
    """Inputs read once, outputs written once; products count two operations a term."""
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "rope":
        rows, heads, hd = case["rows"], case["nq"] + case["nkv"], case["hd"]
        axes, rot = len(_sections(case)), sum(_sections(case))
        values = rows * heads * hd
        return {"bytes": 2 * values * size[case["dtype"]] + 4 * rows * axes + (8 * hd if case["norm"] else 0),
                "flops": rows * heads * 3 * rot + (4 * values if case["norm"] else 0)}
    m, k = case["m"], case["k"]
    n = 2 * case["f"] if case["op"] == "gated" else case["n"] * case["z"]
    out = 2 * m * case["f"] if case["op"] == "gated" else m * n * size[case["ydt"]]
    x = m * k * size[case["xdt"]] if case["op"] == "norm_linear" else m * k + 4 * m
    vec = 8 * n if case.get("bias") else 4 * n
    if case.get("norm", "none") != "none":
        vec += 4 * k * (2 if case["norm"] == "ln" else 1)
    return {"bytes": x + n * k + vec + out, "flops": 2 * m * n * k}
