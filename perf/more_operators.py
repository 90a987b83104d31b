"""Measured cases of attention with a window and sinks, and with a learned relative position bias.

Two operators of an encoder block's attention step, over packed sequences of their own lengths:

* ``sink``  attention with a sliding window (left and right, either may be open) whose first few
            tokens stay visible to every later row (te.attn_sink_fwd)
* ``bias``  the same attention with a learned bias a head and bucket of relative position added to
            the scores before the softmax (te.attn_relbias_fwd)

Key j is visible to row i of its sequence when j <= i + right and (j >= i - left or j < sinks);
-1 is no limit.  The bucket of distance j - i is exact for small distances and logarithmic from
half a side's buckets to max_distance; two-sided buckets take their upper half for j > i, one-sided
ones put every j >= i into bucket 0.

With ``own`` false each is computed in its plain form from elementary torch operations.
"""
import math

import torch

own = False

# 32 texts of 16 to 1024 tokens, as a batch of documents arrives
TEXTS = ("538|85|780|447|955|302|671|219|90|834|613|127|409|733|56|891|364|505|19|648|277|702|163|"
         "820|456|588|341|937|74|490|760|914")


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # two short texts at the smallest model's heads: latency
        case("sink_two_texts", "sink", "37|64", 4, 4, 64, 16, 16, 2),
        # a packed batch of texts through a windowed layer of the text stack
        case("sink_text_batch", "sink", TEXTS, 8, 8, 64, 512, 512, 4),
        # one long document, odd length, a narrow window and a block of global tokens
        case("sink_long_document", "sink", "30001", 12, 12, 64, 256, 256, 64),
        # a causal text encoder with grouped k heads: a long text beside a short one
        case("sink_causal_grouped", "sink", "8191|130|1", 32, 8, 128, 1023, 0, 4),
        # two images of the DiT with register tokens in front, half an image's rows to either side
        case("sink_image_registers", "sink", "4224|4224", 30, 30, 128, 1056, 1056, 32),
        # a query of one token: the smallest call
        case("bias_one_token", "bias", "1", 8, 8, 64, -1, -1, 0, 32, 128, True),
        # two short texts
        case("bias_two_texts", "bias", "37|64", 4, 4, 64, -1, -1, 0, 32, 128, True),
        # the packed batch of texts, every row sees its whole text
        case("bias_text_batch", "bias", TEXTS, 8, 8, 64, -1, -1, 0, 32, 128, True),
        # sound or patches, 4 sequences of 1024, many buckets that reach far
        case("bias_wide_reach", "bias", "1024|1024|1024|1024", 12, 12, 64, -1, -1, 0, 320, 800, True),
        # whole images at the DiT's heads: the largest
        case("bias_image", "bias", "4224|4224", 30, 30, 128, -1, -1, 0, 32, 128, True),
        # one-sided buckets, causal, windowed, one sink, grouped k heads
        case("bias_causal_window", "bias", "6001|999", 16, 4, 128, 2047, 0, 1, 32, 256, False),
    ]


def case(name, op, lens, nq, nkv, hd, left, right, sinks, buckets=0, max_distance=0, two_sided=False):
    c = {"name": name, "op": op, "lens": lens, "nq": nq, "nkv": nkv, "hd": hd, "left": left,
         "right": right, "sinks": sinks}
    if op == "bias":
        c.update(buckets=buckets, max_distance=max_distance, two_sided=two_sided)
    return c


MOST_FLOPS = 4.0 * 128 * 30 * 2 * 4224 * 4224
MOST_TOKENS = 30001
MOST_PLAIN = 5.0e8           # heads x pairs that the plain form goes through


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sink", "bias"])
    hd = rng.choice([64, 128])
    nkv = rng.randint(1, 12)
    nq = nkv * rng.choice([1, 1, 2, 4])
    total = _log(rng, 1, MOST_TOKENS)
    lens = []
    while sum(lens) < total and len(lens) < 40:
        lens.append(min(_log(rng, 1, max(2, total)), total - sum(lens)))
    causal = rng.random() < 0.3
    left = rng.choice([-1, _log(rng, 1, 4096), _log(rng, 16, 2048)])
    right = 0 if causal else rng.choice([left, -1, _log(rng, 1, 2048)])
    sinks = rng.choice([0, _log(rng, 1, 16), _log(rng, 1, 400)])
    if op == "sink" and left == right == -1:
        left = right = _log(rng, 8, 1024)
    c = case("", op, "|".join(map(str, lens)), nq, nkv, hd, left, right, sinks)
    if op == "bias":
        two = not causal and rng.random() < 0.8
        buckets = 2 * rng.choice([rng.randint(2, 16), 16, rng.randint(16, 160)])
        side = buckets // 2 if two else buckets
        c.update(buckets=buckets, max_distance=side + _log(rng, 1, 1024), two_sided=two)
    # lengths shrink until the case costs no more than the largest listed one
    while work(c)["flops"] > MOST_FLOPS or nq * _span_pairs(c) > MOST_PLAIN:
        c["lens"] = "|".join(str(max(1, (2 * n) // 3)) for n in _lens(c))
    del c["name"]
    return c


# ------------------------------------------------------------------------ inputs

def _lens(c):
    return [int(n) for n in c["lens"].split("|")]


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens, nq, nkv, hd = _lens(c), c["nq"], c["nkv"], c["hd"]
    rows = sum(lens)
    qkv = torch.randn(rows, (nq + 2 * nkv) * hd, generator=gen, device="cuda")
    qkv[:, :nq * hd] *= 1.5                       # scores spread past one
    at = 0
    for n in lens:                                # sinks draw more of the rows' attention
        qkv[at:at + min(c["sinks"], n), nq * hd:(nq + nkv) * hd] *= 2.0
        at += n
    d = {"qkv": qkv.to(torch.bfloat16)}
    if c["op"] == "bias":
        d["table"] = 2.0 * torch.randn(c["buckets"], nq, generator=gen, device="cuda")
    return d


def prepare(case, seed):
    c = case
    state = _inputs(c, seed)
    state["case"] = c
    lens = _lens(c)
    state["lens"] = lens
    if c["op"] == "bias":
        # the bucket of each distance, which a program works out once
        state["far"] = _bucket_map(c)
    if own:
        import numpy as np

        import transformer_encoder_forward_gb300 as te
        state["te"] = te
        state["cu"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        state["cu_dev"] = torch.from_numpy(state["cu"]).cuda()
        state["out"] = torch.empty(sum(lens), c["nq"] * c["hd"], device="cuda", dtype=torch.bfloat16)
        if c["op"] == "bias":
            state["plan"] = te.relpos_plan(c["buckets"], c["max_distance"], c["two_sided"])
    return state


# --------------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    te, c = st["te"], st["case"]
    nq, nkv, hd = c["nq"], c["nkv"], c["hd"]
    ld, ko = (nq + 2 * nkv) * hd, nq * hd
    if c["op"] == "sink":
        te.attn_sink_fwd(st["qkv"], ld, 0, ko, ko + nkv * hd, st["cu"], st["cu_dev"], nq, nkv, hd, c["left"],
                         c["right"], c["sinks"], hd ** -0.5, st["out"], nq * hd)
    else:
        te.attn_relbias_fwd(st["qkv"], ld, 0, ko, ko + nkv * hd, st["cu"], st["cu_dev"], nq, nkv, hd, c["left"],
                            c["right"], c["sinks"], hd ** -0.5, st["plan"], st["table"], st["out"], nq * hd)
    return st["out"]


def _firsts(c):
    """The smallest distance of each bucket of one side, in whole numbers: bucket exact + k begins
    where (d / exact)^n reaches (max_distance / exact)^k, n the logarithmic buckets of the side."""
    side = c["buckets"] // 2 if c["two_sided"] else c["buckets"]
    exact_, far = side // 2, c["max_distance"]
    n = side - exact_
    firsts = list(range(exact_ + 1))
    for k in range(1, n):
        lo, hi = firsts[-1], far
        while lo < hi:
            mid = (lo + hi) // 2
            if mid ** n * exact_ ** k >= far ** k * exact_ ** n:
                hi = mid
            else:
                lo = mid + 1
        firsts.append(lo)
    return firsts


def _bucket_map(c):
    """The bucket of distance 0 .. max_distance of one side, on the device."""
    d = torch.arange(c["max_distance"] + 1, device="cuda")
    f = torch.tensor(_firsts(c), device="cuda")
    return (d[:, None] >= f).sum(1) - 1


def _chunks(c, n):
    """Row ranges of a sequence of n tokens with the keys that they can see: (first row, end, the
    first keys' end, first key of the window, its end)."""
    left, right, sinks = c["left"], c["right"], c["sinks"]
    step = max(64, min(1024, (1 << 29) // (max(1, n) * c["nq"])))
    for a in range(0, n, step):
        b = min(n, a + step)
        lo = 0 if left < 0 else max(0, a - left)
        hi = n if right < 0 else min(n, b + right)
        yield a, b, min(sinks, lo), lo, hi


def _plain(st):
    c = st["case"]
    nq, nkv, hd = c["nq"], c["nkv"], c["hd"]
    qkv, outs, at = st["qkv"], [], 0
    two = c.get("two_sided", False)
    for n in st["lens"]:
        rows = qkv[at:at + n].float()
        q = rows[:, :nq * hd].view(n, nkv, nq // nkv, hd).permute(1, 2, 0, 3)
        k = rows[:, nq * hd:(nq + nkv) * hd].view(n, nkv, 1, hd).permute(1, 2, 0, 3)
        v = rows[:, (nq + nkv) * hd:].view(n, nkv, 1, hd).permute(1, 2, 0, 3)
        for a, b, s, lo, hi in _chunks(c, n):
            i = torch.arange(a, b, device="cuda")[:, None]
            j = torch.cat([torch.arange(0, s, device="cuda"), torch.arange(lo, hi, device="cuda")])
            kk = torch.cat([k[:, :, :s], k[:, :, lo:hi]], 2)
            vv = torch.cat([v[:, :, :s], v[:, :, lo:hi]], 2)
            x = torch.matmul(q[:, :, a:b], kk.transpose(2, 3)) * hd ** -0.5
            d = j[None] - i
            if c["op"] == "bias":
                if two:
                    bucket = st["far"][d.abs().clamp(max=c["max_distance"])] + (d > 0) * (c["buckets"] // 2)
                else:
                    bucket = st["far"][(-d).clamp(0, c["max_distance"])]
                x = x + st["table"][bucket].permute(2, 0, 1).view(nkv, nq // nkv, b - a, len(j))
            hidden = torch.zeros_like(d, dtype=torch.bool)
            if c["right"] >= 0:
                hidden |= d > c["right"]
            if c["left"] >= 0:
                hidden |= (d < -c["left"]) & (j[None] >= c["sinks"])
            x = x.masked_fill(hidden, -math.inf)
            x = torch.exp(x - x.amax(3, keepdim=True))
            o = torch.matmul(x, vv) / x.sum(3, keepdim=True)
            outs.append(o.permute(2, 0, 1, 3).reshape(b - a, nq * hd).to(torch.bfloat16))
        at += n
    return torch.cat(outs)


# ----------------------------------------------------------------------- exact

def exact(case, seed):
    c = case
    st = _inputs(c, seed)
    f64 = torch.float64
    nq, nkv, hd = c["nq"], c["nkv"], c["hd"]
    lens = _lens(c)
    qkv = st["qkv"]
    out = torch.empty(sum(lens), nq * hd, dtype=f64, device="cuda")
    at = 0
    for n in lens:
        step = max(1, min(n, (1 << 26) // n))
        pos = torch.arange(n, device="cuda", dtype=f64)
        for a in range(0, n, step):
            b = min(n, a + step)
            # the keys of rows a .. b - 1 lie in [lo, hi) or among the first ones
            lo = 0 if c["left"] < 0 else max(0, a - c["left"])
            hi = n if c["right"] < 0 else min(n, b + c["right"])
            keys = torch.cat([torch.arange(0, min(lo, c["sinks"])), torch.arange(lo, hi)]).to("cuda")
            rel = pos[keys][None, :] - pos[a:b, None]
            seen = torch.ones_like(rel, dtype=torch.bool)
            if c["right"] >= 0:
                seen &= rel <= c["right"]
            if c["left"] >= 0:
                seen &= (rel >= -c["left"]) | (keys < c["sinks"])[None, :]
            if c["op"] == "bias":
                which = _bucket64(c, rel)
            for h in range(nq):
                g = h // (nq // nkv)
                q = qkv[at + a:at + b, h * hd:(h + 1) * hd].to(f64)
                k = qkv[at:at + n, (nq + g) * hd:(nq + g + 1) * hd].to(f64)[keys]
                v = qkv[at:at + n, (nq + nkv + g) * hd:(nq + nkv + g + 1) * hd].to(f64)[keys]
                x = (q @ k.T) / math.sqrt(hd)
                if c["op"] == "bias":
                    x = x + st["table"][:, h].to(f64)[which]
                x[~seen] = -math.inf
                out[at + a:at + b, h * hd:(h + 1) * hd] = torch.softmax(x, 1) @ v
        at += n
    return out


def _bucket64(c, rel):
    """Buckets from the logarithm in 64 bits; where it is a whole number but for the last bits it
    counts as that number."""
    side = c["buckets"]
    up = torch.zeros_like(rel, dtype=torch.long)
    if c["two_sided"]:
        side //= 2
        up = torch.where(rel > 0, side, 0)
        dist = rel.abs()
    else:
        dist = (-rel).clamp(min=0)
    half = side // 2
    ratio = torch.log(dist.clamp(min=half) / half) / math.log(c["max_distance"] / half)
    grown = half + torch.floor(ratio * (side - half) + 1e-9)
    return up + torch.where(dist < half, dist, grown.clamp(max=side - 1)).long()


# ------------------------------------------------------------------------ work

def _sum_to(n):
    return n * (n + 1) // 2


def _pairs(c):
    """Visible (row, key) pairs of all sequences."""
    total = 0
    for n in _lens(c):
        left = n if c["left"] < 0 else min(c["left"], n)
        right = n if c["right"] < 0 else min(c["right"], n)
        # keys j <= i + right, less those before i - left that are no sinks
        ahead = n * n - _sum_to(max(0, n - 1 - right))
        behind = _sum_to(max(0, n - 1 - left))
        s = min(c["sinks"], n)
        # of the keys before i - left, the first s stay: sum over rows of min(s, i - left)
        gone = max(0, n - 1 - left)
        kept = _sum_to(gone) if gone <= s else _sum_to(s) + (gone - s) * s
        total += ahead - behind + kept
    return total


def _span_pairs(c):
    """Pairs that the plain form's chunks go through."""
    return sum((b - a) * (s + hi - lo) for n in _lens(c) for a, b, s, lo, hi in _chunks(c, n))


def work(case):
    """q, k and v read once, the output written once; two operations a term of both products."""
    c = case
    rows, nq, nkv, hd = sum(_lens(c)), c["nq"], c["nkv"], c["hd"]
    table = 4 * c["buckets"] * nq if c["op"] == "bias" else 0
    return {"bytes": 2 * rows * hd * (2 * nq + 2 * nkv) + table, "flops": 4 * hd * nq * _pairs(c)}
