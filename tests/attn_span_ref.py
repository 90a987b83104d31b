"""Plain 64-bit attention with limits to either side, sinks and a bucketed
relative position bias, for the tests of te.attn_sink_fwd and
te.attn_relbias_fwd (torch, on the inputs' device)."""
import math

NEG = float("-inf")


def bucket_of(d, buckets, max_distance, two_sided):
    """The bucket of one distance d = j - i, from the definition: logarithms in
    64 bits, whole values decided in whole numbers."""
    side = buckets // 2 if two_sided else buckets
    up = side if two_sided and d > 0 else 0
    a = abs(d) if two_sided else max(-d, 0)
    exact = side // 2
    n = side - exact
    if a < exact:
        return up + a
    if a >= max_distance:
        return up + side - 1
    k = int(n * math.log(a / exact) / math.log(max_distance / exact))
    # (a / exact)^n against (max_distance / exact)^k
    while k > 0 and a ** n < max_distance ** k * exact ** (n - k):
        k -= 1
    while k + 1 < n and a ** n >= max_distance ** (k + 1) * exact ** (n - k - 1):
        k += 1
    return up + exact + min(k, n - 1)


def bucket_table(n, buckets, max_distance, two_sided):
    """Buckets of the distances -(n - 1) .. n - 1."""
    return [bucket_of(d, buckets, max_distance, two_sided) for d in range(1 - n, n)]


def visible(n, left, right, sinks, device="cpu"):
    import torch
    i = torch.arange(n, device=device)[:, None]
    j = torch.arange(n, device=device)[None]
    see = torch.ones(n, n, dtype=torch.bool, device=device)
    if right >= 0:
        see &= j <= i + right
    if left >= 0:
        see &= (j >= i - left) | (j < sinks)
    return see


def attention(qkv, lens, nq, nkv, hd, left, right, sinks, scale, offs=None, table=None, rel=None):
    """(o, a): the outputs [rows, nq * hd] in f64 and sum_j p_j |v_j|, which the
    weights' rounding scales with.  offs: columns of q, k, v; rel: (buckets,
    max_distance, two_sided)."""
    import torch
    f64 = torch.float64
    q_off, k_off, v_off = offs or (0, nq * hd, (nq + nkv) * hd)
    rows = sum(lens)
    o = torch.zeros(rows, nq * hd, dtype=f64, device=qkv.device)
    mag = torch.zeros_like(o)
    at = 0
    for n in lens:
        x = qkv[at:at + n]
        see = visible(n, left, right, sinks, qkv.device)
        if table is not None:
            b = torch.tensor(bucket_table(n, *rel), device=qkv.device)
            i = torch.arange(n, device=qkv.device)
            which = b[i[None] - i[:, None] + n - 1]
        for h in range(nq):
            g = h // (nq // nkv)
            q = x[:, q_off + h * hd:q_off + (h + 1) * hd].to(f64)
            k = x[:, k_off + g * hd:k_off + (g + 1) * hd].to(f64)
            v = x[:, v_off + g * hd:v_off + (g + 1) * hd].to(f64)
            s = q @ k.T * scale
            if table is not None:
                s = s + table[:, h].to(f64)[which]
            s = torch.where(see, s, torch.full_like(s, NEG))
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - torch.where(m == NEG, torch.zeros_like(m), m))
            den = p.sum(1, keepdim=True)
            p = torch.where(den > 0, p / den, torch.zeros_like(p))
            # a weight of 0 takes nothing, whatever the value
            fin = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
            bad = ((p > 0).to(f64) @ (~torch.isfinite(v)).to(f64)) > 0
            y, a = p @ fin, p @ fin.abs()
            y[bad] = float("nan")
            o[at:at + n, h * hd:(h + 1) * hd] = y
            mag[at:at + n, h * hd:(h + 1) * hd] = a
        at += n
    return o, mag


def bound(o, mag):
    """Largest error of a bf16 output.  Each weight is rounded to bf16 (2^-8 of
    itself, so 2^-8 of mag in all, and what the sum of the unrounded weights
    divides is off by nothing more), the output once more (2^-8 of itself); scores
    carry f32 sums of hd <= 128 products, |score| <= 40 in log2 units, so 128 *
    2^-24 * 40 = 3e-4 of each weight and as much of their sum: 2^-10 and some of
    mag; 2^-126 for outputs that vanish."""
    return mag * (2.0 ** -8 + 2.0 ** -9) + o.abs() * 2.0 ** -8 + 2.0 ** -126
