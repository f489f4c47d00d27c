"""A plain float64 implementation of the paged cache calls, and error bounds for them.

Everything here works slot by slot on CPU tensors, from the definitions in
include/specverify_kv.h.  A rounding to a type is off by at most half a step,
u = finfo(type).eps / 2 relative to the value (bf16 2^-8, fp16 2^-11, fp32 2^-24,
e4m3 2^-4 and, below its normal range, 2^-10 absolute).
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
     torch.float8_e4m3fn: 2.0 ** -4}
E4M3 = torch.float8_e4m3fn


def paths(parents, N):
    """For each node the nodes from itself up to the root (parents None: a chain)."""
    up = [[0]]
    for j in range(1, N):
        up.append([j] + up[j - 1 if parents is None else int(parents[j])])
    return up


def slots(table_row, page_size, count):
    return [(int(table_row[s // page_size]), s % page_size) for s in range(count)]


def entries(pool, scale, table_row, count, head):
    """The first `count` entries of one head in float64."""
    page_size = pool.shape[1]
    got = torch.stack([pool[p, s, head].double() for p, s in slots(table_row, page_size, count)]) \
        if count else torch.zeros(0, pool.shape[-1], dtype=torch.float64)
    return got if scale is None else got * scale[head].double()


def attention(q, k, v, table, kv_len, counts, parents, scale, k_scale=None, v_scale=None):
    """(out, bound, spread): out [B, N, q_heads, dim] float64 (NaN in rows past counts), the largest
    error that the fp32 sums and 16-bit weights may leave in each element, and the typical size of
    the weights' rounding errors in units of their u.

    The bound.  With every weight off by a relative d, |error| <= 2 d sum_l p_l |v_l| (once in the
    numerator, once in the sum).  d is the rounding of the weight to the 16-bit type (u) plus the
    score's error: (dim + 8) additions and products, each within 2^-23 (the tensor cores cut,
    rather than round, some bits) of sum_d |q_d k_d|, times |scale|; plus 2^-20 for the exponential
    and the running sums' rescaling, and 2^-23 per 64 positions for the sums' length.  Rounding
    the result adds u of the result's type.  Halves (fp16 results; the weights of fp16 and float8
    caches, relative to the largest) are rounded to steps of 2^-24 at the finest: half of one of
    the result's, and of every weight's times |v|."""
    B, N, HQ, D = q.shape
    H = k.shape[2]
    out = torch.full((B, N, HQ, D), math.nan, dtype=torch.float64)
    bound, spread = torch.zeros_like(out), torch.zeros_like(out)
    u = U[q.dtype]
    for b in range(B):
        n, m = int(kv_len[b]), int(counts[b])
        up = paths(None if parents is None else parents[b], N)
        for h in range(H):
            ks = entries(k, k_scale, table[b], n + m, h)
            vs = entries(v, v_scale, table[b], n + m, h)
            for j in range(m):
                see = torch.tensor(list(range(n)) + sorted(n + i for i in up[j]))
                kk, vv = ks[see], vs[see]
                for g in range(HQ // H):
                    x = q[b, j, h * (HQ // H) + g].double()
                    s = (kk @ x) * scale
                    p = torch.softmax(s, 0)
                    o = p @ vv
                    at = (b, j, h * (HQ // H) + g)
                    out[at] = o
                    d = u + (D + 8) * 2.0 ** -23 * abs(scale) * float((kk.abs() @ x.abs()).max()) \
                        + 2.0 ** -20 + (len(see) / 64 + 1) * 2.0 ** -23
                    bound[at] = 2 * d * (p @ vv.abs()) + u * o.abs() + 1e-30
                    if q.dtype == torch.float16 or k.dtype == E4M3:
                        bound[at] += 2.0 ** -25 * (1 + vv.abs().sum(0))
                    spread[at] = ((p * p) @ (vv * vv)).sqrt() + o.abs()
    return out, bound, spread


def check_attention(got, q, k, v, table, kv_len, counts, parents, scale, k_scale=None,
                    v_scale=None, before=None):
    """Rows within counts against the bound element by element, and in the 2-norm: independent
    roundings of at most u each, of the weights and of the result, have a norm below u times the
    norm of `spread`; a twentieth more, and 2^-14 of it, for the fp32 part.  Rows past counts
    unchanged."""
    out, bound, spread = attention(q, k, v, table, kv_len, counts, parents, scale, k_scale, v_scale)
    live = ~torch.isnan(out)
    err = (got.double() - out).abs()
    bad = live & ~(err <= bound)
    assert not bool(bad.any()), \
        f"{int(bad.sum())} elements out of bound, first {bad.nonzero()[0].tolist()}: " \
        f"{got[tuple(bad.nonzero()[0])]} for {out[tuple(bad.nonzero()[0])]}"
    norm, most = float(err[live].norm()), float(spread[live].norm())
    assert norm <= (1.05 * U[q.dtype] + 2.0 ** -14) * most, (norm, most)
    if before is not None:
        for b in range(q.shape[0]):
            assert torch.equal(got[b, int(counts[b]):], before[b, int(counts[b]):])


def rates(rot, base, factor=1.0, original=0, low=1.0, high=32.0):
    """Radians per position of each pair."""
    got = []
    for i in range(rot // 2):
        r = base ** (-2.0 * i / rot)
        keep = 0.0
        if original > 0:
            keep = min(1.0, max(0.0, (original * r / (2 * math.pi) - low) / (high - low)))
        got.append(keep * r + (1.0 - keep) * r / factor)
    return torch.tensor(got, dtype=torch.float64)


def rotate(x, pos, rate, interleaved, magnitude=1.0):
    """(rotated, slack) of x [..., dim] at one position; slack: |a| + |b| of each element's pair
    (zero where nothing is rotated)."""
    x = x.double()
    half = len(rate)
    i = torch.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, slack = x.clone(), torch.zeros_like(x)
    if half:
        c, s = torch.cos(pos * rate), torch.sin(pos * rate)
        a, b = x[..., one], x[..., two]
        y[..., one] = magnitude * (a * c - b * s)
        y[..., two] = magnitude * (b * c + a * s)
        slack[..., one] = slack[..., two] = abs(magnitude) * (a.abs() + b.abs())
    return y, slack


def stored_bound(y, slack, dtype, scale=None):
    """Error of a rotated value held in `dtype`: the angle's conversion to fp32 (pi 2^-24), the
    cosine and sine (2^-23 each), their product with the magnitude, two products and a sum
    (4 * 2^-24), of |a| + |b|: below 12 * 2^-24 of it; then (for a scaled entry: the quotient,
    2^-24, and) the rounding to the type."""
    f = 12 * 2.0 ** -24 * slack + 2.0 ** -23 * y.abs()
    b = f + U[dtype] * (y.abs() + f)
    return b + 2.0 ** -10 * scale if dtype == E4M3 else b + 2.0 ** -25
