"""Attention through a window in float64, from the definition in include/specverify_kv.h, with the
error bounds that kv_plain.py derives (the arithmetic is the same; fewer slots are looked at)."""
import math

import torch

import kv_plain
from kv_plain import E4M3, U


def seen(n, m, up, window, sinks):
    """For each of m nodes (up: paths to the root) the slots it looks at, of n committed ones."""
    got = []
    for j in range(m):
        at = n + len(up[j]) - 1
        low = at - window + 1
        old = list(range(min(sinks, n))) + list(range(max(low, min(sinks, n), 0), n))
        new = [n + i for i in sorted(up[j])
               if n + len(up[i]) - 1 >= low or n + len(up[i]) - 1 < sinks]
        got.append(old + new)
    return got


def attention(q, k, v, table, kv_len, counts, parents, scale, window, sinks, k_scale=None,
              v_scale=None):
    """(out, bound, spread) as kv_plain.attention returns them."""
    B, N, HQ, D = q.shape
    H, page = k.shape[2], k.shape[1]
    G = HQ // H
    out = torch.full((B, N, HQ, D), math.nan, dtype=torch.float64)
    bound, spread = torch.zeros_like(out), torch.zeros_like(out)
    u = U[q.dtype]
    for b in range(B):
        n, m = int(kv_len[b]), int(counts[b])
        up = kv_plain.paths(None if parents is None else parents[b], N)
        for j, see in enumerate(seen(n, m, up, window, sinks)):
            at = torch.tensor(see)
            ids, off = table[b].long()[at // page], at % page
            for h in range(H):
                kk = k[:, :, h].view(torch.uint8)[ids, off].view(k.dtype).double() \
                    if k.dtype == E4M3 else k[ids, off, h].double()
                vv = v[:, :, h].view(torch.uint8)[ids, off].view(v.dtype).double() \
                    if v.dtype == E4M3 else v[ids, off, h].double()
                if k_scale is not None:
                    kk, vv = kk * k_scale[h].double(), vv * v_scale[h].double()
                x = q[b, j, h * G:(h + 1) * G].double()
                p = torch.softmax(x @ kk.T * scale, 1)
                o = p @ vv
                rows = (b, j, slice(h * G, (h + 1) * G))
                d = u + (D + 8) * 2.0 ** -23 * abs(scale) \
                    * (x.abs() @ kk.abs().T).amax(dim=1, keepdim=True) \
                    + 2.0 ** -20 + (len(see) / 64 + 1) * 2.0 ** -23
                e = 2 * d * (p @ vv.abs()) + u * o.abs() + 1e-30
                if q.dtype == torch.float16 or k.dtype == E4M3:
                    e += 2.0 ** -25 * (1 + vv.abs().sum(0))
                out[rows], bound[rows] = o, e
                spread[rows] = ((p * p) @ (vv * vv)).sqrt() + o.abs()
    return out, bound, spread


def check(got, want, dtype, counts, before=None):
    """got against (out, bound, spread), as kv_plain.check_attention compares them."""
    out, bound, spread = want
    live = ~torch.isnan(out)
    err = (got.double() - out).abs()
    bad = live & ~(err <= bound)
    assert not bool(bad.any()), \
        f"{int(bad.sum())} elements out of bound, first {bad.nonzero()[0].tolist()}: " \
        f"{got[tuple(bad.nonzero()[0])]} for {out[tuple(bad.nonzero()[0])]}"
    norm, most = float(err[live].norm()), float(spread[live].norm())
    assert norm <= (1.05 * U[dtype] + 2.0 ** -14) * most, (norm, most)
    if before is not None:
        for b in range(got.shape[0]):
            assert torch.equal(got[b, int(counts[b]):], before[b, int(counts[b]):])
