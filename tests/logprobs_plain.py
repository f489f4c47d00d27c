"""Log probabilities, entropy, alternatives and their gradient in float64, from the definitions in
include/specverify_logprobs.h, with bounds on what fp32 arithmetic may leave.

Bounds, x = (l - m) / T <= 0.  The exponent x log2(e) is off by at most 4 * 2^-24 of itself (the
difference, the factor's own rounding, the product, and the running maximum's change), the
exponential by 2^-21 besides.  So a term of S is off by 2^-21 + 4 * 2^-24 |x| relative, S itself by
    rS = 2^-21 + 4 * 2^-24 A + n 2^-24,    A = sum p |x|,
n additions and rescalings on the longest path: a thread's share of the row (V / 256, and three per
batch of 16 at least) and 64 for what joins threads, warps and CTAs.  ln S adds 2^-22 of itself:
    log p:  rS + 2^-22 ln S + 3 * 2^-24 |x| + 2^-24 |log p|;
    H = ln S + A:  rS + 2^-22 ln S + A (rS + rA) + 2^-23 H,   rA the same as rS with
        A2 = sum p x^2 / A in the place of A.
The gradient takes m and ln S as given: x - ln S is off by d = 3 * 2^-24 |x| + 2^-24 |log p|, p by
d + 2^-21 + 2^-23 |log p| relative (the exponent in base 2), the sum of given gradients by 2^-24
per term, the bracket by 2^-22 of its parts, 1 / T by 2^-23; then the rounding to the type.  Below
2^-126 the exponential is zero."""
import math

import torch

F = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def forward(l, tokens, T, top):
    """Of rows l [R, V] (float64) and tokens [R, K]: a dict of (value, bound)."""
    R, V = l.shape
    m = l.max(dim=1).values
    x = (l - m[:, None]) / T
    e = x.exp()
    S = e.sum(1)
    p, ln_s = e / S[:, None], S.log()
    fx = torch.where(p > 0, x, 0.0)  # (x may be -inf where p is 0)
    A = -(p * fx).sum(1)
    A2 = torch.where(A > 0, (p * fx * fx).sum(1) / A.clamp(min=1e-300), 0.0)
    n = V / 256 * (1 + 3 / 16) + 64
    rs = 2.0 ** -21 + 4 * F * A + n * F
    ra = 2.0 ** -21 + 4 * F * A2 + n * F

    def told(at):
        v = x.gather(1, at) - ln_s[:, None]
        b = (rs + 4 * F * ln_s)[:, None] + 3 * F * x.gather(1, at).abs() + F * v.abs()
        return v, torch.where(torch.isinf(v), 0.0, b)

    H = ln_s + A
    r = {"logprobs": told(tokens.clamp(0, V - 1).long()),
         "normalizer": (torch.stack([m, ln_s], 1), torch.stack([0 * m, rs + 4 * F * ln_s], 1)),
         "entropy": (H, rs + 4 * F * ln_s + A * (rs + ra) + 2 * F * H + 1e-30)}
    if top:
        order = l.sort(dim=1, descending=True, stable=True).indices[:, :top]
        tt = torch.full((R, top), -1, dtype=torch.int32)
        tl = torch.full((R, top), -math.inf, dtype=torch.float64)
        tb = torch.zeros(R, top, dtype=torch.float64)
        tt[:, :V] = order.to(torch.int32)
        tl[:, :V], tb[:, :V] = told(order)
        r["top_tokens"], r["top_logprobs"] = (tt, None), (tl, tb)
    return r


def gradient(l, tokens, normalizer, entropy, g, gh, T, dtype):
    """(gradient, bound) of rows l [R, V] (float64); normalizer, entropy, g, gh as the call takes
    them (float64); gh None: no entropy term.  tokens of -1 hold none."""
    R, V = l.shape
    live = tokens >= 0
    g = torch.where(live, g, 0.0)
    x = (l - normalizer[:, :1]) / T
    lp = x - normalizer[:, 1:]
    p = lp.exp()
    fx, flp = (torch.where(p > 0, y, 0.0) for y in (x, lp))
    total, size = g.sum(1, keepdim=True), g.abs().sum(1, keepdim=True)
    bracket = total.expand(R, V)
    parts = total.abs().expand(R, V)
    K = g.shape[1]
    d = 3 * F * fx.abs() + F * flp.abs()
    slip = (K * F * size).expand(R, V)
    if gh is not None:
        ge = torch.where(live.any(1), gh, 0.0)[:, None]
        bracket = bracket + ge * (flp + entropy[:, None])
        parts = parts + ge.abs() * (flp.abs() + entropy[:, None].abs())
        slip = slip + ge.abs() * d
    own = torch.zeros(R, V, dtype=torch.float64).scatter_add_(1, tokens.clamp(min=0).long(), g)
    own_size = torch.zeros(R, V, dtype=torch.float64).scatter_add_(1, tokens.clamp(min=0).long(),
                                                                   g.abs())
    y = (own - p * bracket) / T
    rp = d + 2.0 ** -21 + 2 * F * flp.abs()
    b = (p * (rp * bracket.abs() + slip + 4 * F * parts) + (K + 2) * F * own_size
         + 2.0 ** -126 * parts) / T
    b = b + 2 * F * y.abs()
    return y, b + U[dtype] * (y.abs() + b) + 2.0 ** -133
