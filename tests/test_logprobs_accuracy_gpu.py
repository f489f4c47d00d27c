"""Accuracy of log probabilities, ln S and entropy on the GPU, closer than the worst case that
logprobs_plain.py allows for."""
import math

import pytest
import torch

from test_logprobs_gpu import BF, F32, built, lp, some_tokens, zipf  # noqa: F401

pytestmark = pytest.mark.gpu

F = 2.0 ** -24


def told(lp, rows, tokens, T):
    R, K = tokens.shape
    x = rows.cuda()
    f = lambda *s: torch.zeros(*s, device="cuda")
    out, norm, ent = f(R, K), f(R, 2), f(R)
    lp.spec_logprobs(x, tokens.cuda(), out, lp.logprobs_workspace(x, K), T=T, normalizer=norm,
                     entropy=ent)
    return out.cpu().double(), norm.cpu().double(), ent.cpu().double()


@pytest.mark.parametrize("dtype,T,d", [
    (F32, 1.2035620212554932, -15.0164213180542), (F32, 1.4804391860961914, -18.47092056274414),
    (F32, 1.440392017364502, -17.97126579284668), (F32, 0.6365557909011841, -7.942083358764648),
    (F32, 0.7819513082504272, -9.756132125854492), (BF, 0.8966750502586365, -11.1875),
    (BF, 1.0319277048110962, -12.875)])
@pytest.mark.parametrize("first", [0, 1000, 1 << 18])
def test_exponents_are_rounded_once(lp, dtype, T, d, first):
    """One element at 0 and 2^18 at d, whose exponent d log2(e) / T is less than a tenth of an fp32
    step from -18.  Rounded once it is -18: the weights are 2^-18, their sums whole numbers of it
    below 2^24, and S is 2.  What is left is the exponent's distance from -18 and ln's rounding; an
    exponent that is a step off (2^-19), as after two roundings, is ln S off by 2^-20 ln 2."""
    n = 1 << 18
    rows = torch.full((2, n + 1), d, dtype=dtype)
    rows[:, first] = 0.0
    assert float(rows[0, first - 1]) == d
    _, norm, _ = told(lp, rows, torch.full((2, 1), first, dtype=torch.int32), T)
    far = abs(d / T * math.log2(math.e) + 18)
    assert far < 0.1 * 2.0 ** -19
    want = math.log1p(n * math.exp(d / T))
    off = (norm[:, 1] - want).abs().max()
    assert float(off) <= far * math.log(2) + 2.0 ** -22 * want, float(off)


def in_64_bits(rows, tokens, T):
    x = (rows.double() - rows.double().amax(1, keepdim=True)) / T
    assert float(x.min()) > -32
    ln_s = x.exp().sum(1).log()
    log_p = x - ln_s[:, None]
    return x, log_p.gather(1, tokens.long()), ln_s, -(log_p.exp() * log_p).sum(1)


TEMPERATURES = [1.0, float(torch.tensor(0.7))]
SIZES = [(1 << 18, 4), (1 << 18, 64), (1 << 21, 4)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,R", SIZES)
@pytest.mark.parametrize("T", TEMPERATURES)
def test_rows_like_a_models(lp, dtype, V, R, T):
    """Of different elements, whose roundings are as good as random.  An element's sum takes 100
    additions at most, each off by 2^-25 / sqrt(3) of the sum (together 2^-23.5), and four
    exponentials of 2^-22 at most each, in different warps: S is off by 2^-22.5, one deviation.
    Four of them and the rounding of ln S (below 8: 2^-22): 1e-6.  ln p: (l - m) / T and the
    difference from ln S are below 32 and rounded by 2^-20 each: 3e-6.  H = ln S + A with A below 8
    and two such sums: 4 sqrt(2) 2^-22.5 of 8, and 1e-6: 9e-6; A is nearer to 4 and the two sums go
    together, as they round the same weights: 4e-6."""
    g = torch.Generator().manual_seed(V + R)
    rows, tokens = zipf(R, V, g, dtype), some_tokens(R, V, 16, g)
    out, norm, ent = told(lp, rows, tokens, T)
    x, want, ln_s, H = in_64_bits(rows, tokens, T)
    assert float(ln_s.max()) < 8
    off = [float(e.abs().max()) for e in (out - want, norm[:, 1] - ln_s, ent - H)]
    assert off[0] <= 3e-6 and off[1] <= 1e-6 and off[2] <= 4e-6, off


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,R", SIZES)
@pytest.mark.parametrize("T", TEMPERATURES)
def test_rows_of_many_small_elements(lp, dtype, V, R, T):
    """Nearly equal ones that weigh as much as the large one: their roundings add up.  An exponent
    is off by 2^-24 for the difference and 2^-24 for itself, of |x| <= X; the exponential by 2^-22
    and at most three more that join sums with it (the row has one maximum, so that a warp's
    reference is raised at most once beyond its first batch); a sum of n additions by n 2^-24: 17 in
    a batch of 32 elements, one per batch of a thread (V / 8192, twice that for batches of 16), 5
    and 3 for lanes and warps and 7 for CTAs with a product each."""
    g = torch.Generator().manual_seed(V + R)
    rows = torch.randn(R, V, generator=g) * 0.01 - math.log(V) * T
    rows[torch.arange(R), torch.randint(0, V, (R,), generator=g)] = 0.0
    rows, tokens = rows.to(dtype), some_tokens(R, V, 16, g)
    out, norm, ent = told(lp, rows, tokens, T)
    x, want, ln_s, H = in_64_bits(rows, tokens, T)
    X = float(x.abs().max())
    batches = V / (8192 if dtype == BF else 4096) / (8 if R == 4 else 2)
    n = 17 + batches + 5 + 2 * 3 + 2 * 7
    rs = n * F + 4 * 2.0 ** -22 + 2 * F * X
    s = rs + 4 * F * float(ln_s.max())
    off = [float(e.abs().max()) for e in (out - want, norm[:, 1] - ln_s, ent - H)]
    assert off[1] <= s, (off, s)
    assert off[0] <= s + 2 * 2.0 ** -20, (off, s)
    # H = ln S + A, A <= X with both sums' errors (and a rounding of each difference)
    assert off[2] <= s + X * (2 * rs + 2 * F) + 2 * F * float(H.max()), (off, s)
