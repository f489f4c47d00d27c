"""Log probabilities and their gradient on the GPU against the plain float64 implementation
(logprobs_plain.py): every type, odd and ragged rows, ties, masks, alternatives that lie together,
rows without tokens, bad data, streams, captured graphs, and rounds with the verify calls."""
import math

import pytest
import torch

import logprobs_plain as plain
from parity import Guarded

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verification_18_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(scope="module")
def lp():
    from speculative_decoding_verification_18_gb300 import logprobs
    return logprobs


def zipf(R, V, g, dtype=F32):
    base = -1.1 * torch.arange(1, V + 1, dtype=torch.float32).log()
    return (base[torch.randperm(V, generator=g)] + torch.randn(R, V, generator=g)).to(dtype)


def strided(rows, pitch):
    """A device copy of rows [R, V] that lie `pitch` elements apart, NaN between them."""
    R, V = rows.shape
    held = torch.full((R * pitch + 8,), math.nan, dtype=rows.dtype, device="cuda")
    view = held[:R * pitch].view(R, pitch)[:, :V]
    view.copy_(rows)
    return view


class Told:
    """One call of spec_logprobs on guarded buffers; what rows without tokens hold is 7."""

    def __init__(self, lp, rows, tokens, T=1.0, top=0, entropy=True, normalizer=True, pitch=None,
                 status=True, stream=None):
        R, V = rows.shape
        K = tokens.shape[1]
        gd = Guarded()
        x = strided(rows, pitch or V)
        f = lambda *s: gd.empty(s, F32, fill=7.0)
        self.logprobs = f(R, K)
        self.entropy = f(R) if entropy else None
        self.normalizer = f(R, 2) if normalizer else None
        self.top_tokens = gd.empty((R, top), torch.int32, fill=7) if top else None
        self.top_logprobs = f(R, top) if top else None
        st = gd.empty((R,), torch.int32, fill=0) if status else None
        n = lp.spec_logprobs_workspace_size(R, V, 0 if rows.dtype == BF else 1, K, top)
        ws = gd.empty((n,), torch.uint8, fill=255)
        lp.spec_logprobs(x, tokens.cuda(), self.logprobs, ws, T=T, entropy=self.entropy,
                         normalizer=self.normalizer, top_tokens=self.top_tokens,
                         top_logprobs=self.top_logprobs, status=st)
        gd.check()
        self.status = st.tolist() if status else None

    def check(self, rows, tokens, T=1.0, top=0):
        live = (tokens >= 0).any(1)
        want = plain.forward(rows.double(), tokens, T, top)
        for name, (v, b) in want.items():
            got = getattr(self, name)
            if got is None:
                continue
            got = got.cpu()
            assert bool((got[~live] == 7).all()), name
            got, v = got[live], v[live]
            if name == "top_tokens":
                assert torch.equal(got, v)
                continue
            ok = (got.double() - v).abs() <= b[live]
            ok |= torch.isinf(v) & (got.double() == v)
            if name == "logprobs":
                none = tokens[live] < 0
                assert bool((got[none] == 7).all())
                ok |= none
            assert bool(ok.all()), (name, (~ok).nonzero()[:4].tolist(), got[~ok][:4], v[~ok][:4])


def some_tokens(R, V, K, g, gone=0.0):
    t = torch.randint(0, V, (R, K), generator=g).to(torch.int32)
    return torch.where(torch.rand(R, K, generator=g) < gone, -1, t).to(torch.int32)


# ---------------------------------------------------------------- forward

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 33, 100, 257, 1000, 2049, 4099, 40000, 65537])
@pytest.mark.parametrize("top,given", [(0, 1), (1, 2), (5, 3), (64, 64)])
def test_sizes(lp, dtype, V, top, given):
    g = torch.Generator().manual_seed(V + top)
    rows, tokens = zipf(5, V, g, dtype), some_tokens(5, V, given, g)
    T = 0.7 if given == 2 else 1.0
    Told(lp, rows, tokens, T, top).check(rows, tokens, T, top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,more", [(1000, 1), (1001, 7), (4099, 61), (40000, 3), (50001, 63)])
def test_rows_at_every_alignment(lp, dtype, V, more):
    g = torch.Generator().manual_seed(V)
    rows, tokens = zipf(17, V, g, dtype), some_tokens(17, V, 2, g)
    Told(lp, rows, tokens, 1.3, 9, pitch=V + more).check(rows, tokens, 1.3, 9)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,V", [(1, 300001), (1, 256000), (3, 128256), (40, 32000), (150, 70001),
                                 (700, 20000), (3000, 3001)])
def test_batches(lp, dtype, R, V):
    g = torch.Generator().manual_seed(R)
    rows, tokens = zipf(R, V, g, dtype), some_tokens(R, V, 2, g, gone=0.3)
    Told(lp, rows, tokens, 0.8, 20).check(rows, tokens, 0.8, 20)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_largest_vocabulary(lp, dtype):
    V, g = 1 << 21, torch.Generator().manual_seed(2)
    rows, tokens = zipf(2, V, g, dtype), some_tokens(2, V, 64, g)
    Told(lp, rows, tokens, 1.0, 64).check(rows, tokens, 1.0, 64)
    gradient_case(lp, rows, tokens, 1.0, True, V, V)


@pytest.mark.parametrize("optional", [dict(entropy=False), dict(normalizer=False),
                                      dict(entropy=False, normalizer=False, status=False)])
def test_outputs_that_nobody_wants(lp, optional):
    g = torch.Generator().manual_seed(0)
    rows, tokens = zipf(9, 5000, g), some_tokens(9, 5000, 1, g)
    Told(lp, rows, tokens, 1.0, 0, **optional).check(rows, tokens)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,R", [(1500, 3), (70000, 2), (140000, 2), (40000, 700)])
@pytest.mark.parametrize("what", ["constant", "falling", "rising", "few values", "together",
                                  "one place", "huge"])
@pytest.mark.parametrize("top", [1, 20, 64])
def test_alternatives(lp, dtype, V, R, what, top):
    """Ties go to the lower token; large elements that lie together, in one thread's vectors or
    all over, are found like any others."""
    g = torch.Generator().manual_seed(top)
    v = torch.arange(V, dtype=torch.float32)
    row = {"constant": torch.full((V,), -1.25), "falling": -v / V * 30, "rising": v / V * 30,
           "few values": torch.randint(0, 4, (V,), generator=g).float(),
           "together": torch.where((v >= 700) & (v < 1400), 5.0 + v * 1e-3, -v * 1e-5),
           "one place": torch.where((v.long() // (8 if dtype == BF else 4)) % 256 < 18,
                                    torch.randn(V, generator=g), -50.0 - v / V),
           "huge": torch.randn(V, generator=g) * 1e37}[what]
    some = min(R, 3)
    rows = (row + torch.zeros(some, 1)).to(dtype)
    rows[-1] = rows[-1].flip(0)
    rows = rows[torch.arange(R) % some]
    tokens = some_tokens(R, V, 1, g)
    got = Told(lp, rows, tokens, 1.0, top)
    if R > some:  # the rows repeat: compare their alternatives, and the first ones in full
        assert torch.equal(got.top_tokens.cpu(), got.top_tokens.cpu()[torch.arange(R) % some])
        for n in ("logprobs", "entropy", "normalizer", "top_tokens", "top_logprobs"):
            setattr(got, n, getattr(got, n)[:some])
        rows, tokens = rows[:some], tokens[:some]
    got.check(rows, tokens, 1.0, top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [50, 3000, 70001])
@pytest.mark.parametrize("mask", [-math.inf, None])
def test_masks(lp, dtype, V, mask):
    """Tokens that are not allowed: -inf or the type's lowest value, all but one, a few, whole
    stretches; asked about and among the alternatives."""
    g = torch.Generator().manual_seed(V)
    mask = torch.finfo(dtype).min if mask is None else mask
    rows = zipf(6, V, g, dtype)
    rows[0, :] = mask
    rows[0, V // 2] = -3.0                      # one token left
    rows[1, 1:] = mask
    rows[2, :V - 1] = mask
    rows[3, torch.rand(V, generator=g) < 0.9] = mask
    rows[3, 0] = 0.0
    rows[4, V // 3:] = mask
    rows[5, 5] = mask
    tokens = torch.tensor([[V // 2, 0], [0, V - 1], [V - 1, 0], [0, 1], [0, V - 1], [5, 6]],
                          dtype=torch.int32)
    got = Told(lp, rows, tokens, 1.0, 30)
    assert got.status == [0] * 6
    if mask == -math.inf:
        got.check(rows, tokens, 1.0, 30)
        assert float(got.logprobs[0, 1]) == -math.inf
        assert got.logprobs[:3, :1].cpu().flatten().tolist()[:1] == [0.0]
        assert got.entropy[:3].tolist() == [0.0] * 3
        return
    want = plain.forward(rows.double(), tokens, 1.0, 30)
    assert torch.equal(got.top_tokens.cpu(), want["top_tokens"][0])
    for name in ("logprobs", "top_logprobs", "entropy", "normalizer"):
        v, b = want[name]
        d = (getattr(got, name).cpu().double() - v).abs()
        assert bool((d <= b).all()), name


def test_first_and_lowest_zero(lp):
    """-0 and +0 are equal logits."""
    rows = torch.full((2, 300), -1.0)
    rows[0, [7, 100]] = torch.tensor([-0.0, 0.0])
    rows[1, [7, 100]] = torch.tensor([0.0, -0.0])
    got = Told(lp, rows, torch.zeros(2, 1, dtype=torch.int32), 1.0, 3)
    assert got.top_tokens.tolist() == [[7, 100, 0]] * 2


@pytest.mark.parametrize("T", [1e-30, 1e-3, 0.3, 5.0, 1e30])
def test_temperatures(lp, T):
    """Cold: one token has it all.  Hot: all the same."""
    g = torch.Generator().manual_seed(1)
    rows, tokens = zipf(3, 2000, g), some_tokens(3, 2000, 2, g)
    got = Told(lp, rows, tokens, T, 4)
    assert got.status == [0] * 3
    if T >= 1e-3:
        got.check(rows, tokens, T, 4)
    else:
        assert got.entropy.tolist() == [0.0] * 3
        assert got.top_logprobs[:, 0].tolist() == [0.0] * 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [100, 70001])
def test_bad_rows_and_tokens(lp, dtype, V):
    g = torch.Generator().manual_seed(V)
    rows = zipf(9, V, g, dtype)
    clean = rows.clone()
    rows[0, V - 1] = math.nan
    rows[1, 0] = math.inf
    rows[2, :] = -math.inf
    rows[3, :] = math.nan
    rows[4, V // 2] = -math.nan
    tokens = some_tokens(9, V, 3, g)
    tokens[5, 1] = V
    tokens[6, 0] = -2
    tokens[7] = -1
    rows[7] = math.nan                      # nothing is asked: not read
    tokens[3, 2] = -1
    got = Told(lp, rows, tokens, 1.0, 6)
    R, K = 0x1, 0x2
    assert got.status == [R, R, R, R, R, K, K, 0, 0]
    for b in range(5):
        for x in (got.entropy[b], got.normalizer[b], got.top_logprobs[b]):
            assert bool(torch.isnan(x).all())
        assert got.top_tokens[b].tolist() == [-1] * 6
        at = tokens[b] >= 0
        assert bool(torch.isnan(got.logprobs[b].cpu()[at]).all())
        assert bool((got.logprobs[b].cpu()[~at] == 7).all())
    assert math.isnan(float(got.logprobs[5, 1])) and math.isnan(float(got.logprobs[6, 0]))
    ok = torch.tensor([5, 6, 7, 8])
    got.logprobs[5, 1] = got.logprobs[6, 0] = 7.0
    tokens[5, 1] = tokens[6, 0] = -1
    for n in ("logprobs", "entropy", "normalizer", "top_tokens", "top_logprobs"):
        setattr(got, n, getattr(got, n).cpu()[ok])
    got.check(clean[ok], tokens[ok], 1.0, 6)


def test_rows_past_32_bits(lp):
    """More than 2^32 bytes and 2^31 elements into the logits."""
    R, V = 16500, 131072
    x = torch.zeros(R, V, dtype=BF, device="cuda")
    tokens = torch.full((R, 1), -1, dtype=torch.int32)
    tokens[-1] = 77
    g = torch.Generator().manual_seed(0)
    last = zipf(1, V, g, BF)
    x[-1:] = last.cuda()
    out, norm = torch.full((R, 1), 7.0, device="cuda"), torch.zeros(R, 2, device="cuda")
    tt, tl = torch.zeros(R, 4, dtype=torch.int32, device="cuda"), torch.zeros(R, 4, device="cuda")
    lp.spec_logprobs(x, tokens.cuda(), out, lp.logprobs_workspace(x, 1, 4), normalizer=norm,
                     top_tokens=tt, top_logprobs=tl)
    want = plain.forward(last.double(), tokens[-1:], 1.0, 4)
    assert abs(float(out[-1]) - float(want["logprobs"][0])) <= float(want["logprobs"][1])
    assert torch.equal(tt[-1:].cpu(), want["top_tokens"][0]) and bool((out[:-1] == 7).all())
    g1 = torch.ones(R, 1, device="cuda")
    lp.spec_logprobs_grad(x, tokens.cuda(), norm, g1, x)
    y, b = plain.gradient(last.double(), tokens[-1:], norm[-1:].cpu().double(), None,
                          torch.ones(1, 1, dtype=torch.float64), None, 1.0, BF)
    assert bool(((x[-1:].cpu().double() - y).abs() <= b).all())
    assert int(torch.count_nonzero(x[:-1])) == 0


def test_nothing_to_do(lp):
    x = torch.zeros(0, 100, device="cuda")
    e = torch.zeros(0, 1, device="cuda")
    t = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    lp.spec_logprobs(x, t, e, lp.logprobs_workspace(x))
    lp.spec_logprobs_grad(x, t, torch.zeros(0, 2, device="cuda"), e, x)


# ---------------------------------------------------------------- gradient

def gradient_case(lp, rows, tokens, T, entropy, pitch, out_pitch, seed=0, in_place=False):
    g = torch.Generator().manual_seed(seed)
    R, V = rows.shape
    told = Told(lp, rows, tokens, T, 0)
    norm, ent = told.normalizer, told.entropy
    gl = torch.randn(tokens.shape, generator=g)
    gh = torch.randn(R, generator=g) if entropy else None
    x = strided(rows, pitch)
    gd = Guarded()
    flat = gd.empty((R * out_pitch,), rows.dtype, fill=7.0)
    out = flat.view(R, out_pitch)[:, :V] if not in_place else x
    st = gd.empty((R,), torch.int32, fill=0)
    d = lambda t: None if t is None else t.cuda()
    lp.spec_logprobs_grad(x, tokens.cuda(), norm, d(gl), out, T=T, entropy=ent if entropy else None,
                          grad_entropy=d(gh), status=st)
    gd.check()
    if not in_place:  # between the rows nothing is written
        assert bool((flat.view(R, out_pitch)[:, V:] == 7).all())
    y, b = plain.gradient(rows.double(), tokens, norm.cpu().double(), ent.cpu().double(),
                          gl.double(), None if gh is None else gh.double(), T, rows.dtype)
    live = (tokens >= 0).any(1)
    got = out.cpu().double()
    assert bool((got[~live] == 0).all())
    ok = ((got - y).abs() <= b)[live]
    assert bool(ok.all()), ((~ok).nonzero()[:4].tolist(), got[live][~ok][:4], y[live][~ok][:4])
    assert st.tolist() == [0] * R
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 33, 257, 1000, 16385, 40000, 65537])
@pytest.mark.parametrize("given,entropy,T", [(1, False, 1.0), (3, True, 0.7), (64, True, 1.3)])
def test_gradient_sizes(lp, dtype, V, given, entropy, T):
    g = torch.Generator().manual_seed(V)
    rows, tokens = zipf(5, V, g, dtype), some_tokens(5, V, given, g, gone=0.2)
    gradient_case(lp, rows, tokens, T, entropy, V, V)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,more,out_more", [(1000, 1, 0), (1001, 7, 7), (4099, 61, 1),
                                             (40000, 3, 8), (30001, 63, 0), (3001, 0, 2)])
def test_gradient_alignments(lp, dtype, V, more, out_more):
    g = torch.Generator().manual_seed(V)
    rows, tokens = zipf(17, V, g, dtype), some_tokens(17, V, 4, g)
    gradient_case(lp, rows, tokens, 1.0, True, V + more, V + out_more)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 9, 24, 130, 2047, 8200, 16390])
@pytest.mark.parametrize("more", [1, 3, 4, 5])
def test_gradient_every_shift(lp, dtype, V, more):
    """Logits and gradient at every pair of places of a 16-byte word, row after row; the first and
    the last vectors of rows, of warps and of CTAs' parts."""
    g = torch.Generator().manual_seed(V)
    rows, tokens = zipf(17, V, g, dtype), some_tokens(17, V, 2, g, gone=0.1)
    tokens[0] = V - 1
    even = (V + 15) // 8 * 8
    gradient_case(lp, rows, tokens, 1.0, True, even + more, even)
    gradient_case(lp, rows, tokens, 1.0, False, even, even + more)
    gradient_case(lp, rows, tokens, 1.0, True, even + more, even + 2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_repeated_tokens_in_place(lp, dtype):
    """The same token many times, at part borders and row ends; the gradient over its logits."""
    V = 40001
    g = torch.Generator().manual_seed(3)
    rows = zipf(6, V, g, dtype)
    tokens = some_tokens(6, V, 40, g, gone=0.1)
    tokens[0] = 5
    tokens[1, ::2] = V - 1
    tokens[2, 1::3] = 0
    tokens[3, :20] = torch.arange(16376, 16396)
    tokens[4] = -1
    one = gradient_case(lp, rows, tokens, 0.9, True, V + 7, V, seed=1)
    two = gradient_case(lp, rows, tokens, 0.9, True, V + 7, V, seed=1, in_place=True)
    assert torch.equal(one, two)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_masked_rows(lp, dtype):
    """-inf and lowest logits get no gradient, but a given one its own; the entropy term there is
    zero, not NaN."""
    V = 5001
    g = torch.Generator().manual_seed(4)
    rows = zipf(3, V, g, dtype)
    rows[0, 100:4000] = -math.inf
    rows[1, 100:4000] = torch.finfo(dtype).min
    rows[2, 1:] = -math.inf
    tokens = torch.tensor([[0, 200, 200], [1, 300, -1], [0, 4000, 0]], dtype=torch.int32)
    out = gradient_case(lp, rows, tokens, 1.0, True, V, V).cpu()
    assert bool((out[:2, 1000:4000] == 0).all())


def test_gradient_of_bad_rows(lp):
    V, g = 3000, torch.Generator().manual_seed(5)
    rows = zipf(5, V, g)
    tokens = some_tokens(5, V, 2, g)
    norm = torch.zeros(5, 2)
    norm[:, 1] = 8.0
    norm[0, 0], norm[1, 1], norm[2, 1] = math.nan, math.nan, math.inf
    tokens[3, 1] = V
    out = torch.zeros(5, V, device="cuda")
    st = torch.zeros(5, dtype=torch.int32, device="cuda")
    lp.spec_logprobs_grad(rows.cuda(), tokens.cuda(), norm.cuda(), torch.ones(5, 2, device="cuda"),
                          out, status=st)
    assert st.tolist() == [1, 1, 1, 2, 0]
    assert bool(torch.isnan(out[:4]).all()) and bool(torch.isfinite(out[4]).all())


@pytest.mark.parametrize("R,V,dtype", [(700, 20000, BF), (3000, 3001, BF), (300, 65537, F32)])
def test_gradient_batches(lp, R, V, dtype):
    g = torch.Generator().manual_seed(R)
    rows, tokens = zipf(R, V, g, dtype), some_tokens(R, V, 2, g, gone=0.4)
    gradient_case(lp, rows, tokens, 1.0, True, V, V)


def test_gradient_against_differences(lp):
    """Differences of the forward call.  With f the weighted sum and step h, the central difference
    is off by h^2 / 6 of the third derivative, at most 6 (|g| + |gH| (12 + ln V)) here (T = 1), and by
    the two values' own errors over 2 h."""
    V, R, h = 50, 2, 0.03
    g = torch.Generator().manual_seed(6)
    rows = torch.randn(R, V, generator=g) * 2
    tokens = torch.tensor([[3, 7, 3], [0, -1, 49]], dtype=torch.int32)
    gl, gh = torch.randn(R, 3, generator=g), torch.randn(R, generator=g)

    def value(x):
        t = Told(lp, x, tokens.repeat(x.shape[0] // R, 1))
        lpv = t.logprobs.cpu().double() * (tokens.repeat(x.shape[0] // R, 1) >= 0)
        return (lpv.view(-1, R, 3) * gl.double()).sum(-1) \
            + t.entropy.cpu().double().view(-1, R) * gh.double()

    steps = torch.eye(V).repeat_interleave(R, 0).view(V, R, V) * h
    up, down = (value((rows + s * steps).view(V * R, V)) for s in (1, -1))
    told = Told(lp, rows, tokens)
    out = torch.zeros(R, V, device="cuda")
    lp.spec_logprobs_grad(rows.cuda(), tokens.cuda(), told.normalizer, gl.cuda(), out,
                          entropy=told.entropy, grad_entropy=gh.cuda())
    want = plain.forward(rows.double(), tokens, 1.0, 0)
    size = gl.abs().sum(1) + gh.abs() * (12 + math.log(V))
    slack = h * h / 6 * 6 * size + (gl.abs().sum(1) * want["logprobs"][1].amax(1)
                                    + gh.abs() * want["entropy"][1]) * 2 / h
    err = (out.cpu().double() - ((up - down) / (2 * h)).T).abs()
    assert bool((err <= slack[:, None] + 1e-6).all()), err.max()


# ---------------------------------------------------------------- runs

def test_a_round_and_what_is_told(lp):
    """Sampled verification, then what a server tells about its tokens, from the same buffers."""
    from speculative_decoding_verification_18_gb300 import inputs, specverify as sv
    inp = inputs.make_inputs(mode="sample", B=24, k=5, V=4099, dtype="f32", T=0.8, kind="zipf",
                             seed=11)
    d = lambda a: torch.from_numpy(a).cuda()
    logits = d(inp.logits)
    out, n = sv.verify_sample(logits, d(inp.q), d(inp.x), d(inp.ua), d(inp.ur), 0.8)
    B, k1, V = logits.shape
    f = lambda *s: torch.full(s, 7.0, device="cuda")
    got, ent, tl = f(B, k1), f(B, k1), f(B, k1, 5)
    tt = torch.full((B, k1, 5), 7, dtype=torch.int32, device="cuda")
    lp.spec_logprobs(logits, out, got, lp.logprobs_workspace(logits, 1, 5), T=0.8, entropy=ent,
                     top_tokens=tt, top_logprobs=tl)
    live = torch.arange(k1) <= n.cpu()[:, None]
    assert torch.equal(live, out.cpu() >= 0) and not bool(live.all())
    want = plain.forward(logits.cpu().double().view(-1, V), out.cpu().view(-1, 1), 0.8, 5)
    for name, x in (("logprobs", got), ("entropy", ent), ("top_tokens", tt), ("top_logprobs", tl)):
        v, b = want[name]
        x, at = x.cpu().reshape(v.shape), live.view(-1)
        assert bool((x[~at] == 7).all())
        assert torch.equal(x[at], v[at]) if b is None else \
            bool(((x[at].double() - v[at]).abs() <= b[at]).all()), name
    # the alternatives' log probabilities are those of asking about them
    again = f(B, k1, 5)
    lp.spec_logprobs(logits, torch.where(live.cuda()[:, :, None], tt, -1), again,
                     lp.logprobs_workspace(logits, 5), T=0.8)
    assert torch.equal(again, tl)


def test_a_draft_learns_from_alternatives(lp):
    """The target's alternatives as the draft's targets: forward on both, the loss's gradient to
    the draft's logits, against float64 autograd of the same loss."""
    g = torch.Generator().manual_seed(12)
    R, V, K = 33, 5003, 16
    target, draft = zipf(R, V, g, BF).cuda(), zipf(R, V, g, BF).cuda()
    f = lambda *s: torch.zeros(*s, device="cuda")
    ask = torch.randint(0, V, (R,), generator=g).to(torch.int32).cuda()
    tt, tl, got = torch.zeros(R, K, dtype=torch.int32, device="cuda"), f(R, K), f(R)
    lp.spec_logprobs(target, ask, got, lp.logprobs_workspace(target, 1, K), top_tokens=tt,
                     top_logprobs=tl)
    dl, norm, grad = f(R, K), f(R, 2), torch.zeros_like(draft)
    lp.spec_logprobs(draft, tt, dl, lp.logprobs_workspace(draft, K), normalizer=norm)
    lp.spec_logprobs_grad(draft, tt, norm, -tl.exp(), grad)
    x = draft.double().requires_grad_()
    loss = -(tl.double().exp() * torch.log_softmax(x, 1).gather(1, tt.long())).sum()
    loss.backward()
    y, b = plain.gradient(draft.cpu().double(), tt.cpu(), norm.cpu().double(), None,
                          -tl.exp().cpu().double(), None, 1.0, BF)
    # the formula's m and ln S are rounded to fp32 there: 2^-24 of each in the exponent
    b = b + y.abs() * 2.0 ** -20 + 1e-30
    assert bool(((grad.cpu().double() - x.grad.cpu()).abs() <= b).all())


def test_streams_captures_and_shared_workspaces(lp):
    """Two captured calls over one workspace, replayed in turn with other logits, and another
    stream; the same bits each time."""
    g = torch.Generator().manual_seed(13)
    shapes = [(3, 130000, BF, 20), (900, 3001, F32, 5)]
    cases, size = [], 0
    for R, V, dt, top in shapes:
        size = max(size, lp.spec_logprobs_workspace_size(R, V, 0 if dt == BF else 1, 1, top))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for R, V, dt, top in shapes:
        x, t = zipf(R, V, g, dt).cuda(), some_tokens(R, V, 1, g).cuda()
        f = lambda *s: torch.zeros(*s, device="cuda")
        o = dict(logprobs=f(R, 1), normalizer=f(R, 2), entropy=f(R), top_logprobs=f(R, top),
                 top_tokens=torch.zeros(R, top, dtype=torch.int32, device="cuda"))
        grad = torch.zeros_like(x)
        one = torch.ones(R, 1, device="cuda")

        def call():
            lp.spec_logprobs(x, t, o["logprobs"], ws, entropy=o["entropy"],
                             normalizer=o["normalizer"], top_tokens=o["top_tokens"],
                             top_logprobs=o["top_logprobs"])
            lp.spec_logprobs_grad(x, t, o["normalizer"], one, grad)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        cases.append((graph, x, t, o, grad, top, one))  # (all that the graph uses stays alive)
    for step in range(3):
        for graph, x, t, o, grad, top, _ in cases:
            if step < 2:
                x.copy_(zipf(*x.shape, g, x.dtype))
            before = {n: v.clone() for n, v in o.items()}, grad.clone()
            graph.replay()
            torch.cuda.synchronize()
            if step == 2:
                assert all(torch.equal(o[n], before[0][n]) for n in o)
                assert torch.equal(grad, before[1])
                continue
            told = object.__new__(Told)
            told.__dict__.update(o)
            told.check(x.cpu(), t.cpu(), 1.0, top)
            y, b = plain.gradient(x.cpu().double(), t.cpu(), o["normalizer"].cpu().double(), None,
                                  torch.ones(len(x), 1, dtype=torch.float64), None, 1.0, x.dtype)
            assert bool(((grad.cpu().double() - y).abs() <= b).all())
