"""Alternatives among equal logits, in rows with few tokens allowed, and of crowds of large ones:
which they are, and that rows of them take about as long as others."""
import math

import pytest
import torch

from test_logprobs_gpu import BF, F32, built, lp, strided, zipf  # noqa: F401

pytestmark = pytest.mark.gpu


def alternatives(lp, x, top):
    """top_tokens, top_logprobs of device rows x."""
    R, V = x.shape
    out = torch.zeros(R, 1, device="cuda")
    tt = torch.zeros(R, top, dtype=torch.int32, device="cuda")
    tl = torch.zeros(R, top, device="cuda")
    st = torch.zeros(R, dtype=torch.int32, device="cuda")
    lp.spec_logprobs(x, torch.zeros(R, 1, dtype=torch.int32, device="cuda"), out,
                     lp.logprobs_workspace(x, 1, top), top_tokens=tt, top_logprobs=tl, status=st)
    assert int(st.max()) == 0
    return tt.cpu(), tl.cpu()


def check(lp, rows, top, pitch=None):
    V = rows.shape[1]
    tt, tl = alternatives(lp, strided(rows, pitch or V), top)
    order = rows.float().sort(dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(tt[:, :V].long(), order)
    assert bool((tl[:, :-1] >= tl[:, 1:]).all())
    best = torch.log_softmax(rows.double(), 1).gather(1, order)
    near = (tl[:, :V] - best).abs() <= 1e-4
    assert bool((near | (torch.isinf(best) & (tl[:, :V] == best))).all())


def kinds(V, g, dtype):
    v = torch.arange(V)
    few = torch.full((V,), -math.inf)
    spread, first, last = few.clone(), few.clone(), few.clone()
    spread[::max(1, V // 5)] = 1.0
    first[:40], last[-40:] = 1.0, torch.randn(40, generator=g)
    step = torch.where(v < V // 2, 1.0, 2.0)
    late = torch.full((V,), -3.0)                  # the largest one again behind its first batch
    late[v % 9000 < 30] = 4.0
    late[:200] = -5.0
    return {"constant": torch.full((V,), 0.5), "spread": spread, "first": first, "last": last,
            "four values": torch.randint(0, 4, (V,), generator=g).float(), "step": step,
            "late": late, "zeros": torch.where(v % 3 == 0, -0.0, 0.0),
            "some -inf": torch.where(torch.rand(V, generator=g) < 0.5, -math.inf, 1.0)}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,more", [(300, 0), (2500, 3), (40000, 5), (151937, 0), (330001, 2)])
@pytest.mark.parametrize("top", [1, 5, 24, 25, 64])
def test_equal_logits(lp, dtype, V, more, top):
    g = torch.Generator().manual_seed(V + top)
    rows = torch.stack(list(kinds(V, g, dtype).values())).to(dtype)
    check(lp, rows, top, V + more)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("crowd", [1, 63, 64, 255, 256, 257, 300, 700, 1023, 1024, 1025, 1100,
                                   4000])
@pytest.mark.parametrize("top", [20, 64])
def test_crowds(lp, dtype, crowd, top):
    """So many large logits in a few threads' vectors: as many as are put in order at once, as there
    is room for, and more."""
    V, vec = 40000, 8 if dtype == BF else 4
    v = torch.arange(V)
    at = (v[v // vec % 256 < 32])[:crowd]
    rows = torch.stack([-20.0 - v / V, torch.full((V,), -20.0), -20.0 - v % 7])
    g = torch.Generator().manual_seed(crowd)
    rows[0, at] = torch.randn(len(at), generator=g)
    rows[1, at] = 2.0
    rows[2, at] = at / V
    check(lp, rows.to(dtype), top)


def microseconds(lp, x, top):
    R = x.shape[0]
    out, ws = torch.zeros(R, 1, device="cuda"), lp.logprobs_workspace(x, 1, top)
    t = torch.zeros(R, 1, dtype=torch.int32, device="cuda")
    tt = torch.zeros(R, top, dtype=torch.int32, device="cuda")
    tl = torch.zeros(R, top, device="cuda")
    best = math.inf
    for _ in range(8):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(20):
            lp.spec_logprobs(x, t, out, ws, top_tokens=tt, top_logprobs=tl)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 50)
    return best


@pytest.mark.parametrize("R,V", [(1, 151936), (64, 32000), (1024, 128256)])
@pytest.mark.parametrize("top", [1, 20])
def test_equal_logits_cost_little_more(lp, R, V, top):
    """(Read through once more by every thread, such rows took eight to fifteen times as long.)"""
    g = torch.Generator().manual_seed(0)
    x = zipf(min(R, 8), V, g, BF)[torch.arange(R) % min(R, 8)].cuda()
    usual = microseconds(lp, x, top)
    x.fill_(1.25)
    assert microseconds(lp, x, top) <= 4 * usual
    x.fill_(-math.inf)
    x[:, ::V // 5] = 1.0
    assert microseconds(lp, x, top) <= 4 * usual
