"""Numbers of rows around what the device holds at once."""
import pytest
import torch

from test_logprobs_gpu import BF, F32, Told, built, lp, some_tokens, zipf  # noqa: F401
from test_logprobs_ties_gpu import microseconds

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype,V", [(BF, 65536), (BF, 70001), (F32, 65537)])
@pytest.mark.parametrize("per_sm", [2, 3, 4])
@pytest.mark.parametrize("more", [-1, 1])
@pytest.mark.parametrize("gone", [0.0, 0.5])
def test_a_few_rows_per_multiprocessor(lp, dtype, V, per_sm, more, gone):
    R = per_sm * sms() + more
    g = torch.Generator().manual_seed(R)
    some = zipf(7, V, g, dtype)
    rows = some[torch.arange(R) % 7]
    tokens = some_tokens(R, V, 2, g, gone=gone)
    # (at the same place of a 16-byte word: sums are taken in an order that depends on it)
    got = Told(lp, rows, tokens, 0.8, 20, pitch=(V + 63) // 64 * 64)
    live = (tokens >= 0).any(1)
    assert not gone or 0 < int(live.sum()) < R
    # equal rows are told alike, to the bit; the first live one of each kind in full
    first = [next(r for r in range(k, R, 7) if live[r]) for k in range(7)]
    at = torch.tensor(first)[torch.arange(R) % 7]
    for n in ("entropy", "normalizer", "top_tokens", "top_logprobs"):
        x = getattr(got, n).cpu()
        assert torch.equal(x[live], x[at][live]), n
        assert bool((x[~live] == 7).all()), n
    for n in ("logprobs", "entropy", "normalizer", "top_tokens", "top_logprobs"):
        setattr(got, n, getattr(got, n).cpu()[first])
    got.check(rows[first], tokens[first], 0.8, 20)


@pytest.mark.parametrize("V", [65536, 100000])
def test_fewer_rows_take_no_longer(lp, V):
    """Than as many as are resident at once, all of them with tokens.  (Not one by one: a call's
    CTAs come while those of the one before leave, and a few rows more than two or three per SM may
    meet four on some.)"""
    R = 4 * sms()
    x = zipf(8, V, torch.Generator().manual_seed(1), BF)[torch.arange(R) % 8].cuda()
    times = [microseconds(lp, x[:n], 20) for n in (2 * sms(), 2 * sms() + 1, 3 * sms(), R - 1, R)]
    assert max(times[:-1]) <= 1.15 * times[-1], times
