"""Windows where one form of the attention takes over from another: 33 to 64 rows per key head over
float8 around the most slots that stay with mma.sync, and few sequences around the most that a
cluster per item takes."""
import pytest

from test_window_gpu import BF, E4M3, HF, Windowed, built, good, kv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("slots", [1535, 1536, 1537, 2048, 2049])
@pytest.mark.parametrize("N,sinks", [(5, 4), (8, 70)])
def test_float8_rows_by_slots_and_wide(kv, dtype, dim, slots, N, sinks):
    good(Windowed([2500, 900], N, slots - sinks - N - 128, sinks, "tree", heads=10, group=8,
                  dim=dim, dtype=dtype, cache=E4M3, page=32, seed=slots + N), kv)


@pytest.mark.parametrize("cache", [BF, E4M3])
@pytest.mark.parametrize("slots", [8191, 8192, 8193])
@pytest.mark.parametrize("N,group,sinks", [(1, 4, 4), (4, 8, 0)])
def test_clusters_and_ranges(kv, cache, slots, N, group, sinks):
    good(Windowed([9000, 8100], N, slots - sinks - N - 128, sinks, "chain", heads=2, group=group,
                  dim=64, dtype=BF, cache=cache, page=64, seed=slots + N), kv)
