"""Attention with many query rows per key head on the GPU, over tables that keep the calls with
the form that multiplies in tensor memory: more than 64 rows per key head and room for more slots
than the calls of few items take."""
import pytest
import torch

import kv_plain
import test_kv_gpu
from kv_plain import E4M3
from test_kv_gpu import BF, HF, Round, built, kv  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def part(r, rows):
    """The sequences `rows` of a round, for the plain form."""
    return (r.q[rows], r.k, r.v, r.table[rows], r.lens[rows], r.counts[rows],
            None if r.parents is None else r.parents[rows], r.scale, r.k_scale, r.v_scale)


@pytest.mark.parametrize("dtype,cache,dim", [(BF, E4M3, 64), (HF, E4M3, 16), (HF, HF, 64),
                                             (BF, BF, 128), (BF, E4M3, 128)])
@pytest.mark.parametrize("heads,bad", [(8, "pairs"), (16, "one"), (8, "all"), (5, "pairs")])
def test_bad_pages_of_neighbours(kv, dtype, cache, dim, heads, bad):
    """Many sequences of one tile each, so that the loads run as many pieces ahead as they can, and
    bad pages eight pieces apart and closer: each bad sequence is all NaN and says so, the others
    have the bits that they have without them."""
    N, group = 9, 8
    B = 3200 // heads  # 21 pieces per CTA
    g = torch.Generator().manual_seed(heads)
    lens = torch.randint(0, 100, (B,), generator=g).tolist()
    r = Round(lens, N, "tree", heads=heads, group=group, dim=dim, dtype=dtype, cache=cache,
              page=16, seed=heads + dim, far=True)
    clean, status = r.attend(kv)
    assert status == [0] * B
    some = torch.arange(0, B, B // 6)
    kv_plain.check_attention(clean[some], *part(r, some))
    hit = {"pairs": [b for b in range(B) if b % 6 in (1, 2)], "one": list(range(3, B, 8)),
           "all": list(range(B))}[bad]
    for b in hit:
        r.table[b, 0 if b % 2 else (lens[b] + N - 1) // 16] = -1 if b % 3 else r.k.shape[0]
    out, status = r.attend(kv)
    is_bad = torch.zeros(B, dtype=torch.bool)
    is_bad[hit] = True
    assert [s != 0 for s in status] == is_bad.tolist()
    assert set(status) <= {0, kv.SV_DEV_BAD_PAGE}
    assert bool(torch.isnan(out[is_bad].float()).all())
    # by their bits: among so many float8 entries a few are too large for the type, and NaN
    assert torch.equal(out[~is_bad].view(torch.int16), clean[~is_bad].view(torch.int16))


@pytest.mark.parametrize("N,group,far", [(6, 2, False), (6, 2, True), (6, 5, True), (16, 6, True),
                                         (33, 8, True)])
def test_bad_lengths_leave_rows_behind_the_counts(kv, N, group, far):
    """A bad length makes NaN of the tokens that the sequence has; only a bad count makes NaN of
    all N.  The bit is set for a sequence without tokens too."""
    counts = [N, 3, 0, N - 1, 1, 0, 2, -1, N + 1, 3]
    r = Round([40, 50, 60, 70, 80, 33, 20, 90, 5, 60], N, "tree", counts=[max(0, min(N, n))
                                                                          for n in counts],
              heads=2, group=group, dim=64, seed=9, extra=0, far=far)
    clean = r.lens.clone()
    width = r.table.shape[1] * r.page
    r.counts = torch.tensor(counts, dtype=torch.int32)
    r.lens[1], r.lens[2] = -1, -2           # three tokens, none
    r.lens[3], r.lens[5] = width - N + 2, width + 1
    r.lens[4] = width                       # one token, the first behind the table
    out, status = r.attend(kv)
    L = kv.SV_DEV_BAD_LENGTH
    assert status == [0, L, L, L, L, L, 0, L, L, 0]
    for b, n in ((1, 3), (2, 0), (3, N - 1), (4, 1), (5, 0), (7, N), (8, N)):
        assert bool(torch.isnan(out[b, :n].float()).all()), b
        assert bool((out[b, n:] == 7.0).all()), b
    r.lens = clean
    good = torch.tensor([0, 6, 9])
    kv_plain.check_attention(out[good], *part(r, good), torch.full_like(out[good], 7.0))


FORMS = [(1, 4, False), (1, 4, True), (3, 8, True), (9, 8, False), (16, 8, True), (33, 7, True)]


@pytest.mark.parametrize("N,group,far", FORMS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale", [0.125, -0.125])
def test_negative_scales_of_entries(kv, N, group, far, dtype, scale):
    """An entry stands for its stored value times the head's scale, whatever the sign."""
    r = Round([300, 5, 40], N, "tree", heads=3, group=group, dim=64, dtype=dtype, cache=E4M3,
              seed=N, far=far, spread=3.0)
    r.k_scale[0] *= -1
    r.v_scale[1] *= -1
    r.k_scale[2] *= -1
    r.v_scale[2] *= -1
    r.scale = scale
    out, status = r.attend(kv)
    assert status == [0] * 3
    r.check(out)


@pytest.mark.parametrize("N,group,far", FORMS)
def test_a_scale_that_is_not_a_number_shows(kv, N, group, far):
    r = Round([300, 5], N, "tree", heads=2, group=group, dim=64, cache=E4M3, seed=N, far=far)
    r.k_scale[1] = float("nan")
    out, _ = r.attend(kv)
    assert bool(torch.isnan(out[:, :, group:].float()).all())
    one = torch.arange(group)
    kv_plain.check_attention(out[:, :, one], r.q[:, :, one], r.k[:, :, :1], r.v[:, :, :1], r.table,
                             r.lens, r.counts, r.parents, r.scale, r.k_scale[:1], r.v_scale[:1])


@pytest.mark.parametrize("N,group,far", FORMS)
@pytest.mark.parametrize("power", [126, 112, 90, -60, -100, -120])
def test_queries_of_any_size_over_float8(kv, N, group, far, power):
    """bfloat16 queries are scaled by a power of two per row on the way to halves, which can hold
    no others: rows of 2^126 and of 2^-100, with scales that bring the scores back to a few."""
    r = Round([300, 5], N, "tree", heads=2, group=group, dim=64, cache=E4M3, seed=N, far=far)
    r.q = (r.q.clamp(-1.9, 1.9).double() * 2.0 ** power).to(BF)
    r.k_scale *= 2.0 ** (-power // 2)
    r.scale *= 2.0 ** (-power - -power // 2)
    out, status = r.attend(kv)
    assert status == [0] * 2 and not bool(torch.isnan(out.float()).any())
    r.check(out)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4M3), (HF, E4M3)])
@pytest.mark.parametrize("dim,page", [(64, 4), (128, 1), (80, 2)])
@pytest.mark.parametrize("N,group", [(9, 8), (65, 3), (33, 16)])
def test_many_rows_over_the_smallest_pages(kv, dtype, cache, dim, page, N, group):
    """Pages of fewer slots than the swizzle's eight: the form for few rows takes them, in row
    tiles of 32, as it takes every call where the other one cannot be launched."""
    counts = [N, 0, N - 2, 1]
    r = Round([70, 3, 500, 0], N, "tree", counts=counts, heads=1, group=group, dim=dim,
              dtype=dtype, cache=cache, page=page, seed=N + dim, far=True)
    out, status = r.attend(kv)
    assert status == [0] * 4
    kv_plain.check_attention(out, *part(r, torch.arange(4)), torch.full_like(out, 7.0))


# dtype, cache, N, group: row tiles of 128 (one, and a part), and of 256 with a short last one
WIDE = [(BF, BF, 16, 8), (HF, HF, 9, 4), (BF, E4M3, 9, 8), (HF, E4M3, 16, 8), (BF, BF, 33, 8),
        (HF, HF, 65, 8), (BF, E4M3, 65, 8), (HF, E4M3, 20, 13)]


@pytest.mark.parametrize("dtype,cache,N,group", WIDE)
@pytest.mark.parametrize("scale", [0.0, -0.3, -0.125, 1e-30, 0.9])
def test_scales(kv, dtype, cache, N, group, scale):
    r = Round([300, 70, 0], N, "tree", heads=2, group=group, dim=64, dtype=dtype, cache=cache,
              seed=4, far=True)
    r.scale = scale
    out, status = r.attend(kv)
    assert status == [0] * 3
    r.check(out)


@pytest.mark.parametrize("dtype,cache,N,group", WIDE)
@pytest.mark.parametrize("dim", [16, 32, 48, 80, 96, 112])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_elements_and_orders(kv, dtype, cache, N, group, dim, order):
    r = Round([150, 0, 127], N, "tree", counts=[N, N - 1, 9], heads=3, group=group, dim=dim,
              dtype=dtype, cache=cache, order=order, page=8, seed=dim, far=True)
    out, status = r.attend(kv)
    assert status == [0] * 3
    kv_plain.check_attention(out, *part(r, torch.arange(3)), torch.full_like(out, 7.0))


@pytest.mark.parametrize("dtype,cache,N,group", WIDE)
@pytest.mark.parametrize("page", [8, 64, 128, 256, 2048])
def test_pages_and_borders(kv, dtype, cache, N, group, page):
    """Lengths that end on, before and behind borders of pages, of tiles of 128 slots and of words
    of the masks, and new tokens that begin there."""
    lens = [0, 1, 63, 64, 95, 127 - N, 127, 128, 129, 255 - N, 255, 256, 257]
    r = Round(lens, N, "tree", heads=1, group=group, dim=64, dtype=dtype, cache=cache, page=page,
              seed=page, far=True)
    out, status = r.attend(kv)
    assert status == [0] * len(lens)
    r.check(out)


@pytest.mark.parametrize("dtype,cache,N,group", WIDE)
def test_repeats_bit_for_bit(kv, dtype, cache, N, group):
    r = Round([3000, 10, 777, 129], N, "tree", heads=2, group=group, dim=128, dtype=dtype,
              cache=cache, seed=11, far=True)
    first, _ = r.attend(kv)
    for _ in range(3):
        assert torch.equal(r.attend(kv)[0], first)


@pytest.mark.parametrize("dtype,cache,N,group", WIDE)
def test_rows_that_overflow_are_nan_and_stay_alone(kv, dtype, cache, N, group):
    r = Round([300, 30], N, "tree", heads=1, group=group, dim=64, dtype=dtype, cache=cache, seed=2,
              far=True)
    hit = [(0, 1, 0, float("inf")), (0, N - 1, group - 1, float("-inf")), (1, 3, 2, float("nan"))]
    for b, j, h, x in hit:
        r.q[b, j, h] = x
    out, _ = r.attend(kv)
    for b, j, h, _ in hit:
        assert bool(torch.isnan(out[b, j, h].float()).all())
        r.q[b, j, h] = 0
    want, bound, _ = kv_plain.attention(*part(r, torch.arange(2)))
    err = (out.double() - want).abs()
    for b, j, h, _ in hit:
        err[b, j, h] = 0
    assert bool((err <= bound).all())


@pytest.mark.parametrize("N,group", [(16, 8), (33, 8)])
def test_lowest_and_large_scores(kv, N, group):
    """As for few rows: scores of +-60000 that differ by thousands."""
    r = Round([200, 64, 300], N, "tree", heads=1, group=group, dim=16, spread=1.0, seed=8, far=True)
    for b in range(3):
        for i, (p, s) in enumerate(kv_plain.slots(r.table[b], r.page, int(r.lens[b]))):
            if i % 3 == 0:
                r.k[p, s] = 3000.0 * r.k[p, s]
    r.q[0] = 40.0 * r.q[0]
    out, status = r.attend(kv)
    assert status == [0] * 3 and bool(torch.isfinite(out.float()).all())
    want, bound, _ = kv_plain.attention(*part(r, torch.arange(3)))
    err, tell = (out.double() - want).abs(), bound < 0.5
    assert float(tell.double().mean()) > 0.2 and bool((err <= bound)[tell].all())


@pytest.mark.parametrize("dtype,cache,N,group", WIDE)
def test_bad_trees(kv, dtype, cache, N, group):
    lens = [40, 300, 60, 70]
    counts = [N, N, N, 3]
    r = Round(lens, N, "tree", counts=counts, heads=2, group=group, dim=64, dtype=dtype,
              cache=cache, seed=9, far=True)
    r.parents[0, 2], r.parents[1, N - 1], r.parents[3, 4] = 2, -1, 77  # the last one is not read
    out, status = r.attend(kv)
    assert status == [0x40, 0x40, 0, 0]
    assert bool(torch.isnan(out[:2].float()).all())
    r.parents[3, 4] = 0
    good = torch.tensor([2, 3])
    kv_plain.check_attention(out[good], *part(r, good), torch.full_like(out[good], 7.0))


@pytest.mark.parametrize("dtype,cache,N,group", WIDE)
def test_strided_queries_and_far_pages(kv, dtype, cache, N, group):
    """Queries are a slice of a wider projection, and pages lie more than 2^32 bytes into the cache
    (by way of the tensor map here)."""
    page, heads, dim = 64, 2, 128
    r = Round([200, 64], N, "tree", heads=heads, group=group, dim=dim, dtype=dtype, cache=cache,
              page=page, seed=4, extra=0, far=True)
    each = page * heads * dim * (1 if cache == E4M3 else 2)
    pages = (5 << 30) // each
    k, v = (torch.empty(pages * each, dtype=torch.uint8, device="cuda").view(cache)
            .view(pages, page, heads, dim) for _ in range(2))
    raw = lambda x: x.view(torch.uint8)
    table = r.table.clone()
    held = (200 + N + page - 1) // page
    for b in range(2):
        for i in range(held):
            table[b, i] = pages - 1 - (b * held + i)
            raw(k)[int(table[b, i])] = raw(r.k)[int(r.table[b, i])].cuda()
            raw(v)[int(table[b, i])] = raw(r.v)[int(r.table[b, i])].cuda()
    d = lambda x: None if x is None else x.cuda()
    c = kv.PagedCache(k, v, table.cuda(), d(r.k_scale), d(r.v_scale))
    hq = heads * group
    wide = torch.zeros(2, N, hq + 2 * heads, dim, dtype=dtype, device="cuda")
    wide[:, :, heads:heads + hq] = r.q.cuda()
    out = torch.full_like(r.q, 7.0, device="cuda")
    kv.spec_kv_attention(c, wide[:, :, heads:heads + hq], r.lens.cuda(), out,
                         kv.attention_workspace(c, 2, N, hq), r.scale, parents=r.parents.cuda())
    r.check(out.cpu())


@pytest.mark.parametrize("capture", [False, True])
def test_whole_rounds_over_roomy_tables(kv, capture, monkeypatch):
    """The rounds of append, attention, tree verify and commit with 36 rows per key head, over a
    table with room for 9700 slots, which takes them off the form of few items."""
    made = kv.PagedCache

    def roomy(k, v, table):
        more = torch.full((table.shape[0], 600), -1, dtype=torch.int32, device=table.device)
        return made(k, v, torch.cat([table, more], dim=1))

    monkeypatch.setattr(kv, "PagedCache", roomy)
    test_kv_gpu.test_whole_rounds(kv, capture)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, E4M3)])
@pytest.mark.parametrize("N,heads,group", [(65, 1, 128), (2, 1, 1024), (1, 1024, 1), (3, 128, 8),
                                           (17, 2, 8), (32, 1, 4)])
@pytest.mark.parametrize("far", [False, True])
def test_many_query_heads(kv, dtype, cache, N, heads, group, far):
    """From one key head for 1024 query heads to as many of both: 33 row tiles of 256, tiles with
    their second half nearly empty, and 1024 items per sequence."""
    r = Round([130, 5], N, "tree", counts=[N, max(1, N - 1)], heads=heads, group=group, dim=16,
              dtype=dtype, cache=cache, seed=N, far=far)
    out, status = r.attend(kv)
    assert status == [0] * 2
    kv_plain.check_attention(out, *part(r, torch.arange(2)), torch.full_like(out, 7.0))
