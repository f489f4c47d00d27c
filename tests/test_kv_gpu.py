"""The paged cache calls on the GPU against the plain float64 implementation (kv_plain.py).

Cases are small and go where the calls can go wrong: lengths around page and tile borders, empty
caches, ragged numbers of new tokens, trees, every type and layout, values that are not finite in
places that must not be read, bad lengths, trees and pages, other streams, captured graphs, and
whole rounds through the tree verifier."""
import math

import pytest
import torch

import kv_plain
from kv_plain import E4M3
from parity import Guarded

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verification_18_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(scope="module")
def kv():
    from speculative_decoding_verification_18_gb300 import kvcache
    return kvcache


def tree(N, form, g):
    """Parents of N nodes: a chain, a random tree, a star (all children of the root), or None."""
    if form == "chain":
        return None
    if form == "star":
        return torch.zeros(N, dtype=torch.int32)
    return torch.tensor([0] + [int(torch.randint(0, j, (1,), generator=g)) for j in range(1, N)],
                        dtype=torch.int32)


class Round:
    """One layer's cache and new tokens on the CPU; paged() makes the device's copies.  Slots that
    no sequence holds are NaN (or, in a float8 cache, its NaN), tables of shared pools shuffled.
    far: the table has room for more than 8192 slots, which calls of few sequences take another
    way than tables for short contexts."""

    def __init__(self, lens, N, form="chain", counts=None, heads=2, group=4, dim=64, page=16,
                 dtype=BF, cache=None, order="slot", seed=0, spread=1.5, extra=1, far=False):
        g = torch.Generator().manual_seed(seed)
        self.g, self.N, self.heads, self.group, self.dim, self.page = g, N, heads, group, dim, page
        self.dtype, self.cache = dtype, cache or dtype
        B = len(lens)
        self.B = B
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.counts = torch.tensor(counts if counts is not None else [N] * B, dtype=torch.int32)
        self.ragged = counts is not None
        self.parents = None if form == "chain" else torch.stack([tree(N, form, g)
                                                                 for _ in range(B)])
        width = max(1, max((l + N + page - 1) // page for l in lens)) + extra
        pages = B * width + 1
        self.table = torch.randperm(pages, generator=g)[:B * width].view(B, width).to(torch.int32)
        if far:  # a table for long contexts, whose entries past the held pages mean nothing
            self.table = torch.cat([self.table, torch.full((B, 8192 // page + 1), -1,
                                                           dtype=torch.int32)], dim=1)
        shape = (pages, page, heads, dim)
        lay = (lambda x: x) if order == "slot" else (
            lambda x: x.transpose(1, 2).contiguous().transpose(1, 2))
        self.k_scale = self.v_scale = None
        if self.cache == E4M3:
            self.k_scale = torch.rand(heads, generator=g) * 0.02 + 0.01
            self.v_scale = torch.rand(heads, generator=g) * 0.02 + 0.01
        self.k, self.v = (torch.full(shape, math.nan).to(self.cache) for _ in range(2))
        for pool, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            for b in range(B):
                for p, s in kv_plain.slots(self.table[b], page, int(self.lens[b])
                                           + int(self.counts[b])):
                    x = torch.randn(heads, dim, generator=g)
                    pool[p, s] = (x if scale is None else x / scale[:, None]).to(self.cache)
        self.k, self.v = lay(self.k), lay(self.v)
        self.q = (torch.randn(B, N, heads * group, dim, generator=g) * spread).to(dtype)
        self.scale = dim ** -0.5

    def paged(self, kv):
        d = lambda x: None if x is None else x.cuda()
        self.kd, self.vd = self.k.cuda(), self.v.cuda()
        if self.k.stride() != self.kd.stride():
            self.kd, self.vd = (torch.empty_strided(self.k.shape, self.k.stride(),
                                                    dtype=self.k.dtype, device="cuda").copy_(x)
                                for x in (self.k, self.v))
        return kv.PagedCache(self.kd, self.vd, d(self.table), d(self.k_scale), d(self.v_scale))

    def attend(self, kv, stream=None, ws=None):
        d = lambda x: None if x is None else x.cuda()
        c, gd = self.paged(kv), Guarded()
        out = gd.empty(self.q.shape, self.dtype, fill=7.0)
        n = kv.spec_kv_attention_workspace_size(self.B, self.N, self.heads * self.group, self.heads,
                                                self.dim)
        ws = gd.empty((n,), torch.uint8, fill=255)  # NaN wherever it is read unwritten
        status = gd.empty((self.B,), torch.int32, fill=0)
        kv.spec_kv_attention(c, d(self.q), d(self.lens), out, ws, self.scale,
                             parents=d(self.parents),
                             num_new=d(self.counts) if self.ragged else None, status=status)
        gd.check()
        return out.cpu(), status.cpu().tolist()

    def check(self, out, v=None, k=None):
        kv_plain.check_attention(out, self.q, self.k if k is None else k,
                                 self.v if v is None else v, self.table, self.lens, self.counts,
                                 self.parents, self.scale, self.k_scale, self.v_scale,
                                 torch.full_like(out, 7.0))


TYPES = [(BF, BF), (HF, HF), (BF, E4M3), (HF, E4M3)]


@pytest.mark.parametrize("far", [False, True])
# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_attention_types_and_heads(kv, far, dtype, cache, dim, order):
    r = Round([37, 0, 130, 64], 3, heads=3, group=2, dim=dim, dtype=dtype, cache=cache,
              order=order, seed=dim, far=far)
    out, status = r.attend(kv)
    assert status == [0] * 4
    r.check(out)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("N,form", [(1, "chain"), (2, "chain"), (17, "chain"), (65, "chain"),
                                    (5, "tree"), (16, "tree"), (40, "tree"), (65, "tree"),
                                    (65, "star"), (33, "star")])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 8), (1, 5)])
def test_attention_chains_and_trees(kv, far, N, form, heads, group):
    r = Round([100, 7, 0], N, form, heads=heads, group=group, dim=64, seed=N, far=far)
    out, status = r.attend(kv)
    assert status == [0] * 3
    r.check(out)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("page", [1, 2, 16, 64, 256])
@pytest.mark.parametrize("N", [1, 6])
def test_attention_lengths_around_borders(kv, far, page, N):
    lens = [0, 1, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257]
    r = Round(lens, N, heads=1, group=3, dim=64, page=page, seed=page, far=far)
    out, status = r.attend(kv)
    assert status == [0] * len(lens)
    r.check(out)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("N,group,form", [(1, 4, "chain"), (4, 8, "tree"), (16, 8, "tree"),
                                          (33, 7, "tree")])
def test_attention_split_over_a_long_cache(kv, far, dtype, cache, N, group, form):
    """One sequence, long enough for every SM to hold a part of it, and a short one beside it."""
    r = Round([5003, 40], N, form, heads=1, group=group, dim=128, dtype=dtype, cache=cache,
              page=32, seed=N, far=far)
    out, status = r.attend(kv)
    assert status == [0, 0]
    r.check(out)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("N,group,form", [(6, 4, "chain"), (16, 8, "tree"), (20, 8, "tree")])
def test_attention_ragged_counts(kv, far, N, group, form):
    counts = [N, 0, 1, N // 2, N - 1, 0, 2]
    r = Round([50, 60, 0, 129, 300, 0, 16], N, form, counts=counts, heads=2, group=group,
              dim=64, seed=3, far=far)
    out, status = r.attend(kv)
    assert status == [0] * 7
    r.check(out)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("B", [1, 150, 700])
@pytest.mark.parametrize("N,group", [(1, 2), (12, 8)])
def test_attention_many_sequences(kv, far, B, N, group):
    """Every third sequence has nothing new, every fourth nothing cached."""
    g = torch.Generator().manual_seed(B)
    lens = [0 if b % 4 == 3 else int(torch.randint(0, 40, (1,), generator=g)) for b in range(B)]
    counts = [0 if b % 3 == 2 else 1 + b % N for b in range(B)]
    r = Round(lens, N, "tree", counts=counts, heads=1, group=group, dim=16, page=8, seed=B, far=far)
    out, status = r.attend(kv)
    assert status == [0] * B
    r.check(out)


@pytest.mark.parametrize("far", [False, True])
def test_attention_without_work(kv, far):
    r = Round([5, 9], 4, counts=[0, 0], far=far)
    out, status = r.attend(kv)
    assert status == [0, 0] and bool((out == 7.0).all())


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("N,group,form", [(7, 4, "star"), (16, 8, "tree"), (40, 8, "tree")])
def test_attention_masked_places_may_hold_anything(kv, far, dtype, cache, N, group, form):
    """A leaf whose key and value are NaN or infinite changes its own row only."""
    r = Round([70, 33, 0, 128], N, form, heads=2, group=group, dim=64, dtype=dtype, cache=cache,
              seed=5, far=far)
    clean_k, clean_v = r.k.clone(), r.v.clone()
    for b, bad in enumerate((math.nan, math.inf, -math.inf, math.nan)):
        p, s = kv_plain.slots(r.table[b], r.page, int(r.lens[b]) + N)[-1]  # node N - 1: a leaf
        for pool in (r.k, r.v):
            pool[p, s] = torch.full_like(pool[p, s].float(), bad if cache != E4M3 else math.nan
                                         ).to(pool.dtype)
    out, status = r.attend(kv)
    assert status == [0] * 4
    assert bool(torch.isnan(out[:, N - 1].float()).any(dim=-1).all())
    # the leaf's row apart, the results are those of the clean cache
    r.k, r.v = clean_k, clean_v
    want, bound, _ = kv_plain.attention(r.q, r.k, r.v, r.table, r.lens, r.counts, r.parents,
                                        r.scale, r.k_scale, r.v_scale)
    err = (out.double() - want).abs()[:, :N - 1]
    assert bool((err <= bound[:, :N - 1]).all())


@pytest.mark.parametrize("far", [False, True])
def test_attention_lowest_and_large_scores(kv, far):
    """Keys so large that scores reach +-60000 and differ by thousands; one key whose scores are
    the type's lowest: weights are one-hot or exactly shared, never NaN."""
    r = Round([200, 64, 3], 3, heads=1, group=2, dim=16, spread=1.0, seed=8, far=far)
    for b in range(3):
        for i, (p, s) in enumerate(kv_plain.slots(r.table[b], r.page, int(r.lens[b]))):
            if i % 3 == 0:
                r.k[p, s] = 3000.0 * r.k[p, s]
    r.q[0] = 40.0 * r.q[0]
    out, status = r.attend(kv)
    assert bool(torch.isfinite(out.float()).all())
    want, bound, _ = kv_plain.attention(r.q, r.k, r.v, r.table, r.lens, r.counts, r.parents,
                                        r.scale)
    # a score off by e moves a weight by a factor exp(e): with e large the bound is the spread of
    # the values themselves, and only rows whose bound says something are compared
    err = (out.double() - want).abs()
    tell = bound < 0.5
    assert float(tell.double().mean()) > 0.2 and bool((err <= bound)[tell].all())


@pytest.mark.parametrize("far", [False, True])
def test_attention_rows_that_overflow_are_nan_and_stay_alone(kv, far):
    """A query of infinities gives NaN in its own row; the others keep their values."""
    r = Round([90, 30], 4, heads=1, group=2, dim=64, seed=2, far=far)
    r.q[0, 1, 0] = math.inf
    out, _ = r.attend(kv)
    assert bool(torch.isnan(out[0, 1, 0].float()).all())
    r.q[0, 1, 0] = 0
    want, bound, _ = kv_plain.attention(r.q, r.k, r.v, r.table, r.lens, r.counts, r.parents,
                                        r.scale)
    err = (out.double() - want).abs()
    err[0, 1, 0] = 0
    assert bool((err <= bound).all())


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
def test_attention_scales(kv, far, scale):
    r = Round([40, 70], 4, "tree", seed=4, far=far)
    r.scale = scale
    out, _ = r.attend(kv)
    r.check(out)


def test_attention_shared_prefix_and_strided_queries(kv):
    """Two sequences read the same committed pages; queries are a slice of a wider projection."""
    r = Round([64, 64], 3, heads=2, group=2, dim=64, seed=6)
    r.table[1, :4] = r.table[0, :4]
    c = r.paged(kv)
    wide = torch.zeros(2, 3, 4 + 2 * 2, 64, dtype=BF, device="cuda")
    wide[:, :, :4] = r.q.cuda()
    out = torch.full_like(r.q, 7.0, device="cuda")
    ws = kv.attention_workspace(c, 2, 3, 4)
    kv.spec_kv_attention(c, wide[:, :, :4], r.lens.cuda(), out, ws, r.scale)
    r.check(out.cpu())


@pytest.mark.parametrize("far", [False, True])
def test_attention_bad_data(kv, far):
    """Bad lengths, counts, trees and pages: NaN rows and the bit, the others untouched by it."""
    N = 6
    r = Round([40, 50, 60, 70, 80, 33, 20, 90], N, "tree", counts=[6, 6, 6, 6, 6, 6, 3, 6],
              heads=2, group=3, dim=64, seed=9, extra=0, far=far)
    clean = (r.lens.clone(), r.counts.clone(), r.parents.clone(), r.table.clone())
    width = r.table.shape[1] * r.page
    r.lens[0] = -1
    r.lens[1] = width - 5
    r.counts[2] = 7
    r.counts[3] = -1
    r.parents[4, 2] = 2
    r.parents[5, 3] = -1
    r.parents[6, 4] = 77          # behind its three tokens: not read
    r.table[7, 2] = r.k.shape[0]  # a page behind the last one
    out, status = r.attend(kv)
    L, T, G = kv.SV_DEV_BAD_LENGTH, 0x40, kv.SV_DEV_BAD_PAGE
    assert status == [L, L, L, L, T, T, 0, G]
    assert bool(torch.isnan(out[[0, 1, 2, 3, 4, 5, 7]].float()).all())
    r.lens, r.counts, r.parents, r.table = clean
    want, bound, _ = kv_plain.attention(r.q, r.k, r.v, r.table, r.lens, r.counts, r.parents,
                                        r.scale)
    assert bool(((out[6, :3].double() - want[6, :3]).abs() <= bound[6, :3]).all())
    assert bool((out[6, 3:] == 7.0).all())


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("N,group", [(1, 4), (16, 8), (24, 8)])
def test_attention_bad_page_far_from_the_end(kv, far, N, group):
    """The bad page is in one part of a split sequence; every row of it is NaN."""
    r = Round([4000, 100], N, "tree", heads=1, group=group, dim=64, seed=1, far=far)
    good = r.table.clone()
    r.table[0, 3] = -1
    out, status = r.attend(kv)
    assert status == [kv.SV_DEV_BAD_PAGE, 0]
    assert bool(torch.isnan(out[0].float()).all())
    r.table = good
    want, bound, _ = kv_plain.attention(r.q[1:], r.k, r.v, r.table[1:], r.lens[1:], r.counts[1:],
                                        r.parents[1:], r.scale)
    assert bool(((out[1:].double() - want).abs() <= bound).all())


def test_attention_offsets_past_32_bits(kv):
    """Pages more than 2^32 bytes into the cache."""
    page, heads, dim, N = 64, 4, 128, 4
    pages = (5 << 30) // (page * heads * dim * 2)
    k = torch.empty(pages, page, heads, dim, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    r = Round([100, 64], N, heads=heads, group=2, dim=dim, page=page, seed=4, extra=0)
    far = pages - 1 - torch.arange(r.table.numel(), dtype=torch.int32).view_as(r.table)
    for b in range(2):
        for i in range(r.table.shape[1]):
            k[int(far[b, i])] = r.k[int(r.table[b, i])].cuda()
            v[int(far[b, i])] = r.v[int(r.table[b, i])].cuda()
    c = kv.PagedCache(k, v, far.cuda())
    out = torch.full_like(r.q, 7.0, device="cuda")
    kv.spec_kv_attention(c, r.q.cuda(), r.lens.cuda(), out, kv.attention_workspace(c, 2, N, 8),
                         r.scale)
    r.check(out.cpu())


@pytest.mark.parametrize("far", [False, True])
def test_attention_repeats_bit_for_bit(kv, far):
    """The split does not depend on timing: the same call gives the same bits."""
    r = Round([3000, 10, 777], 5, "tree", heads=2, group=4, dim=128, seed=11, far=far)
    first, _ = r.attend(kv)
    for _ in range(3):
        assert torch.equal(r.attend(kv)[0], first)


# ---------------------------------------------------------------- append

def append_case(kv, r, rot, interleaved, base=10000.0, factor=1.0, original=0, magnitude=1.0,
                with_q=True, in_place=False, wide=False):
    """Runs the call on r's tokens and checks queries, entries and everything else's bits."""
    g = torch.Generator().manual_seed(99)
    B, N, H, D = r.B, r.N, r.heads, r.dim
    hq = H * r.group
    kn = torch.randn(B, N, H, D, generator=g).to(r.dtype)
    vn = torch.randn(B, N, H, D, generator=g).to(r.dtype)
    d = lambda x: None if x is None else x.cuda()
    c, gd = r.paged(kv), Guarded()
    rope = kv.Rope(rot, base, interleaved, factor, original, magnitude=magnitude) if rot else None
    q_in, k_in, v_in = d(r.q), d(kn), d(vn)
    if wide:
        qkv = torch.cat([q_in, k_in, v_in], dim=2)
        q_in, k_in, v_in = qkv.split([hq, H, H], dim=2)
    out = gd.empty((B, N, hq, D), r.dtype, fill=7.0)
    if in_place:
        out.copy_(q_in)
        q_in = out
    status = gd.empty((B,), torch.int32, fill=0)
    kv.spec_kv_append(c, k_in, v_in, d(r.lens), q=q_in if with_q else None,
                      q_out=out if with_q else None, rope=rope, parents=d(r.parents),
                      num_new=d(r.counts) if r.ragged else None, status=status)
    gd.check()
    rate = kv_plain.rates(rot, base, factor, original) if rot else torch.zeros(0,
                                                                              dtype=torch.float64)
    k_got, v_got, out = r.kd.cpu(), r.vd.cpu(), out.cpu()
    k_want, v_want = r.k.clone(), r.v.clone()
    for b in range(B):
        up = kv_plain.paths(None if r.parents is None else r.parents[b], N)
        for j in range(int(r.counts[b])):
            pos = int(r.lens[b]) + len(up[j]) - 1
            s = int(r.lens[b]) + j
            p, s = int(r.table[b, s // r.page]), s % r.page
            if with_q:
                y, slack = kv_plain.rotate(r.q[b, j], pos, rate, interleaved, magnitude)
                err = (out[b, j].double() - y).abs()
                assert bool((err <= kv_plain.stored_bound(y, slack, r.dtype)).all()), (b, j)
            y, slack = kv_plain.rotate(kn[b, j], pos, rate, interleaved, magnitude)
            for got, y, slack, sc in ((k_got, y, slack, r.k_scale),
                                      (v_got, vn[b, j].double(), 0 * slack, r.v_scale)):
                x = got[p, s].double()
                one = 1.0
                if sc is not None:
                    one = sc.double()[:, None]
                    x, y = x * one, torch.clamp(y, -448 * one, 448 * one)
                    assert bool(((x - y).abs() <= kv_plain.stored_bound(y, slack, E4M3, one)).all())
                elif got is v_got:
                    assert torch.equal(x, y)
                else:
                    assert bool(((x - y).abs() <= kv_plain.stored_bound(y, slack, r.dtype)).all())
            k_want[p, s], v_want[p, s] = k_got[p, s], v_got[p, s]
        if with_q and not in_place:
            assert bool((out[b, int(r.counts[b]):] == 7.0).all())
    bits = torch.uint8 if r.cache == E4M3 else torch.int16
    assert torch.equal(k_got.view(bits), k_want.view(bits))  # nothing else was written
    assert torch.equal(v_got.view(bits), v_want.view(bits))
    return status.cpu().tolist()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 64), (80, 80), (80, 40), (96, 32), (96, 50),
                                     (16, 2), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_types_and_layouts(kv, dtype, cache, dim, rot, interleaved):
    r = Round([37, 0, 130], 5, "tree", heads=2, group=3, dim=dim, dtype=dtype, cache=cache,
              order="head" if interleaved else "slot", seed=dim + rot)
    assert append_case(kv, r, rot, interleaved) == [0] * 3


@pytest.mark.parametrize("N,form", [(1, "chain"), (65, "chain"), (65, "tree"), (65, "star"),
                                    (9, "tree")])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_append_chains_and_trees(kv, N, form, page):
    r = Round([37, 0, 63, 64], N, form, counts=[N, 1, N // 2, 0], heads=1, group=2, page=page,
              seed=N)
    assert append_case(kv, r, 64, False, wide=True) == [0] * 4


@pytest.mark.parametrize("kw", [dict(factor=8.0, base=500000.0, original=8192),
                                dict(factor=4.0), dict(magnitude=1.27),
                                dict(with_q=False), dict(in_place=True), dict(wide=True)])
def test_append_options(kv, kw):
    r = Round([4000, 11], 3, heads=2, group=2, seed=7)
    append_case(kv, r, 64, False, **kw)
    append_case(kv, r, 32, True, **kw)


def test_append_far_positions(kv):
    """Positions of a million and of nearly 2^30: the angle is exact modulo a turn, so the error
    is that of position 0 (the rates' own 2^-63 turns times the position stay below 2^-32)."""
    r = Round([3], 2, heads=1, group=1, dim=16, page=4, seed=3)
    pages, page = 2, 1 << 20
    r.k = torch.zeros(pages, page, 1, 16, dtype=BF)
    r.v = torch.zeros(pages, page, 1, 16, dtype=BF)
    r.page = page
    r.table = torch.zeros(1, 1024, dtype=torch.int32)
    for at in (1000003, (1 << 30) - 7):
        r.lens = torch.tensor([at], dtype=torch.int32)
        assert append_case(kv, r, 16, False) == [0]


def test_append_saturates_and_keeps_nan(kv):
    """Past the largest float8 value entries saturate; NaN stays NaN; zeros and signs are kept."""
    r = Round([2], 1, heads=1, group=1, dim=16, cache=E4M3, seed=1)
    c = r.paged(kv)
    x = torch.tensor([1e4, -1e4, math.inf, -math.inf, math.nan, 0.0, -0.0, 1.0] * 2, dtype=BF)
    x = x.view(1, 1, 1, 16).cuda()
    kv.spec_kv_append(c, x, x.clone(), r.lens.cuda())
    p, s = kv_plain.slots(r.table[0], r.page, 3)[-1]
    for pool, scale in ((r.kd, r.k_scale), (r.vd, r.v_scale)):
        got = pool[p, s, 0].cpu().float()[:8]
        assert got[:4].tolist() == [448.0, -448.0, 448.0, -448.0]
        assert math.isnan(got[4]) and got[5] == 0 and got[6] == 0
        assert math.copysign(1, got[6]) == -1
        assert abs(got[7] * scale[0] - 1) <= 2.0 ** -4


def test_append_bad_data(kv):
    N = 6
    r = Round([40, 50, 60, 70, 80, 33, 20, 90], N, "tree", counts=[6, 6, 6, 6, 6, 6, 3, 6],
              heads=2, group=3, dim=64, seed=9, extra=1)
    width = r.table.shape[1] * r.page
    r.lens[0] = -1
    r.lens[1] = width - 5
    r.counts[2] = 7
    r.counts[3] = -1
    r.parents[4, 2] = 2
    r.parents[5, 3] = -1
    r.parents[6, 4] = 77                # behind its three tokens: not read
    r.table[7, 90 // r.page + 1] = -5   # the page of slot 96 and on: no token needs it
    r.table[6, 20 // r.page] = 1 << 30
    d = lambda x: None if x is None else x.cuda()
    c = r.paged(kv)
    new = torch.randn(r.B, N, 2, 64, generator=r.g).to(BF).cuda()
    out = torch.full_like(r.q, 7.0, device="cuda")
    status = torch.zeros(r.B, dtype=torch.int32, device="cuda")
    kv.spec_kv_append(c, new, new, d(r.lens), q=d(r.q), q_out=out, parents=d(r.parents),
                      num_new=d(r.counts), status=status)
    L, T, G = kv.SV_DEV_BAD_LENGTH, 0x40, kv.SV_DEV_BAD_PAGE
    assert status.cpu().tolist() == [L, L, L, L, T, T, G, 0]
    assert bool((out[:6] == 7.0).all()) and torch.equal(out[6, :3].cpu(), r.q[6, :3])
    k_want = r.k.clone()
    for j in range(N):
        s = 90 + j
        k_want[int(r.table[7, s // r.page]), s % r.page] = new[7, j].cpu()
    assert torch.equal(r.kd.cpu().view(torch.int16), k_want.view(torch.int16))


# ---------------------------------------------------------------- commit

def commit_plain(pools, table, page, lens, nodes, acc):
    for b in range(len(lens)):
        for i in range(max(0, int(acc[b]))):
            src, dst = int(lens[b]) + int(nodes[b, i]), int(lens[b]) + i + 1
            for p in pools:
                p[..., int(table[b, dst // page]), dst % page, :, :] = \
                    p[..., int(table[b, src // page]), src % page, :, :]


@pytest.mark.parametrize("cache", [BF, HF, E4M3])
@pytest.mark.parametrize("layers,order", [(1, "slot"), (3, "head")])
@pytest.mark.parametrize("N,page,heads,dim", [(2, 16, 1, 16), (16, 16, 2, 80), (65, 8, 8, 128),
                                              (65, 64, 3, 64), (30, 1, 1, 64)])
def test_commit(kv, cache, layers, order, N, page, heads, dim):
    g = torch.Generator().manual_seed(N)
    B = 9
    lens = torch.randint(0, 100, (B,), generator=g).to(torch.int32)
    width = (100 + N + page) // page + 1
    pages = B * width
    table = torch.randperm(pages, generator=g).view(B, width).to(torch.int32)
    inner = (page, heads, dim) if order == "slot" else (heads, page, dim)
    bits = torch.uint8 if cache == E4M3 else torch.int16
    pools = [torch.randint(-100 if bits == torch.int16 else 0, 100, (layers, pages) + inner,
                           generator=g).to(bits) for _ in range(2)]
    look = (lambda x: x) if order == "slot" else (lambda x: x.transpose(2, 3))
    nodes = torch.full((B, N), -1, dtype=torch.int32)
    acc = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        pick = torch.randperm(N - 1, generator=g)[:int(torch.randint(0, N, (1,), generator=g))]
        pick = (pick.sort().values + 1) if b else torch.arange(1, N)  # b = 0: all, nothing moves
        acc[b] = len(pick)
        nodes[b, :len(pick)] = pick.to(torch.int32)
    acc[3], nodes[3, :] = -1, 5     # an invalid sequence: its nodes are not looked at
    gd = Guarded()
    dev = [gd.empty(p.shape, bits) for p in pools]
    for x, p in zip(dev, pools):
        x.copy_(p)
    c = kv.PagedCache(look(dev[0].view(cache)) if layers > 1 else look(dev[0].view(cache))[0],
                      look(dev[1].view(cache)) if layers > 1 else look(dev[1].view(cache))[0],
                      table.cuda(), *([torch.ones(*((layers, heads) if layers > 1 else (heads,)),
                                                  device="cuda")] * 2 if cache == E4M3 else []))
    out = gd.empty((B,), torch.int32, fill=-7)
    status = gd.empty((B,), torch.int32, fill=0)
    kv.spec_kv_commit(c, lens.cuda(), acc.cuda(), out, nodes.cuda(), status=status)
    gd.check()
    commit_plain([look(p) for p in pools], table, page, lens, nodes, acc)
    assert status.cpu().tolist() == [0] * B
    assert torch.equal(out.cpu(), lens + acc + 1)
    for x, p in zip(dev, pools):
        assert torch.equal(x.cpu(), p)


def test_commit_chain_and_bad_data(kv):
    """A chain moves nothing; bad counts, nodes, lengths and pages leave the sequence as it is."""
    B, N, page, width = 9, 6, 16, 4
    k = torch.randn(B * width, page, 2, 16).to(BF).cuda()
    v = torch.randn(B * width, page, 2, 16).to(BF).cuda()
    k0, v0 = k.clone(), v.clone()
    table = torch.arange(B * width, dtype=torch.int32).view(B, width)
    lens = torch.tensor([10, 11, 12, 13, 14, 58, -2, 10, 57], dtype=torch.int32)
    acc = torch.tensor([3, 0, -1, 5, 1, 4, 1, 2, 5], dtype=torch.int32)
    out = torch.empty(B, dtype=torch.int32, device="cuda")
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    c = kv.PagedCache(k, v, table.cuda())
    kv.spec_kv_commit(c, lens.cuda(), acc.cuda(), out, status=status)
    want = (lens + acc + 1).tolist()
    want[6] = -2
    assert out.cpu().tolist() == want
    assert status.cpu().tolist() == [0, 0, 0, 0, 0, 0, kv.SV_DEV_BAD_LENGTH, 0, 0]
    assert torch.equal(k, k0) and torch.equal(v, v0)
    nodes = torch.full((B, N), -1, dtype=torch.int32)
    acc = torch.tensor([6, -2, 2, 2, 1, 1, 1, 1, 2], dtype=torch.int32)
    nodes[2, :2] = torch.tensor([3, 3])     # the same node twice
    nodes[3, :2] = torch.tensor([4, 2])     # not increasing
    nodes[4, 0] = 6                         # no such node
    nodes[5, 0] = 0                         # the root
    nodes[6, 0] = 3                         # its length is bad
    nodes[7, 0] = 2                         # its page is bad
    nodes[8, :2] = torch.tensor([2, 7 - 0]) # beyond both N and the table
    table[7, 0] = -1
    status.zero_()
    c = kv.PagedCache(k, v, table.cuda())
    kv.spec_kv_commit(c, lens.cuda(), acc.cuda(), out, nodes.cuda(), status=status)
    L, T, G = kv.SV_DEV_BAD_LENGTH, 0x40, kv.SV_DEV_BAD_PAGE
    assert status.cpu().tolist() == [L, L, T, T, T, T, L, G, T]
    assert out.cpu().tolist() == lens.tolist()
    assert torch.equal(k, k0) and torch.equal(v, v0)


# ---------------------------------------------------------------- together

def test_another_stream_and_two_at_once(kv):
    """Two calls on two streams, each with its own workspace, and one stream given by hand."""
    r = Round([3000, 50], 5, "tree", heads=2, group=4, dim=128, seed=1)
    c = r.paged(kv)
    q, lens, par = r.q.cuda(), r.lens.cuda(), r.parents.cuda()
    outs = [torch.full_like(q, 7.0) for _ in range(2)]
    wss = [kv.attention_workspace(c, r.B, r.N, 8) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(streams[0]):
            kv.spec_kv_attention(c, q, lens, outs[0], wss[0], r.scale, parents=par)
        kv.spec_kv_attention(c, q, lens, outs[1], wss[1], r.scale, parents=par,
                             stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    r.check(outs[0].cpu())


def test_workspace_reused_by_other_sizes(kv):
    """One workspace, of the largest call, through calls of different shapes on one stream."""
    a = Round([3000, 50], 16, "tree", heads=1, group=8, dim=128, seed=1)
    b = Round([400, 5, 77], 1, heads=1, group=8, dim=128, seed=2)
    ca, cb = a.paged(kv), b.paged(kv)
    n = max(kv.spec_kv_attention_workspace_size(r.B, r.N, 8, 1, 128) for r in (a, b))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for r, c in ((a, ca), (b, cb)):
            out = torch.full_like(r.q, 7.0, device="cuda")
            kv.spec_kv_attention(c, r.q.cuda(), r.lens.cuda(), out, ws, r.scale,
                                 parents=None if r.parents is None else r.parents.cuda())
            r.check(out.cpu())


def rounds(kv, sv, steps, capture):
    """Greedy tree decoding of a toy attention model, every call on the device: tokens have fixed
    random q, k, v; logits are out @ head.  Returns the state after `steps` rounds."""
    g = torch.Generator().manual_seed(5)
    B, N, H, G, D, V, page, layers = 3, 9, 2, 4, 64, 6, 16, 2
    hq = H * G
    emb = [torch.randn(V, n, D, generator=g).to(BF).cuda() for n in (hq, H, H)] * layers
    head = torch.randn(hq * D, V, generator=g).cuda()
    width = 8
    table = torch.randperm(B * width, generator=g).view(B, width).to(torch.int32).cuda()
    k = torch.full((layers, B * width, page, H, D), math.nan, dtype=BF, device="cuda")
    v = torch.full_like(k, math.nan)
    cache = kv.PagedCache(k, v, table)
    rope = kv.Rope(D)
    par = torch.tensor([[0, 0, 0, 0, 1, 1, 2, 4, 4]] * B, dtype=torch.int32, device="cuda")
    tokens = torch.randint(0, V, (B, 1), generator=g).to(torch.int32).cuda()
    kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    new_len = torch.zeros_like(kv_len)
    ws = kv.attention_workspace(cache, B, N, hq)
    vws = sv.workspace(B, N - 1, V, torch.float32)
    out = torch.zeros(B, N, hq, D, dtype=BF, device="cuda")
    q = torch.zeros_like(out)
    logits = torch.zeros(B, N, V, device="cuda")
    out_tokens, out_nodes = (torch.zeros(B, N, dtype=torch.int32, device="cuda") for _ in range(2))
    acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    drafts = torch.zeros(B, N, dtype=torch.int32, device="cuda")

    def step():
        t = drafts.long()
        for i in range(layers):
            eq, ek, ev = emb[3 * i:3 * i + 3]
            kv.spec_kv_append(cache, ek[t], ev[t], kv_len, q=eq[t], q_out=q, rope=rope,
                              parents=par, layer=i)
            kv.spec_kv_attention(cache, q, kv_len, out, ws, D ** -0.5, parents=par, layer=i)
        logits.copy_(out.float().reshape(B, N, hq * D) @ head)
        sv.spec_verify_tree(sv.SV_MODE_GREEDY, logits, None, drafts, par, None, None, 1.0,
                            out_tokens, out_nodes, acc, vws)
        kv.spec_kv_commit(cache, kv_len, acc, new_len, out_nodes)
        kv_len.copy_(new_len)

    committed = [[int(x)] for x in tokens[:, 0]]
    graph = None
    took = []
    for s in range(steps):
        d = torch.randint(0, V, (B, N), generator=g).to(torch.int32)
        d[:, 0] = torch.tensor([c[-1] for c in committed])
        drafts.copy_(d)
        if capture and s == 1:
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        if graph is not None:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        n = acc.cpu().tolist()
        ot = out_tokens.cpu()
        for b in range(B):
            committed[b] += ot[b, :n[b] + 1].tolist()
        took.append(n)
    return dict(committed=committed, kv_len=kv_len.cpu(), k=k.cpu(), v=v.cpu(),
                table=table.cpu(), emb=[e.cpu() for e in emb], head=head.cpu(), took=took,
                sizes=(B, N, H, G, D, V, page, layers))


@pytest.mark.parametrize("capture", [False, True])
def test_whole_rounds(kv, capture):
    """append, attention, tree verify and commit for several rounds, eager and as one captured
    graph replayed: the cache holds exactly the committed tokens' rotated keys and their values,
    and each emitted token is the argmax of plain causal attention over the committed ones."""
    from speculative_decoding_verification_18_gb300 import specverify as sv
    s = rounds(kv, sv, 12, capture)
    B, N, H, G, D, V, page, layers = s["sizes"]
    rate = kv_plain.rates(D, 10000.0)
    told = 0  # tokens that the comparison rules out
    for b in range(B):
        toks = s["committed"][b]
        n = int(s["kv_len"][b])
        assert n == len(toks) - 1  # the last emitted token is the next round's root
        at = kv_plain.slots(s["table"][b], page, n)
        for i in range(layers):
            eq, ek, ev = s["emb"][3 * i:3 * i + 3]
            for t in range(n):
                y, slack = kv_plain.rotate(ek[toks[t]], t, rate, False)
                err = (s["k"][i][at[t]].double() - y).abs()
                assert bool((err <= kv_plain.stored_bound(y, slack, BF)).all())
                assert torch.equal(s["v"][i][at[t]], ev[toks[t]])
        # the last layer's attention of the token at t gives token t + 1
        eq, ek, ev = s["emb"][3 * (layers - 1):]
        kk = torch.stack([s["k"][layers - 1][a] for a in at]).double()
        vv = torch.stack([s["v"][layers - 1][a] for a in at]).double()
        for t in range(n):
            y, slack = kv_plain.rotate(eq[toks[t]], t, rate, False)
            x = y.to(BF).double().view(H, G, D)
            p = torch.softmax(torch.einsum("hgd,lhd->hgl", x, kk[:t + 1]) * D ** -0.5, -1)
            o = torch.einsum("hgl,lhd->hgd", p, vv[:t + 1]).reshape(-1)
            logits = o @ s["head"].double()
            # each weight is off by at most 2^-8 twice (its own rounding and the query's), the
            # result by 2^-8: the emitted token's logit is that near the top one
            off = (5 * 2.0 ** -8) * torch.einsum("hgl,lhd->hgd", p, vv[:t + 1].abs()).reshape(-1)
            slack = off @ s["head"].double().abs()
            assert logits[toks[t + 1]] + 2 * slack.max() >= logits.max()
            told += int((logits < logits.max() - 2 * slack.max()).sum())
    assert told > 0 and sum(sum(n) for n in s["took"]) > 0


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch, kv_plain
from test_kv_gpu import Round
from speculative_decoding_verification_18_gb300 import kvcache as kv
for N, far in ((1, False), (1, True), (16, True)):
    r = Round([300, 40], N, "tree", heads=1, group=8, dim=128, seed=N, far=far)
    c, q, lens, par = r.paged(kv), r.q.cuda(), r.lens.cuda(), r.parents.cuda()
    out, ws = torch.full_like(q, 7.0), kv.attention_workspace(c, 2, N, 8)
    acc, new = torch.zeros_like(lens), torch.zeros_like(lens)
    k = torch.stack([r.k[r.table[b, (int(r.lens[b]) + j) // r.page].item(),
                         (int(r.lens[b]) + j) % r.page] for b in range(2) for j in range(N)])
    v = torch.stack([r.v[r.table[b, (int(r.lens[b]) + j) // r.page].item(),
                         (int(r.lens[b]) + j) % r.page] for b in range(2) for j in range(N)])
    k, v = k.view(2, N, 1, 128).cuda(), v.view(2, N, 1, 128).cuda()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        kv.spec_kv_append(c, k, v, lens, parents=par)
        kv.spec_kv_attention(c, q, lens, out, ws, r.scale, parents=par)
        kv.spec_kv_commit(c, lens, acc, new)
    for _ in range(2):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        r.check(out.cpu())
        assert new.cpu().tolist() == [301, 41]
print("captured")
"""


def test_first_calls_of_a_process_inside_a_capture(kv):
    """Nothing that the calls set up on a device needs an eager call first."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests)
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "captured" in got.stdout, got.stderr[-2000:]


def test_two_graphs_share_a_workspace(kv):
    """Two captured calls of different sizes on one workspace, replayed in turn on one stream."""
    a = Round([3000, 50], 16, "tree", heads=1, group=8, dim=128, seed=1, far=True)
    b = Round([400, 5, 77], 2, heads=1, group=8, dim=128, seed=2, far=True)
    n = max(kv.spec_kv_attention_workspace_size(r.B, r.N, 8, 1, 128) for r in (a, b))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    held = []
    for r in (a, b):
        c, q, lens = r.paged(kv), r.q.cuda(), r.lens.cuda()
        par = None if r.parents is None else r.parents.cuda()
        out = torch.full_like(q, 7.0)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            kv.spec_kv_attention(c, q, lens, out, ws, r.scale, parents=par)
        held.append((r, graph, out, (c, q, lens, par)))
    for _ in range(3):
        for r, graph, out, _ in held:
            out.fill_(7.0)
            graph.replay()
        torch.cuda.synchronize()
        for r, graph, out, _ in held:
            r.check(out.cpu())
