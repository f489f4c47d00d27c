"""Attention through a window on the GPU against the plain float64 implementation
(window_plain.py): windows and first slots around page and tile borders, pages given back, trees
whose rows differ in what they see, every type and form, values that are not finite in hidden
places, bad data, streams and captured graphs."""
import math

import pytest
import torch

import kv_plain
import window_plain
from kv_plain import E4M3
from parity import Guarded
from test_kv_gpu import Round

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
TYPES = [(BF, BF), (HF, HF), (BF, E4M3), (HF, E4M3)]
ALL = 1 << 30  # a window or a number of first slots that hides nothing


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verification_18_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(scope="module")
def kv():
    from speculative_decoding_verification_18_gb300 import kvcache
    return kvcache


class Windowed(Round):
    """A round whose slots outside of every node's view are NaN and whose pages wholly outside have
    left the table.  (far: the table has room for more than 8192 slots, and so has the window
    where it hides nothing: ranges of slots instead of a cluster per item.)"""

    def __init__(self, lens, N, window, sinks, *a, **kw):
        super().__init__(lens, N, *a, **kw)
        self.window, self.sinks = window, sinks
        for b in range(self.B):
            n, m = int(self.lens[b]), int(self.counts[b])
            low = max(0, n - window + 1)
            hidden = [s for s in range(n + m) if sinks <= s < low]
            at = kv_plain.slots(self.table[b], self.page, n + m)
            for s in hidden:
                for pool in (self.k, self.v):
                    pool[at[s]] = torch.full((self.heads, self.dim), math.nan).to(self.cache)
            for p in range((n + m) // self.page):
                if all(s in hidden for s in range(p * self.page, (p + 1) * self.page)):
                    self.table[b, p] = -1 if b % 2 else 1 << 20

    def attend(self, kv, stream=None, ws=None):
        d = lambda x: None if x is None else x.cuda()
        c, gd = self.paged(kv), Guarded()
        out = gd.empty(self.q.shape, self.dtype, fill=7.0)
        n = kv.spec_kv_attention_workspace_size(self.B, self.N, self.heads * self.group, self.heads,
                                                self.dim)
        ws = gd.empty((n,), torch.uint8, fill=255)  # NaN wherever it is read unwritten
        status = gd.empty((self.B,), torch.int32, fill=0)
        kv.spec_kv_attention_window(c, d(self.q), d(self.lens), out, ws, self.scale, self.window,
                                    self.sinks, parents=d(self.parents),
                                    num_new=d(self.counts) if self.ragged else None, status=status)
        gd.check()
        return out.cpu(), status.cpu().tolist()

    def plain(self):
        return window_plain.attention(self.q, self.k, self.v, self.table, self.lens, self.counts,
                                      self.parents, self.scale, self.window, self.sinks,
                                      self.k_scale, self.v_scale)

    def check(self, out):
        window_plain.check(out, self.plain(), self.dtype, self.counts, torch.full_like(out, 7.0))


def good(r, kv):
    out, status = r.attend(kv)
    assert status == [0] * r.B
    r.check(out)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 128])
@pytest.mark.parametrize("order", ["slot", "head"])
@pytest.mark.parametrize("N,group", [(3, 2), (3, 5), (4, 6), (5, 5), (6, 8), (20, 8)])
def test_types_and_heads(kv, dtype, cache, dim, order, N, group):
    """(Three heads: a cluster per item; ten: ranges.)"""
    good(Windowed([37, 0, 230, 64], N, 50, 3, "tree", heads=3 if order == "slot" else 10,
                  group=group, dim=dim, dtype=dtype, cache=cache, order=order, seed=dim + N), kv)


@pytest.mark.parametrize("window", [1, 3, 16, 64, 65, 129, ALL])
@pytest.mark.parametrize("sinks", [0, 1, 70, ALL])
@pytest.mark.parametrize("N,form,heads,group", [
    (1, "chain", 1, 4), (9, "chain", 1, 3),    # a cluster per item
    (2, "chain", 20, 1), (9, "tree", 10, 2),   # ranges, few rows
    (12, "tree", 10, 8), (50, "star", 10, 4), (65, "chain", 5, 4)])  # many rows
def test_windows_and_first_slots(kv, window, sinks, N, form, heads, group):
    good(Windowed([0, 2, 130, 333], N, window, sinks, form, heads=heads, group=group, dim=64,
                  seed=window % 97 + sinks % 89), kv)


@pytest.mark.parametrize("page", [1, 4, 16, 64, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 4), (100, 20)])
@pytest.mark.parametrize("N,heads,group", [(1, 1, 3), (1, 3, 3), (6, 1, 3), (6, 3, 3), (12, 1, 8)])
def test_lengths_around_borders(kv, page, window, sinks, N, heads, group):
    lens = [0, 1, 15, 16, 17, 32, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 300]
    good(Windowed(lens, N, window, sinks, heads=heads, group=group, dim=64, page=page, seed=page),
         kv)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("N,group,form", [(1, 4, "chain"), (4, 8, "tree"), (16, 8, "tree"),
                                          (33, 7, "tree")])
def test_split_over_a_long_window(kv, dtype, cache, N, group, form):
    """A sequence with a window that several CTAs hold a part of, and a short one beside it."""
    good(Windowed([1503, 40], N, 1000, 150, form, heads=20, group=group, dim=128, dtype=dtype,
                  cache=cache, page=32, seed=N), kv)


@pytest.mark.parametrize("B", [1, 150, 700])
@pytest.mark.parametrize("N,group", [(1, 2), (6, 4), (12, 8)])
def test_many_sequences(kv, B, N, group):
    """Every third sequence has nothing new, every fourth nothing cached."""
    g = torch.Generator().manual_seed(B)
    lens = [0 if b % 4 == 3 else int(torch.randint(0, 200, (1,), generator=g)) for b in range(B)]
    counts = [0 if b % 3 == 2 else 1 + b % N for b in range(B)]
    good(Windowed(lens, N, 20, 2, "tree", counts=counts, heads=1, group=group, dim=16, page=8,
                  seed=B), kv)


@pytest.mark.parametrize("N,group,form", [(1, 4, "chain"), (6, 4, "chain"), (16, 8, "tree"),
                                          (65, 8, "star")])
@pytest.mark.parametrize("dtype,cache", TYPES)
def test_a_window_that_hides_nothing(kv, N, group, form, dtype, cache):
    """The same bits as without a window."""
    r = Windowed([300, 0, 77], N, 300 + N, 0, form, heads=2, group=group, dim=64, dtype=dtype,
                 cache=cache)
    out, status = r.attend(kv)
    assert status == [0] * 3
    full, _ = Round.attend(r, kv)
    assert torch.equal(out, full)
    r.window, r.sinks = 1, 300 + N
    out, _ = r.attend(kv)
    assert torch.equal(out, full)


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (1, 2 ** 31 - 1),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("N,heads,group", [(3, 1, 4), (3, 20, 4), (9, 10, 8)])
def test_the_largest_windows(kv, window, sinks, N, heads, group):
    good(Windowed([200, 0, 31], N, window, sinks, "tree", heads=heads, group=group, dim=64), kv)


@pytest.mark.parametrize("N,group", [(1, 4), (6, 4), (16, 8), (65, 4)])
def test_the_same_bits_each_time(kv, N, group):
    r = Windowed([900, 300, 0], N, 500, 20, "tree", heads=14, group=group, dim=64, seed=N)
    first, _ = r.attend(kv)
    for _ in range(4):
        assert torch.equal(r.attend(kv)[0], first)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("N,group,form", [(6, 2, "chain"), (7, 4, "tree"), (16, 8, "tree"),
                                          (40, 8, "chain")])
@pytest.mark.parametrize("heads", [2, 10])
def test_hidden_places_may_hold_anything(kv, heads, dtype, cache, N, group, form):
    """The first slot of the root's window is out of its descendants' reach: NaN or an infinity
    there reaches the root's row only; behind a first slot it would reach all."""
    r = Windowed([270, 133, 160, 500], N, 40, 3, form, heads=heads, group=group, dim=64,
                 dtype=dtype, cache=cache, seed=5)
    want, bound, _ = r.plain()
    for b, bad in enumerate((math.nan, math.inf, -math.inf, math.nan)):
        s = int(r.lens[b]) - 39
        at = int(r.table[b, s // r.page]), s % r.page
        for pool in (r.k, r.v):
            pool[at] = torch.full((heads, 64), bad if cache != E4M3 else math.nan).to(cache)
    out, status = r.attend(kv)
    assert status == [0] * 4
    assert bool(torch.isnan(out[:, 0].float()).any(dim=-1).all())
    err = (out.double() - want).abs()[:, 1:]
    assert bool((err <= bound[:, 1:]).all())


@pytest.mark.parametrize("heads", [1, 20])
@pytest.mark.parametrize("N,group", [(5, 2), (16, 8)])
def test_new_tokens_out_of_reach(kv, heads, N, group):
    """A window shorter than the chain: a new token that is not finite is seen by those behind it
    that its window still reaches."""
    r = Windowed([100, 0], N, 3, 0, heads=heads, group=group, dim=64, seed=6)
    want, bound, _ = r.plain()
    for b in range(2):
        s = int(r.lens[b]) + 1
        r.v[int(r.table[b, s // r.page]), s % r.page] = math.inf
    out, _ = r.attend(kv)
    assert bool((~torch.isfinite(out[:, 1:4].float())).all())
    err = (out.double() - want).abs()
    assert bool((err <= bound)[:, 0].all()) and bool((err <= bound)[:, 4:].all())


@pytest.mark.parametrize("heads", [2, 6])
@pytest.mark.parametrize("N,group", [(6, 3), (20, 8)])
def test_bad_data(kv, heads, N, group):
    """Bad lengths, counts, trees and pages: NaN rows and the bit, the others untouched by it."""
    r = Windowed([240, 250, 260, 270, 280, 233, 220, 290], N, 30, 4, "tree",
                 counts=[N, N, N, N, N, N, 3, N], heads=heads, group=group, dim=64, seed=9)
    want, bound, _ = r.plain()
    width = r.table.shape[1] * r.page
    r.lens[0] = -1
    r.lens[1] = width - N + 1
    r.counts[2] = N + 1
    r.counts[3] = -1
    r.parents[4, 2] = 2
    r.parents[5, 3] = -1
    r.parents[6, 4] = 77                # behind its three tokens: not read
    r.table[7, 0] = r.k.shape[0]        # the page of the first slots
    out, status = r.attend(kv)
    L, T, G = kv.SV_DEV_BAD_LENGTH, 0x40, kv.SV_DEV_BAD_PAGE
    assert status == [L, L, L, L, T, T, 0, G]
    assert bool(torch.isnan(out[[0, 1, 2, 3, 4, 5, 7]].float()).all())
    assert bool(((out[6, :3].double() - want[6, :3]).abs() <= bound[6, :3]).all())
    assert bool((out[6, 3:] == 7.0).all())


@pytest.mark.parametrize("heads", [1, 20])
@pytest.mark.parametrize("N,group", [(1, 4), (16, 8)])
def test_bad_page_where_the_window_begins(kv, heads, N, group):
    r = Windowed([1000, 1000], N, 100, 4, heads=heads, group=group, dim=64, seed=1)
    want, bound, _ = r.plain()
    r.table[0, 901 // r.page] = -1
    out, status = r.attend(kv)
    assert status == [kv.SV_DEV_BAD_PAGE, 0]
    assert bool(torch.isnan(out[0].float()).all())
    assert bool(((out[1].double() - want[1]).abs() <= bound[1]).all())


@pytest.mark.parametrize("heads", [1, 40])
@pytest.mark.parametrize("N,group,dtype,cache", [(1, 4, BF, BF), (9, 8, BF, BF), (9, 8, HF, E4M3),
                                                 (3, 8, BF, E4M3)])
def test_positions_up_to_the_last_slot(kv, heads, N, group, dtype, cache):
    """Positions just below 2^31, of which a window and four first slots are held."""
    page, W, S, dim = 128, 300, 4, 64
    width = (1 << 31) // page - 1
    n = width * page - N
    g = torch.Generator().manual_seed(N)
    pages = 6
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    first = (n - W + 1) // page
    table[0, 0] = 5
    table[0, first:] = torch.arange(width - first, dtype=torch.int32, device="cuda")
    assert width - first <= 5
    k, v = ((torch.randn(pages, page, heads, dim, generator=g) * 4).to(cache) for _ in range(2))
    q = torch.randn(1, N, heads * group, dim, generator=g).to(dtype)
    scales = [torch.full((heads,), 0.25)] * 2 if cache == E4M3 else [None] * 2
    d = lambda x: None if x is None else x.cuda()
    c = kv.PagedCache(k.cuda(), v.cuda(), table, *(d(x) for x in scales))
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    ws = kv.attention_workspace(c, 1, N, heads * group)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.spec_kv_attention_window(c, q.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                out, ws, dim ** -0.5, W, S, status=status)
    assert status.tolist() == [0]
    # the same slots in a short sequence whose window begins at the same place of a page
    cut = S + (n - W + 1) % page
    short = torch.tensor([[5] + list(range(width - first))], dtype=torch.int32)
    m = n - first * page + page  # slots: one page of first ones, then the window's pages
    want = window_plain.attention(q, k, v, short, [m], [N], None, dim ** -0.5, W, S, *scales)
    assert cut > 0
    window_plain.check(out.cpu(), want, dtype, [N])


def test_streams_and_captured_graphs(kv):
    """Two graphs over one workspace, replayed in turn with other queries, and another stream."""
    rs = [Windowed([200, 90], 4, 50, 4, heads=20, group=4, dim=64, seed=1),
          Windowed([700, 300], 20, 64, 4, "tree", heads=2, group=8, dim=64, seed=2)]
    size = max(kv.spec_kv_attention_workspace_size(2, r.N, r.heads * r.group, r.heads, 64)
               for r in rs)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    held = []
    for r in rs:
        c, q, lens = r.paged(kv), r.q.cuda(), r.lens.cuda()
        par, out = None if r.parents is None else r.parents.cuda(), torch.zeros_like(q)
        call = lambda: kv.spec_kv_attention_window(c, q, lens, out, ws, r.scale, r.window, r.sinks,
                                                   parents=par)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        r.check(out.cpu())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        held.append((graph, out, q, (c, lens, par)))
    for step in range(2):
        for r, (graph, out, q, _) in zip(rs, held):
            r.q = torch.randn(r.q.shape, generator=r.g).to(r.dtype)
            q.copy_(r.q)
            graph.replay()
            torch.cuda.synchronize()
            r.check(out.cpu())


def test_a_round_through_the_window(kv):
    """Append, attention through a window and commit, round after round, while pages that leave the
    window are given back: the same rows as the plain form over everything that was committed."""
    B, H, G, D, page, W, S, N, rounds = 2, 2, 4, 64, 16, 40, 4, 5, 12
    g = torch.Generator().manual_seed(7)
    width = (rounds * N + N + page - 1) // page + 1
    pages = B * width
    k = torch.full((pages, page, H, D), math.nan, dtype=BF, device="cuda")
    v = k.clone()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, width)
    c = kv.PagedCache(k, v, table)
    ws = kv.attention_workspace(c, B, N, H * G)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    after = torch.zeros_like(lens)
    past = [[], []]  # committed entries (key, value), unrotated keys: no rotation here
    for _ in range(rounds):
        kn, vn = (torch.randn(B, N, H, D, generator=g).to(BF) for _ in range(2))
        q = torch.randn(B, N, H * G, D, generator=g).to(BF)
        out = torch.empty_like(q, device="cuda")
        kv.spec_kv_append(c, kn.cuda(), vn.cuda(), lens)
        kv.spec_kv_attention_window(c, q.cuda(), lens, out, ws, D ** -0.5, W, S)
        taken = torch.randint(0, N, (B,), generator=g).to(torch.int32)
        kv.spec_kv_commit(c, lens, taken.cuda(), after)
        for b in range(B):
            n = len(past[b])
            rows = past[b] + [(kn[b, j], vn[b, j]) for j in range(N)]
            kk, vv = (torch.stack([x[i] for x in rows])[None] for i in range(2))
            want = window_plain.attention(q[b:b + 1], kk, vv, torch.zeros(1, 1, dtype=torch.int32),
                                          [n], [N], None, D ** -0.5, W, S)
            window_plain.check(out[b:b + 1].cpu(), want, BF, [N])
            past[b] = rows[:n + 1 + int(taken[b])]
            assert int(after[b]) == len(past[b])
            for p in range(1, max(0, len(past[b]) - W + 1) // page):  # wholly behind the window
                table[b, p] = -1
        lens.copy_(after)
