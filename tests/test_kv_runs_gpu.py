"""Cache calls over many tokens and many planes on the GPU: there a CTA of append takes several
tokens in turn and a CTA of commit several layers' keys and values.  Compared on the device with
float64 (append) or bit by bit (commit)."""
import pytest
import torch

import kv_plain
from kv_plain import E4M3
from parity import Guarded
from test_kv_gpu import BF, HF, Round, built, kv, tree  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def depths(parents, B, N):
    """[B, N] depth of each node on the CPU."""
    if parents is None:
        return torch.arange(N).expand(B, N)
    d = torch.zeros(B, N, dtype=torch.long)
    for j in range(1, N):
        d[:, j] = d.gather(1, parents[:, j:j + 1].long())[:, 0] + 1
    return d


def entries_at(pool, place):
    """pool[page, slot] for an index pair, float8 by its bytes."""
    return pool[place] if pool.element_size() > 1 else \
        pool.view(torch.uint8)[place].view(pool.dtype)


# Tokens per CTA: those of all sequences over six per SM, four at most.
@pytest.mark.parametrize("run", [2, 3, 4])
@pytest.mark.parametrize("heads,group,dim,rot,dtype,cache,form,kw", [
    (1, 0, 16, 0, BF, BF, "chain", {}),              # two threads per CTA
    (1, 0, 16, 16, HF, HF, "tree", {}),
    (1, 1, 16, 0, BF, E4M3, "tree", {}),             # three
    (1, 1, 16, 16, BF, BF, "chain", dict(in_place=True)),
    (1, 2, 16, 16, BF, BF, "tree", {}),              # four
    (2, 4, 64, 64, BF, BF, "tree", {}),
    (2, 4, 64, 20, HF, E4M3, "tree", dict(interleaved=True)),
    (8, 16, 128, 128, BF, BF, "tree", dict(in_place=True)),  # more heads than one pass takes
    (8, 16, 128, 64, HF, HF, "chain", dict(interleaved=True)),
    (3, 5, 80, 40, BF, E4M3, "star", {}),
])
def test_append_runs_of_tokens(kv, run, heads, group, dim, rot, dtype, cache, form, kw):
    g = torch.Generator().manual_seed(run * 100 + heads)
    N = 65 if run > 2 else 33
    B = (6 * sms() * run + N - 1) // N
    page, hq = 16, heads * group
    lens = torch.randint(0, 50, (B,), generator=g).to(torch.int32)
    # ragged, with counts of 0, of N, and of every remainder by the run's length
    counts = torch.tensor([N if b % 5 == 0 else (b * 7) % (N + 1) for b in range(B)],
                          dtype=torch.int32)
    parents = None if form == "chain" else torch.stack([tree(N, form, g) for _ in range(B)])
    width = (50 + N + page - 1) // page
    pages = B * width
    table = torch.randperm(pages, generator=g).to(torch.int32).view(B, width).cuda()
    rand = lambda *s: torch.randn(*s, generator=g).cuda()
    gd = Guarded()
    pools = [gd.empty((pages, page, heads, dim), torch.uint8 if cache == E4M3 else dtype)
             for _ in range(2)]
    for p in pools:
        p.view(torch.uint8).fill_(0x31)
    pools = [p.view(cache) for p in pools]
    scales = [None, None]
    if cache == E4M3:
        scales = [torch.rand(heads, generator=g).cuda() * 0.02 + 0.01 for _ in range(2)]
    before = [p.view(torch.uint8).clone() for p in pools]
    c = kv.PagedCache(*pools, table, *scales)
    q = rand(B, N, hq, dim).to(dtype) if group else None
    k, v = rand(B, N, heads, dim).to(dtype), rand(B, N, heads, dim).to(dtype)
    out = gd.empty((B, N, hq, dim), dtype, fill=7.0) if group else None
    if kw.get("in_place"):
        out.copy_(q)
    held = None if out is None else out.clone()
    interleaved = kw.get("interleaved", False)
    rope = kv.Rope(rot, interleaved=interleaved) if rot else None
    status = gd.empty((B,), torch.int32, fill=0)
    kv.spec_kv_append(c, k, v, lens.cuda(), q=out if kw.get("in_place") else q, q_out=out,
                      rope=rope, parents=None if parents is None else parents.cuda(),
                      num_new=counts.cuda(), status=status)
    gd.check()
    assert not bool(status.any())

    live = (torch.arange(N) < counts[:, None]).cuda()
    pos = (lens[:, None] + depths(parents, B, N)).cuda()[:, :, None, None].double()
    rate = kv_plain.rates(rot, 10000.0).cuda()

    def turned(x):
        x = x.double()
        i = torch.arange(rot // 2, device="cuda")
        one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y, slack = x.clone(), torch.zeros_like(x)
        a, b, co, si = x[..., one], x[..., two], torch.cos(pos * rate), torch.sin(pos * rate)
        y[..., one], y[..., two] = a * co - b * si, b * co + a * si
        slack[..., one] = slack[..., two] = a.abs() + b.abs()
        return y, slack

    if group:
        y, slack = turned(q)
        off = (out.double() - y).abs()
        assert bool((off <= kv_plain.stored_bound(y, slack, dtype))[live].all())
        assert torch.equal(out[~live], held[~live])
    slot = (lens[:, None] + torch.arange(N)).long().cuda()
    place = table.long().gather(1, slot // page)[live], (slot % page)[live]
    for pool, was, x, scale, turn in zip(pools, before, (k, v), scales, (True, False)):
        y, slack = turned(x) if turn else (x.double(), torch.zeros_like(x, dtype=torch.float64))
        y, slack = y[live], slack[live]
        got, one = entries_at(pool, place).double(), None
        if cache == E4M3:
            one = scale.double()[:, None]
            got, y = got * one, y.clamp(-448 * one, 448 * one)
        assert bool(((got - y).abs() <= kv_plain.stored_bound(y, slack, cache, one)).all())
        now = pool.view(torch.uint8).clone()
        now[place], was[place] = 0, 0
        assert torch.equal(now, was)  # nothing else was written


# Planes (a layer's keys or values) per CTA: those of all sequences over eight CTAs per SM.
@pytest.mark.parametrize("cache,heads,dim,order", [
    (BF, 8, 128, "slot"),     # 128 columns of 16 bytes: a plane fills the block
    (BF, 9, 128, "head"),     # 144: two blocks, the second mostly empty
    (E4M3, 16, 128, "slot"),
    (HF, 2, 64, "head"),      # 16: eight planes side by side
    (E4M3, 1, 16, "slot"),    # one
    (BF, 3, 80, "slot"),      # 30: four planes, eight threads left over
])
@pytest.mark.parametrize("N,few", [(65, False), (9, True), (2, True)])
def test_commit_runs_of_planes(kv, cache, heads, dim, order, N, few):
    """Every CTA takes more planes than it has side by side, with 0 to N - 1 moves in each."""
    g = torch.Generator().manual_seed(N + heads)
    size = 1 if cache == E4M3 else 2
    units = heads * dim * size // 16
    side = max(1, 128 // units)
    layers = 24
    blocks = (units + 127) // 128
    B = 8 * sms() * (2 * side + 1) // (2 * layers * blocks) + 1  # more than two turns per CTA
    if 2 * side + 1 > 2 * layers:
        layers, B = 140, 8 * sms() * 270 // 280 + 1
    page, span = 8, 40
    width = (span + N + page) // page
    # all pages but those of the committed slots are a sequence's own
    pages = B * width
    lens = torch.randint(0, span, (B,), generator=g).to(torch.int32)
    table = torch.randperm(pages, generator=g).view(B, width).to(torch.int32).cuda()
    nodes = torch.full((B, N), -1, dtype=torch.int32)
    acc = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        most = 1 + (b % 3 if few else N - 1)
        n = int(torch.randint(0, min(N, most + 1), (1,), generator=g))
        pick = torch.randperm(N - 1, generator=g)[:n].sort().values + 1
        if b % 4 == 0:  # the first ones stay where they are
            pick[:n // 2] = torch.arange(1, n // 2 + 1)
            pick = pick.unique()
        acc[b] = len(pick)
        nodes[b, :len(pick)] = pick.to(torch.int32)
    bits = torch.uint8 if size == 1 else torch.int16
    inner = (page, heads, dim) if order == "slot" else (heads, page, dim)
    gd, want = Guarded(), []
    pools = [gd.empty((layers, pages) + inner, bits) for _ in range(2)]
    dg = torch.Generator(device="cuda").manual_seed(7)
    look = (lambda x: x) if order == "slot" else (lambda x: x.transpose(2, 3))
    to = torch.arange(1, N + 1).expand(B, N)
    moved = (torch.arange(N) < acc[:, None])

    def place(node):
        slot = (lens[:, None] + node.long()).cuda()
        m = moved.cuda()
        return table.long().gather(1, (slot // page).clamp(0, width - 1))[m], (slot % page)[m]

    src, dst = place(nodes.clamp(min=0)), place(to)
    for p in pools:
        p.random_(0, 120, generator=dg)
        x = look(p.clone())
        x[:, dst[0], dst[1]] = x[:, src[0], src[1]]
        want.append(x)
    c = kv.PagedCache(look(pools[0].view(cache)), look(pools[1].view(cache)), table)
    out = gd.empty((B,), torch.int32, fill=-7)
    status = gd.empty((B,), torch.int32, fill=0)
    kv.spec_kv_commit(c, lens.cuda(), acc.cuda(), out, nodes.cuda(), status=status)
    gd.check()
    assert not bool(status.any())
    assert torch.equal(out.cpu(), lens + acc + 1)
    for p, w in zip(pools, want):
        assert torch.equal(look(p), w)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_float8_is_the_quotient_rounded(kv, dtype):
    """Entries are the quotient by the head's scale, rounded to nearest even, in every bit: among
    them quotients half way between two float8 values, where the product with the scale's rounded
    reciprocal lies on the other side."""
    ties = torch.tensor([t * 2.0 ** e for t in range(17, 32, 2) for e in range(-6, 5)])
    odd = torch.arange(3, 128, 2).float()
    odd[1::2] *= -1
    heads, D = len(odd), 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 60, heads, D, generator=g)
    x[0, :, :, :len(ties)] = ties * odd[:, None]  # exact in the type for the smaller scales
    x[0, 1::2] *= -1
    x = x.to(dtype)
    N = x.shape[1]
    lens = torch.tensor([5], dtype=torch.int32)
    k, v = (torch.zeros(5, 16, heads, D, dtype=torch.uint8, device="cuda").view(E4M3)
            for _ in range(2))
    table = torch.arange(5, dtype=torch.int32).view(1, 5).cuda()
    c = kv.PagedCache(k, v, table, odd.cuda(), (odd / 3).cuda())
    kv.spec_kv_append(c, x.cuda(), x.cuda(), lens.cuda())
    for pool, scale in ((k, odd), (v, odd / 3)):
        got = pool.view(torch.uint8).view(-1, heads, D)[5:5 + N].cpu()
        want = (x[0].float() / scale[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("cache,N,group", [(BF, 1, 4), (BF, 4, 4), (BF, 4, 8), (BF, 9, 8),
                                           (BF, 33, 8), (E4M3, 4, 8), (E4M3, 33, 8)])
def test_attention_up_to_the_last_slot(kv, cache, N, group):
    """A table of 2^31 - 8 slots, filled to the last one: 2^28 - 1 pages of eight, all but the new
    tokens' the same.  With queries of zero all weights are equal: committed values are zero, a
    new token's is 2^31 times its number, so that each row is the sum of the numbers it sees."""
    page, dim, width = 8, 16, (1 << 28) - 1
    slots = width * page
    own = (N + page - 1) // page + 1
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[0, width - own:] = torch.arange(1, own + 1, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(own + 1, page, 1, dim, dtype=BF, device="cuda") for _ in range(2))
    numbers = torch.arange(1, N + 1, device="cuda") % 5
    one = 1.0 if cache == E4M3 else 2.0 ** 31  # float8: the scale has it
    v.view(-1, dim)[(own + 1) * page - N:] = (numbers.double() * one).to(BF)[:, None]
    scales = [torch.ones(1, device="cuda"), torch.full((1,), 2.0 ** 31, device="cuda")]
    g = torch.Generator().manual_seed(N)
    parents = tree(N, "tree", g)
    lens = torch.tensor([slots - N], dtype=torch.int32, device="cuda")
    c = kv.PagedCache(k.to(cache), v.to(cache), table, *(scales if cache == E4M3 else []))
    q = torch.zeros(1, N, group, dim, dtype=BF, device="cuda")
    out, status = torch.full_like(q, 7.0), torch.zeros_like(lens)
    kv.spec_kv_attention(c, q, lens, out, kv.attention_workspace(c, 1, N, group), 1.0,
                         parents=parents.view(1, N).cuda(), status=status)
    assert status.tolist() == [0], status.tolist()
    up = kv_plain.paths(parents, N)
    seen = torch.tensor([len(p) for p in up]).double()  # of them and of the committed slots
    want = torch.tensor([sum(int(numbers[i]) for i in p) for p in up]).double()
    want = want * 2.0 ** 31 / (slots - N + seen)
    # whole numbers: the sums are exact, but for those of the pieces' counts (2^-24 per piece)
    off = (out.cpu().double() - want[None, :, None, None]).abs()
    assert bool((off <= (kv_plain.U[BF] + 305 * 2.0 ** -24) * want[None, :, None, None]).all())


@pytest.mark.parametrize("cache,group", [(BF, 1), (BF, 64), (E4M3, 1), (E4M3, 80)])
def test_the_largest_batch(kv, cache, group):
    """65535 sequences of one token and nothing cached: each attends to itself alone, so that the
    result is its own value; then the chain of none is committed.  Every seventh has no token."""
    B, page, dim = 65535, 4, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    gd = Guarded()
    k, v = (gd.empty((B, page, 1, dim), torch.uint8 if cache == E4M3 else BF).view(cache)
            for _ in range(2))
    for p in (k, v):
        p.view(torch.uint8).fill_(0x7f)  # NaN, or (bfloat16) large
    table = torch.randperm(B, generator=g, device="cuda").to(torch.int32).view(B, 1)
    table = torch.cat([table, torch.full((B, 2048), -1, dtype=torch.int32, device="cuda")], 1)
    ones = [torch.ones(1, device="cuda")] * 2 if cache == E4M3 else []
    c = kv.PagedCache(k, v, table, *ones)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    counts = (torch.arange(B, device="cuda") % 7 != 3).to(torch.int32)
    kn, vn = rand(B, 1, 1, dim), rand(B, 1, 1, dim)
    q, out = rand(B, 1, group, dim), gd.empty((B, 1, group, dim), BF, fill=7.0)
    status = gd.empty((B,), torch.int32, fill=0)
    kv.spec_kv_append(c, kn, vn, lens, num_new=counts, status=status)
    kv.spec_kv_attention(c, q, lens, out, kv.attention_workspace(c, B, 1, group), 0.25,
                         num_new=counts, status=status)
    new = gd.empty((B,), torch.int32, fill=-7)
    kv.spec_kv_commit(c, lens, counts - 1, new, status=status)
    gd.check()
    assert not bool(status.any())
    live = counts.bool()
    own = vn.to(cache).to(BF) if cache == E4M3 else vn
    assert torch.equal(out[live], own.expand(-1, -1, group, -1)[live])
    assert bool((out[~live] == 7.0).all()) and torch.equal(new, counts)
    for pool, x in ((k, kn), (v, vn)):
        got = pool.view(torch.uint8)[table[:, 0].long(), 0]
        assert torch.equal(got[live], x.view(B, 1, dim).to(cache).view(torch.uint8)[live])
        assert bool((got[~live] == 0x7f).all())
        assert bool((pool.view(torch.uint8)[:, 1:] == 0x7f).all())


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, E4M3)])
@pytest.mark.parametrize("N,group", [(3, 4), (9, 9), (33, 8)])
def test_keys_and_values_side_by_side(kv, dtype, cache, N, group):
    """Caches that are slices of one pool [layers, pages, 2, heads, page, dim], with a gap behind
    each entry: append, attention and commit of a layer of three, the others untouched."""
    r = Round([200, 7, 64], N, "tree", counts=[N, 2, N], heads=2, group=group, dim=48, dtype=dtype,
              cache=cache, page=16, seed=N, far=N > 3)
    heads, page, dim, pages = 2, 16, 48, r.k.shape[0]
    raw = lambda x: x.view(torch.uint8)
    size = 1 if cache == E4M3 else 2
    pool = torch.full((3, pages, 2, heads, page, (dim + 16) * size), 0x31, dtype=torch.uint8,
                      device="cuda")
    k, v = (pool.view(cache)[:, :, i, :, :, :dim].transpose(2, 3) for i in range(2))
    put = lambda x, y: raw(x).copy_(raw(y).cuda())
    put(pool.view(cache)[1, :, 0, :, :, :dim].transpose(1, 2), r.k)
    put(pool.view(cache)[1, :, 1, :, :, :dim].transpose(1, 2), r.v)
    scales = [] if r.k_scale is None else [x.cuda().expand(3, heads).contiguous()
                                           for x in (r.k_scale, r.v_scale)]
    c = kv.PagedCache(k, v, r.table.cuda(), *scales)
    lens, counts, parents = r.lens.cuda(), r.counts.cuda(), r.parents.cuda()
    # the new tokens' entries once more, from the cache (float8: off by a step where 16 bits are)
    kn = torch.zeros(3, N, heads, dim, dtype=dtype)
    vn = torch.zeros_like(kn)
    for b in range(3):
        for j in range(int(r.counts[b])):
            s = int(r.lens[b]) + j
            at = int(r.table[b, s // page]), s % page
            for new, old, sc in ((kn, r.k, r.k_scale), (vn, r.v, r.v_scale)):
                x = old[at].float()
                new[b, j] = (x if sc is None else x * sc[:, None]).to(dtype)
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    kv.spec_kv_append(c, kn.cuda(), vn.cuda(), lens, num_new=counts, parents=parents, layer=1,
                      status=status)
    out = torch.full_like(r.q, 7.0, device="cuda")
    kv.spec_kv_attention(c, r.q.cuda(), lens, out, kv.attention_workspace(c, 3, N, heads * group),
                         r.scale, parents=parents, num_new=counts, layer=1, status=status)
    now_k, now_v = (raw(x[1]).cpu().contiguous().view(cache) for x in (k, v))
    kv_plain.check_attention(out.cpu(), r.q, now_k, now_v, r.table, r.lens, r.counts, r.parents,
                             r.scale, r.k_scale, r.v_scale, torch.full_like(r.q, 7.0))
    if cache != E4M3:
        assert torch.equal(raw(now_k), raw(r.k)) and torch.equal(raw(now_v), raw(r.v))
    before = pool.clone()
    nodes = torch.full((3, N), -1, dtype=torch.int32)
    nodes[0, 0], nodes[2, 0] = N - 1, 1
    acc = torch.tensor([1, 0, 1], dtype=torch.int32)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    kv.spec_kv_commit(c, lens, acc.cuda(), new, nodes.cuda(), status=status)
    assert status.tolist() == [0] * 3 and torch.equal(new.cpu(), r.lens + acc + 1)
    (sp, ss), (dp, ds) = (kv_plain.slots(r.table[0], page, 200 + i + 1)[-1] for i in (N - 1, 1))
    before[:, dp, :, :, ds, :dim * size] = before[:, sp, :, :, ss, :dim * size]
    assert torch.equal(pool, before)
