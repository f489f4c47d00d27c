"""What a speculative round does to the target's paged key-value cache, measured operator by operator.

append     rotates the round's queries and keys to their positions and writes the keys and values
           of the N drafted tokens (a chain or a tree) into the cache's pages;
attention  every drafted token attends to the cached positions and to its own ancestors among the
           drafted tokens (N = 1: plain decoding of one new token);
commit     after verification, moves the accepted tree nodes' entries up behind the committed ones,
           in every layer, and advances the lengths.

`own` False: plain torch forms of the same operators in 32 bits (angles in 64).  `own` True: the
calls a user makes of the library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "e4m3": 1}


# ---------------------------------------------------------------- the cases

def _attention(name, B, N, form, heads, group, dim, length, page, dtype="bf16", cache="bf16",
               order="slot", ragged=False):
    return dict(name=name, op="attention", B=B, N=N, form=form, heads=heads, group=group, dim=dim,
                length=length, page=page, dtype=dtype, cache=cache, order=order, ragged=ragged)


def _append(name, B, N, form, heads, group, dim, length, page, dtype="bf16", cache="bf16",
            order="slot", ragged=False, rot=0, pairs="half", base=10000.0, factor=1.0,
            original=0):
    return dict(name=name, op="append", B=B, N=N, form=form, heads=heads, group=group, dim=dim,
                length=length, page=page, dtype=dtype, cache=cache, order=order, ragged=ragged,
                rot=rot or dim, pairs=pairs, base=base, factor=factor, original=original)


def _commit(name, B, N, form, heads, dim, length, page, layers, cache="bf16", order="slot"):
    return dict(name=name, op="commit", B=B, N=N, form=form, heads=heads, dim=dim, length=length,
                page=page, layers=layers, cache=cache, order=order)


def listed():
    return [
        # one user's short chat, one new token: the latency of a single decoding step
        _attention("attention one token", 1, 1, "chain", 2, 4, 64, 700, 16),
        # a serving batch that decodes token by token over ragged contexts
        _attention("attention batch decode", 64, 1, "chain", 8, 4, 128, 8000, 16),
        # one long document, eight drafts and the last committed token judged at once
        _attention("attention long chain", 1, 9, "chain", 8, 4, 128, 131071, 64, dtype="f16",
                   cache="f16", order="head"),
        # a batch whose sequences have different numbers of drafts, over an 8-bit cache
        _attention("attention chain 8-bit", 96, 6, "chain", 8, 4, 128, 8191, 32, cache="e4m3",
                   ragged=True),
        # static trees of 16 nodes over ragged contexts: 128 query rows per key head
        _attention("attention tree", 32, 16, "tree", 8, 8, 128, 12345, 32, order="head"),
        # the widest trees the verifier takes: the tensor cores' case
        _attention("attention wide tree", 8, 65, "tree", 8, 8, 128, 32768, 64),
        # one token of one sequence: the latency of a write
        _append("append one token", 1, 1, "chain", 2, 4, 64, 700, 16),
        # trees in a batch, an 8-bit cache, part of the head rotated, stretched frequencies
        _append("append tree 8-bit", 64, 16, "tree", 8, 4, 128, 40000, 16, cache="e4m3",
                ragged=True, rot=64, pairs="interleaved", base=500000.0, factor=8.0,
                original=8192),
        # many long chains at once
        _append("append wide chain", 256, 65, "chain", 8, 8, 128, 4000, 32),
        # one sequence, one layer at a time
        _commit("commit one layer", 1, 9, "tree", 8, 128, 700, 16, 1),
        # a batch of trees, all layers of a model at once
        _commit("commit all layers", 64, 16, "tree", 8, 128, 2000, 16, 32, order="head"),
        # the widest trees, an 8-bit cache
        _commit("commit wide tree", 256, 65, "tree", 8, 128, 2000, 32, 16, cache="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _drawn(rng)
    del c["name"]
    return c


def _drawn(rng):
    op = rng.choice(["attention", "attention", "append", "commit"])
    B = _log(rng, 1, 192)
    form = rng.choice(["chain", "tree"])
    N = rng.choice([1, _log(rng, 2, 12), _log(rng, 5, 65)])
    heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
    dim = rng.choice([64, 80, 96, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    order = rng.choice(["slot", "head"])
    ragged = rng.random() < 0.5
    if op == "attention":
        length = _log(rng, 1, 131072)
        # at most a gigabyte of cache and the work of the widest listed tree
        most = min(1.0e9 / (heads * dim * 2 * BYTES[cache]),
                   5.0e11 / (4.0 * heads * group * dim * N))
        length = max(1, min(length, int(most / B)))
        return _attention(None, B, N, form, heads, group, dim, length, page, dtype, cache, order,
                          ragged)
    if op == "append":
        length = _log(rng, 1, 60000)
        return _append(None, B, N, form, heads, group, dim, length, page, dtype, cache, order,
                       ragged, rot=rng.choice([dim, dim, dim // 2]),
                       pairs=rng.choice(["half", "interleaved"]),
                       base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 8.0]),
                       original=rng.choice([0, 4096, 8192]))
    N = max(N, 2)  # a lone root has no nodes to move
    layers = _log(rng, 1, 32)
    layers = max(1, min(layers, int(1.0e9 / (B * (N + 2 * page) * heads * dim * 2))))
    return _commit(None, B, N, form, heads, dim, _log(rng, 1, 8000), page, layers, cache,
                   order)


# ---------------------------------------------------------------- the inputs

def _lengths(c):
    """Cached positions of each sequence: between half of `length` and all of it, evenly spread."""
    B, L = c["B"], c["length"]
    return [L - (L // 2) * i // max(1, B) for i in range(B)]


def _counts(c):
    """New tokens of each sequence: N, or with `ragged` between 1 and N, evenly spread."""
    B, N = c["B"], c["N"]
    return [1 + (i * 7) % N for i in range(B)] if c.get("ragged") else [N] * B


def _pool(c, pages, gen, layers=None):
    """Keys and values of all pages, logically [layers,] pages, slots, heads, dim."""
    lead = [] if layers is None else [layers]
    inner = [c["page"], c["heads"]] if c["order"] == "slot" else [c["heads"], c["page"]]
    t = torch.empty(lead + [pages] + inner + [c["dim"]], dtype=torch.bfloat16, device=DEV)
    got = []
    for _ in range(2):
        x = t.normal_(generator=gen).to(TYPES[c["cache"]])
        got.append(x.clone() if x is t else x)
    at = len(lead) + 1
    return [x if c["order"] == "slot" else x.transpose(at, at + 1) for x in got]


def _parents(c, gen):
    B, N = c["B"], c["N"]
    j = torch.arange(N, device=DEV)
    if c["form"] == "chain":
        return (j - 1).clamp(min=0).to(torch.int32).expand(B, N).contiguous()
    # each node's parent is one of the nodes before it, the nearer half more often
    u = torch.rand(B, N, generator=gen, device=DEV)
    return (u.sqrt() * j).floor().long().clamp(min=0).minimum((j - 1).clamp(min=0)).to(torch.int32)


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, N, page, heads = c["B"], c["N"], c["page"], c["heads"]
    turn = torch.randperm(B, generator=gen, device=DEV)
    lengths = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)[turn]
    counts = torch.tensor(_counts(c), dtype=torch.int32, device=DEV)[turn]
    width = (c["length"] + N + page - 1) // page
    s = {"case": c, "kv_len": lengths, "parents": _parents(c, gen), "own": {}}
    if c["op"] == "attention":
        pages = B * width
        s["table"] = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).view(B, width)
        s["k"], s["v"] = _pool(c, pages, gen)
    else:
        # the cached positions are a long prefix that all sequences share; the tails are their own
        tail = (N + page - 1) // page + 1
        shared = c["length"] // page + 1
        first = (lengths // page).long()
        at = torch.arange(width, device=DEV)
        mine = (at - first[:, None]).clamp(0, tail - 1) + shared
        mine = mine + tail * torch.arange(B, device=DEV)[:, None]
        s["table"] = torch.where(at < first[:, None], at, mine).to(torch.int32).contiguous()
        s["k"], s["v"] = _pool(c, shared + B * tail, gen, c.get("layers"))
    if c["op"] == "commit":
        # the accepted nodes, in order: each node after the root with probability 0.15
        keep = torch.rand(B, N, generator=gen, device=DEV)
        nodes = torch.where(keep < 0.15, torch.arange(N, device=DEV), N)
        nodes[:, 0] = N
        nodes = nodes.sort(dim=1).values
        s["num_accepted"] = (nodes < N).sum(dim=1).to(torch.int32)
        s["out_nodes"] = torch.where(nodes < N, nodes, -1).to(torch.int32)
        s["kv_len_out"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        return s
    s["num_new"] = counts if c["ragged"] else None
    dt, hq, d = TYPES[c["dtype"]], heads * c["group"], c["dim"]
    if c["cache"] == "e4m3":
        s["k_scale"] = torch.rand(heads, generator=gen, device=DEV) * 0.02 + 0.01
        s["v_scale"] = torch.rand(heads, generator=gen, device=DEV) * 0.02 + 0.01
    if c["op"] == "attention":
        # logits with a spread of about two, as trained heads have them
        f = 2.0 / (s["k_scale"].repeat_interleave(c["group"])[:, None] if "k_scale" in s else 1.0)
        s["q"] = (torch.randn(B, N, hq, d, generator=gen, device=DEV) * f).to(dt)
        s["out"] = torch.zeros(B, N, hq, d, dtype=dt, device=DEV)
    else:
        # one projection's output holds queries, keys and values side by side
        qkv = torch.randn(B, N, hq + 2 * heads, d, generator=gen, device=DEV).to(dt)
        s["q"], s["k_new"], s["v_new"] = qkv.split([hq, heads, heads], dim=2)
        s["q_out"] = torch.zeros(B, N, hq, d, dtype=dt, device=DEV)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"attention": _plain_attention, "append": _plain_append, "commit": _plain_commit}[
        s["case"]["op"]](s)


def _own(s):
    from speculative_decoding_verification_18_gb300 import kvcache as kv
    c, keep = s["case"], s["own"]
    if not keep:  # the handle, the workspace and the rotation table that a program keeps
        keep["cache"] = kv.PagedCache(s["k"], s["v"], s["table"], s.get("k_scale"),
                                      s.get("v_scale"))
        if c["op"] == "attention":
            keep["ws"] = kv.attention_workspace(keep["cache"], c["B"], c["N"],
                                                c["heads"] * c["group"])
        if c["op"] == "append":
            keep["rope"] = kv.Rope(c["rot"], base=c["base"], interleaved=c["pairs"] != "half",
                                   factor=c["factor"], original_length=c["original"],
                                   device=s["q"].device)
    parents = None if c["form"] == "chain" else s["parents"]
    if c["op"] == "attention":
        kv.spec_kv_attention(keep["cache"], s["q"], s["kv_len"], s["out"], keep["ws"],
                             c["dim"] ** -0.5, parents=parents, num_new=s["num_new"])
        return s["out"]
    if c["op"] == "append":
        kv.spec_kv_append(keep["cache"], s["k_new"], s["v_new"], s["kv_len"], q=s["q"],
                          q_out=s["q_out"], rope=keep["rope"], parents=parents,
                          num_new=s["num_new"])
        return s["q_out"], s["k"], s["v"]
    kv.spec_kv_commit(keep["cache"], s["kv_len"], s["num_accepted"], s["kv_len_out"],
                      out_nodes=s["out_nodes"])
    return _as_held(s["k"]), _as_held(s["v"]), s["kv_len_out"]


def _as_held(x):
    """A cache that was only moved about: its bits, so that they are compared exactly."""
    return x.view(torch.uint8 if x.element_size() == 1 else torch.int16)


def _ancestors(parents):
    """[B, N, N]: whether node i is node j or one of its ancestors."""
    N = parents.shape[1]
    step = torch.nn.functional.one_hot(parents.long(), N).float()
    step[:, 0] = 0
    eye = torch.eye(N, device=parents.device)
    return torch.linalg.matrix_power(step + eye, 64) > 0  # a path of at most 64 steps


def _plain_attention(s):
    c = s["case"]
    B, N, H, G, D, page = c["B"], c["N"], c["heads"], c["group"], c["dim"], c["page"]
    counts = s["num_new"] if s["num_new"] is not None else torch.full_like(s["kv_len"], N)
    at = torch.arange(c["length"] + N, device=DEV)
    held = s["table"].long()[:, at // page], at % page
    k = s["k"].view(torch.uint8)[held].view(s["k"].dtype).float() if c["cache"] == "e4m3" else \
        s["k"][held].float()
    v = s["v"].view(torch.uint8)[held].view(s["v"].dtype).float() if c["cache"] == "e4m3" else \
        s["v"][held].float()
    if c["cache"] == "e4m3":
        k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    q = s["q"].float().view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * D ** -0.5
    new = at - s["kv_len"][:, None]  # which drafted token a slot holds; negative: cached before
    kin = _ancestors(s["parents"])
    kin = kin.gather(2, new.clamp(0, N - 1)[:, None, :].expand(B, N, -1))
    seen = (new < 0)[:, None, :] | (kin & (new < counts[:, None])[:, None, :])
    seen = seen.repeat_interleave(G, dim=1)[:, None]
    score = score.masked_fill(~seen, -math.inf)
    e = torch.exp(score - score.amax(dim=-1, keepdim=True))
    e = torch.where(seen, e, 0.0)
    out = torch.matmul(e, v.permute(0, 2, 1, 3)) / e.sum(dim=-1, keepdim=True)
    out = out.view(B, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H * G, D)
    live = torch.arange(N, device=DEV) < counts[:, None]
    return torch.where(live[:, :, None, None], out.to(s["out"].dtype), s["out"])


def _turn_rates(c):
    """Radians per position of each rotated pair, in 64 bits."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
    rate = c["base"] ** (-2.0 * i / c["rot"])
    if not c["original"]:
        return rate / c["factor"]
    # pairs that turn often within the original length keep their rate, slow ones are stretched
    keep = ((c["original"] * rate / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return rate * keep + rate / c["factor"] * (1.0 - keep)


def _plain_append(s):
    c = s["case"]
    B, N, R, page = c["B"], c["N"], c["rot"], c["page"]
    counts = s["num_new"] if s["num_new"] is not None else torch.full_like(s["kv_len"], N)
    depth = _ancestors(s["parents"]).sum(dim=2) - 1
    angle = (s["kv_len"][:, None] + depth)[:, :, None, None].double() * _turn_rates(c)
    cos, sin = angle.cos().float(), angle.sin().float()
    live = torch.arange(N, device=DEV) < counts[:, None]

    def rotated(x):
        x = x.float()
        a, b, rest = (x[..., :R // 2], x[..., R // 2:R], x[..., R:]) if c["pairs"] == "half" else \
            (x[..., 0:R:2], x[..., 1:R:2], x[..., R:])
        pair = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat(pair, dim=-1) if c["pairs"] == "half" else \
            torch.stack(pair, dim=-1).flatten(-2)
        return torch.cat([turned, rest], dim=-1)

    q = torch.where(live[:, :, None, None], rotated(s["q"]).to(s["q_out"].dtype), s["q_out"])
    k, v = rotated(s["k_new"]), s["v_new"].float()
    if c["cache"] == "e4m3":
        k = (k / s["k_scale"][:, None]).clamp(-448.0, 448.0)
        v = (v / s["v_scale"][:, None]).clamp(-448.0, 448.0)
    slot = (s["kv_len"][:, None] + torch.arange(N, device=DEV)).long()
    place = s["table"].long().gather(1, slot // page)[live], (slot % page)[live]
    for pool, x in ((s["k"], k), (s["v"], v)):
        x = x.to(pool.dtype)[live] if pool.element_size() > 1 else \
            x.to(pool.dtype).view(torch.uint8)[live]
        (pool if pool.element_size() > 1 else pool.view(torch.uint8))[place] = x
    return q, s["k"], s["v"]


def _plain_commit(s):
    c = s["case"]
    B, N, page = c["B"], c["N"], c["page"]
    to = torch.arange(1, N + 1, device=DEV).expand(B, N)
    moved = s["out_nodes"] >= 0
    base = s["kv_len"].long()[:, None]
    t = s["table"].long()

    def place(node):
        slot = (base + node.long()).clamp(0, t.shape[1] * page - 1)
        return t.gather(1, slot // page)[moved], (slot % page)[moved]

    src, dst = place(s["out_nodes"].clamp(min=0)), place(to)
    for pool in (_as_held(s["k"]), _as_held(s["v"])):
        pool[:, dst[0], dst[1]] = pool[:, src[0], src[1]]
    s["kv_len_out"].copy_(s["kv_len"] + s["num_accepted"] + 1)
    return _as_held(s["k"]), _as_held(s["v"]), s["kv_len_out"]


# ---------------------------------------------------------------- work and exact values

def work(c):
    B, N, H, D = c["B"], c["N"], c["heads"], c["dim"]
    if c["op"] == "commit":
        # on average 0.15 (N - 1) accepted nodes, nearly all of them at a new place: K and V, read
        # and written, in every layer; the node lists and the lengths
        moved = 0.15 * (N - 1) * B
        return {"bytes": moved * c["layers"] * H * D * BYTES[c["cache"]] * 4 + B * (4 * N + 12.0),
                "flops": 0.0}
    hq, counts = H * c["group"], _counts(c)
    rows = sum(counts)
    if c["op"] == "append":
        e = BYTES[c["dtype"]]
        return {"bytes": rows * D * (2.0 * hq * e + 2 * H * (e + BYTES[c["cache"]])) + 8.0 * B * N,
                "flops": rows * (hq + H) * c["rot"] * 3.0}
    lengths = _lengths(c)
    held = sum(n + m for n, m in zip(lengths, counts))
    seen = sum((n + 1.0) * m for n, m in zip(lengths, counts))
    return {"bytes": held * H * D * 2.0 * BYTES[c["cache"]]
            + rows * hq * D * 2.0 * BYTES[c["dtype"]] + 4.0 * held / c["page"],
            "flops": 4.0 * seen * hq * D}


def exact(c, seed):
    """The same outputs in 64 bits, sequence by sequence, from the definitions."""
    s = prepare(c, seed)
    if c["op"] == "commit":
        return None  # only whole entries move: the plain form's bits are the exact ones
    B, N, H, G, D, page = c["B"], c["N"], c["heads"], c["group"], c["dim"], c["page"]
    lengths, parents = s["kv_len"].tolist(), s["parents"].tolist()
    counts = s["num_new"].tolist() if s["num_new"] is not None else [N] * B
    table = s["table"].tolist()
    above = []  # the path from each node up to the root
    for b in range(B):
        up = [[0]]
        for j in range(1, N):
            up.append([j] + up[parents[b][j]])
        above.append(up)
    if c["op"] == "attention":
        out = torch.zeros(B, N, H * G, D, dtype=torch.float64, device=DEV)
        for b in range(B):
            n, m = lengths[b], counts[b]
            ids = torch.tensor(table[b][:(n + m + page - 1) // page], device=DEV)
            for h in range(H):
                # one head at a time keeps the 64-bit copies small
                k = s["k"][:, :, h].index_select(0, ids) if c["cache"] != "e4m3" else \
                    s["k"].view(torch.uint8)[:, :, h].index_select(0, ids).view(s["k"].dtype)
                v = s["v"][:, :, h].index_select(0, ids) if c["cache"] != "e4m3" else \
                    s["v"].view(torch.uint8)[:, :, h].index_select(0, ids).view(s["v"].dtype)
                k, v = k.double().reshape(-1, D)[:n + m], v.double().reshape(-1, D)[:n + m]
                if c["cache"] == "e4m3":
                    k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
                blind = torch.ones(m, m, dtype=torch.bool)
                for j in range(m):
                    blind[j, above[b][j]] = False
                q = s["q"][b, :m, h * G:(h + 1) * G].double()
                x = torch.einsum("jgd,ld->jgl", q, k) / math.sqrt(D)
                x[:, :, n:].masked_fill_(blind.to(DEV)[:, None, :], -math.inf)
                out[b, :m, h * G:(h + 1) * G] = torch.einsum("jgl,ld->jgd", torch.softmax(x, -1), v)
        return out
    half = c["rot"] // 2
    rates = []
    for i in range(half):
        f = math.pow(c["base"], -i / half)
        turns = c["original"] * f / (2.0 * math.pi)
        share = 0.0 if not c["original"] else min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
        rates.append(share * f + (1.0 - share) * f / c["factor"])
    w = torch.tensor(rates, dtype=torch.float64)
    depth = torch.tensor([[len(p) - 1 for p in up] for up in above], dtype=torch.float64)
    phase = (torch.tensor(lengths, dtype=torch.float64)[:, None] + depth)[..., None] * w
    unit = torch.polar(torch.ones_like(phase), phase).to(DEV)[:, :, None, :]

    def turn(x):
        x = x.double()
        i = torch.arange(half, device=DEV)
        one, two = (i, i + half) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., one], x[..., two]) * unit
        y = x.clone()
        y[..., one], y[..., two] = z.real, z.imag
        return y

    q, k, v = turn(s["q"]), turn(s["k_new"]), s["v_new"].double()
    pools = [s["k"].double(), s["v"].double()]
    if c["cache"] == "e4m3":
        k = (k / s["k_scale"].double()[:, None]).clamp(-448.0, 448.0)
        v = (v / s["v_scale"].double()[:, None]).clamp(-448.0, 448.0)
    for b in range(B):
        q[b, counts[b]:] = 0.0
        for j in range(counts[b]):
            at = lengths[b] + j
            p = table[b][at // page]
            pools[0][p, at % page], pools[1][p, at % page] = k[b, j], v[b, j]
    return q, pools[0], pools[1]
