"""Operators beside the verify step and the paged cache, measured one by one.

window     attention of a round's new tokens over the paged cache through a sliding window, the
           first few slots (sinks) always visible: what layers with a window do, and what a drafter
           does that looks at a part of the target's cache only;
logprobs   log probabilities of given tokens, the entropy and the most probable alternatives of
           every judged logits row;
gradient   of log probabilities and entropy to the logits (training a draft).

`own` False: plain torch forms of the same operators in 32 bits.  `own` True: the calls a user
makes of the library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ---------------------------------------------------------------- the cases

def _window(name, B, N, form, heads, group, dim, length, window, sinks, page, dtype="bf16",
            cache="bf16", order="slot", ragged=False):
    return dict(name=name, op="window", B=B, N=N, form=form, heads=heads, group=group, dim=dim,
                length=length, window=window, sinks=sinks, page=page, dtype=dtype, cache=cache,
                order=order, ragged=ragged)


def _rows(name, op, B, rows, V, dtype, T, given=1, top=0, entropy=True, padded=False, live=1.0):
    """B sequences of `rows` logits rows; `given` tokens asked about in each row; `top`
    alternatives; `padded`: rows lie a multiple of 64 elements apart; `live`: the chance that a
    sequence goes on by one more row (rows behind its last one hold no token)."""
    return dict(name=name, op=op, B=B, rows=rows, V=V, dtype=dtype, T=T, given=given, top=top,
                entropy=entropy, padded=padded, live=live)


def listed():
    return [
        # one user's short window, one new token: the latency of a single step
        _window("window one token", 1, 1, "chain", 2, 4, 64, 700, 256, 4, 16),
        # a serving batch that decodes token by token, long contexts behind a window
        _window("window batch decode", 64, 1, "chain", 8, 4, 128, 32000, 4096, 4, 16),
        # different numbers of drafts, an 8-bit cache, a drafter's short window
        _window("window chain 8-bit", 96, 6, "chain", 8, 4, 128, 100000, 1024, 16, 32,
                cache="e4m3", ragged=True),
        # static trees of 16 nodes: 128 query rows per key head
        _window("window tree", 32, 16, "tree", 8, 8, 128, 60000, 4096, 64, 32, order="head"),
        # the widest trees the verifier takes, halves, one long window
        _window("window wide tree", 8, 65, "tree", 8, 8, 128, 40000, 16384, 4, 64, dtype="f16",
                cache="f16"),
        # what one user is told about a round's tokens: latency, the largest vocabulary
        _rows("logprobs one round", "logprobs", 1, 9, 256000, "bf16", 0.7, top=5, live=0.9),
        # the same for a serving batch after the verdict
        _rows("logprobs batch", "logprobs", 64, 9, 151936, "bf16", 1.0, top=20, live=0.8),
        # 32-bit rows of an odd length, two candidates per row
        _rows("logprobs odd rows", "logprobs", 300, 1, 65537, "f32", 0.8, given=2, top=8),
        # the draft's log probabilities of the target's 32 alternatives, for every position
        _rows("logprobs training", "logprobs", 4, 1024, 128256, "bf16", 1.0, given=32,
              entropy=False),
        # one short sequence
        _rows("gradient one round", "gradient", 1, 9, 32000, "bf16", 1.0, entropy=False),
        # one token per position, prompts left out
        _rows("gradient training", "gradient", 4, 1024, 128256, "bf16", 1.0, live=0.999),
        # 32 alternatives per position and an entropy term, 32-bit rows of an odd length
        _rows("gradient odd rows", "gradient", 8, 128, 65537, "f32", 0.8, given=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _drawn(rng)
    del c["name"]
    return c


def _drawn(rng):
    op = rng.choice(["window", "window", "logprobs", "gradient"])
    if op == "window":
        B = _log(rng, 1, 192)
        N = rng.choice([1, _log(rng, 2, 12), _log(rng, 5, 65)])
        heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
        dim = rng.choice([64, 80, 96, 128, 128])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        cache = rng.choice([dtype, dtype, "e4m3"])
        sinks = rng.choice([0, 1, 4, 4, 64, _log(rng, 1, 300)])
        length, window = _log(rng, 1, 1000000), _log(rng, 1, 32768)
        # at most a gigabyte that is looked at, and the work of the widest listed tree
        most = min(1.0e9 / (heads * dim * 2 * BYTES[cache]),
                   2.5e11 / (4.0 * heads * group * dim * N))
        window = max(1, min(window, int(most / B)))
        return _window(None, B, N, rng.choice(["chain", "tree"]), heads, group, dim, length,
                       window, sinks, rng.choice([16, 32, 64, 128]), dtype, cache,
                       rng.choice(["slot", "head"]), rng.random() < 0.5)
    V = _log(rng, 1000, 262144)
    V = V if rng.random() < 0.5 else (V + 63) // 64 * 64
    dtype = rng.choice(["bf16", "bf16", "f32"])
    # as many bytes of logits as the largest listed case at most
    most = 1.05e9 / (V * BYTES[dtype])
    total = _log(rng, 1, most)
    rows = rng.choice([1, 5, 9, max(1, total // rng.choice([1, 2, 8]))])
    return _rows(None, op, max(1, total // rows), min(rows, total), V, dtype,
                 rng.choice([1.0, 1.0, 0.7, 1.3]), given=rng.choice([1, 1, 2, 8, 32, 64]),
                 top=rng.choice([0, 1, 5, 20, 64]) if op == "logprobs" else 0,
                 entropy=rng.random() < 0.6, padded=rng.random() < 0.5,
                 live=rng.choice([1.0, 0.999, 0.8]))


# ---------------------------------------------------------------- the inputs

def _lengths(c):
    """Cached positions of each sequence: between half of `length` and all of it, evenly spread."""
    B, L = c["B"], c["length"]
    return [L - (L // 2) * i // max(1, B) for i in range(B)]


def _counts(c):
    """New tokens of each sequence: N, or with `ragged` between 1 and N, evenly spread."""
    B, N = c["B"], c["N"]
    return [1 + (i * 7) % N for i in range(B)] if c["ragged"] else [N] * B


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
    return _prepare_window(c, gen) if c["op"] == "window" else _prepare_rows(c, gen)


def _prepare_window(c, gen):
    B, N, page, heads, dim = c["B"], c["N"], c["page"], c["heads"], c["dim"]
    turn = torch.randperm(B, generator=gen, device=DEV)
    lengths = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)[turn]
    s = {"case": c, "kv_len": lengths, "parents": _parents(c, gen), "own": {}}
    s["num_new"] = torch.tensor(_counts(c), dtype=torch.int32, device=DEV)[turn] \
        if c["ragged"] else None
    # pages that have left the window are given back: their table entries are -1
    width = (c["length"] + N + page - 1) // page
    at = torch.arange(width, device=DEV)
    first = (lengths.long() - c["window"] + 1).clamp(min=0) // page
    last = (lengths.long() + N - 1) // page
    first_pages = (c["sinks"] + page - 1) // page
    held = ((at >= first[:, None]) | (at < first_pages)) & (at <= last[:, None])
    pages = int(held.sum())
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    s["table"] = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    s["table"][held] = order
    inner = [page, heads] if c["order"] == "slot" else [heads, page]
    t = torch.empty([pages] + inner + [dim], dtype=torch.bfloat16, device=DEV)
    for name in ("k", "v"):
        x = t.normal_(generator=gen).to(TYPES[c["cache"]])
        x = x.clone() if x is t else x
        s[name] = x if c["order"] == "slot" else x.transpose(1, 2)
    if c["cache"] == "e4m3":
        s["k_scale"] = torch.rand(heads, generator=gen, device=DEV) * 0.02 + 0.01
        s["v_scale"] = torch.rand(heads, generator=gen, device=DEV) * 0.02 + 0.01
    # logits with a spread of about two, as trained heads have them
    f = 2.0 / (s["k_scale"].repeat_interleave(c["group"])[:, None] if "k_scale" in s else 1.0)
    hq, dt = heads * c["group"], TYPES[c["dtype"]]
    s["q"] = (torch.randn(B, N, hq, dim, generator=gen, device=DEV) * f).to(dt)
    s["out"] = torch.zeros(B, N, hq, dim, dtype=dt, device=DEV)
    return s


def _prepare_rows(c, gen):
    B, n, V, K = c["B"], c["rows"], c["V"], c["given"]
    pitch = (V + 63) // 64 * 64 if c["padded"] else V
    # Zipf-like rows: -1.1 ln(rank) + noise under a permutation of the vocabulary
    base = torch.empty(V, device=DEV)
    base[torch.randperm(V, generator=gen, device=DEV)] = \
        -1.1 * torch.arange(1, V + 1, device=DEV, dtype=torch.float32).log()
    held = torch.empty(B, n, pitch, dtype=TYPES[c["dtype"]], device=DEV)
    logits = held[:, :, :V]
    tokens = torch.empty(B * n, K, dtype=torch.int32, device=DEV)
    flat = held.view(B * n, pitch)[:, :V]
    some = max(1, (1 << 25) // V)
    for i in range(0, B * n, some):
        x = base + torch.randn(min(some, B * n - i), V, generator=gen, device=DEV)
        flat[i:i + some] = x.to(held.dtype)
        # given tokens: what another, similar distribution has on top
        x = x.mul_(0.8).add_(torch.randn(x.shape, generator=gen, device=DEV))
        tokens[i:i + some] = x.topk(K, dim=1).indices.to(torch.int32)
    # rows behind a sequence's last one hold no token
    u = torch.rand(B, n, generator=gen, device=DEV)
    u[:, 0] = 0.0
    gone = (u > c["live"]).cumsum(dim=1) > 0
    tokens = torch.where(gone[:, :, None], -1, tokens.view(B, n, K)).contiguous()
    s = {"case": c, "logits": logits, "tokens": tokens, "own": {}}
    f32 = lambda *shape: torch.zeros(*shape, dtype=torch.float32, device=DEV)
    if c["op"] == "logprobs":
        s["logprobs"], s["normalizer"] = f32(B, n, K), f32(B, n, 2)
        s["entropy"] = f32(B, n) if c["entropy"] else None
        s["top_tokens"] = s["top_logprobs"] = None
        if c["top"]:
            s["top_tokens"] = torch.zeros(B, n, c["top"], dtype=torch.int32, device=DEV)
            s["top_logprobs"] = f32(B, n, c["top"])
        return s
    # what the pass forward has left, and the gradients that come back to it
    s["normalizer"], s["entropy"] = f32(B, n, 2), f32(B, n)
    z, h = s["normalizer"].view(B * n, 2), s["entropy"].view(B * n)
    for i in range(0, B * n, some):
        x = flat[i:i + some].double()
        m = x.amax(dim=1)
        x = (x - m[:, None]) / c["T"]
        e = x.exp()
        total = e.sum(dim=1)
        z[i:i + some, 0], z[i:i + some, 1] = m.float(), total.log().float()
        h[i:i + some] = (total.log() - (e * x).sum(dim=1) / total).float()
    s["grad_logprobs"] = torch.rand(B, n, K, generator=gen, device=DEV) * (-2.0 / K)
    s["grad_entropy"] = torch.randn(B, n, generator=gen, device=DEV) * 0.1 if c["entropy"] else None
    s["grad_logits"] = torch.zeros(B, n, V, dtype=held.dtype, device=DEV)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"window": _plain_window, "logprobs": _plain_logprobs,
            "gradient": _plain_gradient}[s["case"]["op"]](s)


def _own(s):
    c, keep = s["case"], s["own"]
    if c["op"] == "window":
        from speculative_decoding_verification_18_gb300 import kvcache as kv
        if not keep:  # the handle and the workspace that a program keeps
            keep["cache"] = kv.PagedCache(s["k"], s["v"], s["table"], s.get("k_scale"),
                                          s.get("v_scale"))
            keep["ws"] = kv.attention_workspace(keep["cache"], c["B"], c["N"],
                                                c["heads"] * c["group"])
        kv.spec_kv_attention_window(keep["cache"], s["q"], s["kv_len"], s["out"], keep["ws"],
                                    c["dim"] ** -0.5, c["window"], c["sinks"],
                                    parents=None if c["form"] == "chain" else s["parents"],
                                    num_new=s["num_new"])
        return s["out"]
    from speculative_decoding_verification_18_gb300 import logprobs as lp
    if c["op"] == "logprobs":
        if not keep:
            keep["ws"] = lp.logprobs_workspace(s["logits"], c["given"], c["top"])
        lp.spec_logprobs(s["logits"], s["tokens"], s["logprobs"], keep["ws"], T=c["T"],
                         entropy=s["entropy"], normalizer=s["normalizer"],
                         top_tokens=s["top_tokens"], top_logprobs=s["top_logprobs"])
        return _told(s)
    lp.spec_logprobs_grad(s["logits"], s["tokens"], s["normalizer"], s["grad_logprobs"],
                          s["grad_logits"], T=c["T"],
                          entropy=s["entropy"] if c["entropy"] else None,
                          grad_entropy=s["grad_entropy"])
    return s["grad_logits"]


def _told(s):
    return {n: s[n] for n in ("logprobs", "normalizer", "entropy", "top_tokens", "top_logprobs")
            if s[n] is not None}


def _kin(parents):
    """[B, N, N] whether node i is node j or one of its ancestors, and [B, N] the depths."""
    N = parents.shape[1]
    step = torch.nn.functional.one_hot(parents.long(), N).float()
    step[:, 0] = 0
    eye = torch.eye(N, device=parents.device)
    kin = torch.linalg.matrix_power(step + eye, 64) > 0  # a path of at most 64 steps
    return kin, kin.sum(dim=2) - 1


def _plain_window(s):
    c = s["case"]
    B, N, H, G, D, page = c["B"], c["N"], c["heads"], c["group"], c["dim"], c["page"]
    W, first = c["window"], c["sinks"]
    n = s["kv_len"].long()[:, None]
    counts = s["num_new"] if s["num_new"] is not None else torch.full_like(s["kv_len"], N)
    # the slots that any node of a sequence sees: the first ones, the root's window, the new ones
    low = (n - W + 1).clamp(min=0)
    most = min(W - 1, c["length"]) + N
    slot = low + torch.arange(most, device=DEV)
    there = slot < n + counts[:, None]
    if first:
        a = torch.arange(first, device=DEV).expand(B, first)
        slot, there = torch.cat([a, slot], dim=1), torch.cat([a < low, there], dim=1)
    slot = torch.where(there, slot, n)
    ids = s["table"].long().gather(1, slot // page)
    held = ids, slot % page
    bits = lambda x: x.view(torch.uint8)[held].view(x.dtype) if x.element_size() == 1 else x[held]
    k, v = bits(s["k"]).float(), bits(s["v"]).float()
    if c["cache"] == "e4m3":
        k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    q = s["q"].float().view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * D ** -0.5
    kin, depth = _kin(s["parents"])
    new = slot - n  # which new token a slot holds; negative: cached before
    node = new.clamp(0, N - 1)
    mine = kin.gather(2, node[:, None, :].expand(B, N, -1))
    place = torch.where(new < 0, slot, n + depth.gather(1, node))  # the entry's position
    near = place[:, None, :] > (n + depth)[:, :, None] - W
    seen = there[:, None, :] & (near | (place < first)[:, None, :]) & ((new < 0)[:, None, :] | mine)
    seen = seen.repeat_interleave(G, dim=1)[:, None]
    score = score.masked_fill(~seen, -math.inf)
    e = torch.exp(score - score.amax(dim=-1, keepdim=True))
    e = torch.where(seen, e, 0.0)
    out = torch.matmul(e, v.permute(0, 2, 1, 3)) / e.sum(dim=-1, keepdim=True)
    out = out.view(B, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H * G, D)
    live = torch.arange(N, device=DEV) < counts[:, None]
    return torch.where(live[:, :, None, None], out.to(s["out"].dtype), s["out"])


def _plain_logprobs(s):
    c = s["case"]
    x, live = s["logits"].float(), s["tokens"] >= 0
    some = live.any(dim=-1)
    m = x.amax(dim=-1)
    a = (x - m[..., None]) / c["T"]
    e = torch.exp(a)
    total = e.sum(dim=-1)
    log_total = torch.log(total)
    told = a.gather(-1, s["tokens"].long().clamp(min=0)) - log_total[..., None]
    r = {"logprobs": torch.where(live, told, s["logprobs"]),
         "normalizer": torch.where(some[..., None], torch.stack([m, log_total], dim=-1),
                                   s["normalizer"])}
    if c["entropy"]:
        r["entropy"] = torch.where(some, log_total - (e * a).sum(dim=-1) / total, s["entropy"])
    if c["top"]:
        del e
        # a whole number per element that orders by value, then by the lower index
        V = c["V"]
        key = (x + 0.0).view(torch.int32)
        key = torch.where(key < 0, key ^ 0x7fffffff, key).long()
        key = key * V + (V - 1 - torch.arange(V, device=DEV))
        top = key.topk(c["top"], dim=-1).indices
        r["top_tokens"] = torch.where(some[..., None], top.to(torch.int32), s["top_tokens"])
        r["top_logprobs"] = torch.where(some[..., None],
                                        a.gather(-1, top) - log_total[..., None],
                                        s["top_logprobs"])
    return r


def _plain_gradient(s):
    c = s["case"]
    live = s["tokens"] >= 0
    g = torch.where(live, s["grad_logprobs"], 0.0)
    log_p = (s["logits"].float() - s["normalizer"][..., :1]) / c["T"] - s["normalizer"][..., 1:]
    p = torch.exp(log_p)
    d = p * -g.sum(dim=-1, keepdim=True)
    if c["entropy"]:
        gh = torch.where(live.any(dim=-1), s["grad_entropy"], 0.0)
        d -= gh[..., None] * p * (log_p + s["entropy"][..., None])
    d.scatter_add_(-1, s["tokens"].long().clamp(min=0), g)
    return (d / c["T"]).to(s["grad_logits"].dtype)


# ---------------------------------------------------------------- work and exact values

def _rows_alive(c):
    """Rows that hold tokens: each sequence's first, and one more with chance `live` each time."""
    q = c["live"]
    return c["B"] * (c["rows"] if q >= 1.0 else (1.0 - q ** c["rows"]) / (1.0 - q))


def work(c):
    if c["op"] != "window":
        e, K = BYTES[c["dtype"]], c["given"]
        alive, rows = _rows_alive(c), c["B"] * c["rows"]
        if c["op"] == "logprobs":
            told = 4.0 * K + 8 + 4 * c["entropy"] + 8 * c["top"]
            # subtract, scale, exp, add, largest; the entropy's product and sum
            return {"bytes": alive * (c["V"] * e + told) + rows * K * 4.0,
                    "flops": alive * c["V"] * (7.0 if c["entropy"] else 5.0)}
        back = 4.0 * K + 8 + 8 * c["entropy"]
        return {"bytes": alive * (c["V"] * e + back) + rows * (c["V"] * e + 4.0 * K),
                "flops": alive * c["V"] * (7.0 if c["entropy"] else 4.0)}
    B, H, D, W = c["B"], c["heads"], c["dim"], c["window"]
    hq, counts = H * c["group"], _counts(c)
    held = seen = 0.0
    for n, m in zip(_lengths(c), counts):
        low = max(0, n - W + 1)
        slots = n - low + min(c["sinks"], low)
        held += slots + m
        seen += (slots + 1.0) * m
    return {"bytes": held * H * D * 2.0 * BYTES[c["cache"]]
            + sum(counts) * hq * D * 2.0 * BYTES[c["dtype"]] + 4.0 * held / c["page"],
            "flops": 4.0 * seen * hq * D}


def exact(c, seed):
    """The same outputs in 64 bits, from the definitions."""
    s = prepare(c, seed)
    return _exact_window(c, s) if c["op"] == "window" else _exact_rows(c, s)


def _exact_window(c, s):
    B, N, H, G, D, page = c["B"], c["N"], c["heads"], c["group"], c["dim"], c["page"]
    lengths, parents = s["kv_len"].tolist(), s["parents"].tolist()
    counts = s["num_new"].tolist() if s["num_new"] is not None else [N] * B
    out = torch.zeros(B, N, H * G, D, dtype=torch.float64, device=DEV)
    for b in range(B):
        n, m = lengths[b], counts[b]
        above = [[0]]  # the path from each node up to the root
        for j in range(1, m):
            above.append([j] + above[parents[b][j]])
        low = max(0, n - c["window"] + 1)
        slots = list(range(min(c["sinks"], low))) + list(range(low, n + m))
        see = torch.zeros(m, len(slots), dtype=torch.bool)
        old = torch.tensor([x for x in slots if x < n], dtype=torch.long)
        for j in range(m):
            place = n + len(above[j]) - 1
            see[j, :len(old)] = (old < c["sinks"]) | (old >= place - c["window"] + 1)
            for i in above[j]:
                at = n + len(above[i]) - 1
                see[j, len(old) + i] = at < c["sinks"] or place - at < c["window"]
        see = see.to(DEV)[:, None, :]
        slots = torch.tensor(slots, device=DEV)
        ids, at = s["table"][b].long()[slots // page], slots % page
        for h in range(H):
            k, v = ((x.view(torch.uint8)[ids, at, h].view(x.dtype) if c["cache"] == "e4m3" else
                     x[ids, at, h]).double() for x in (s["k"], s["v"]))
            if c["cache"] == "e4m3":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            q = s["q"][b, :m, h * G:(h + 1) * G].double()
            x = torch.einsum("jgd,ld->jgl", q, k) / math.sqrt(D)
            x = torch.softmax(torch.where(see, x, -math.inf), dim=-1)
            out[b, :m, h * G:(h + 1) * G] = torch.einsum("jgl,ld->jgd", x, v)
    return out


def _exact_rows(c, s):
    B, n, V, T = c["B"], c["rows"], c["V"], c["T"]
    full = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=DEV)
    if c["op"] == "gradient":
        r = {"d": full(B * n, V)}
    else:
        r = {"logprobs": full(B * n, c["given"]), "normalizer": full(B * n, 2)}
        if c["entropy"]:
            r["entropy"] = full(B * n)
        if c["top"]:
            r["top_tokens"] = torch.zeros(B * n, c["top"], dtype=torch.int32, device=DEV)
            r["top_logprobs"] = full(B * n, c["top"])
    tokens = s["tokens"].view(B * n, -1).long()
    rows = (tokens >= 0).any(dim=1).nonzero().flatten()
    some = max(1, (1 << 25) // V)
    for i in range(0, len(rows), some):
        at = rows[i:i + some]
        l = s["logits"].reshape(B * n, V)[at] if B * n * V < 1 << 28 else \
            torch.stack([s["logits"][int(j) // n, int(j) % n] for j in at])
        y = torch.log_softmax(l.double() / T, dim=1)
        x = tokens[at]
        if c["op"] == "gradient":
            g = torch.where(x >= 0, s["grad_logprobs"].view(B * n, -1)[at].double(), 0.0)
            p = y.exp()
            d = torch.zeros_like(p).scatter_add_(1, x.clamp(min=0), g) - p * g.sum(1, keepdim=True)
            if c["entropy"]:
                h = -(p * y).sum(dim=1, keepdim=True)
                d -= s["grad_entropy"].view(-1, 1)[at].double() * p * (y + h)
            r["d"][at] = d / T
            continue
        r["logprobs"][at] = y.gather(1, x)
        best = l.double().amax(dim=1)
        r["normalizer"][at] = torch.stack([best, torch.logsumexp(l.double() / T, 1) - best / T], 1)
        if c["entropy"]:
            r["entropy"][at] = -(y.exp() * y).sum(dim=1)
        if c["top"]:
            pick = l.float().sort(dim=1, descending=True, stable=True).indices[:, :c["top"]]
            r["top_tokens"][at] = pick.to(torch.int32)
            r["top_logprobs"][at] = y.gather(1, pick)
    if c["op"] == "gradient":
        return r["d"].view(B, n, V)
    return {k: x.view(B, n) if x.dim() == 1 else x.view(B, n, -1) for k, x in r.items()}
