"""The paged cache calls without a GPU: declared symbols, argument errors (returned before any
launch), the binding's checks, and the rotation's rates."""
import ctypes
import math
import os
import re

import pytest
import torch

import kv_plain
from conftest import ROOT


@pytest.fixture(scope="module")
def kv():
    from speculative_decoding_verification_18_gb300 import build, kvcache
    build.build()
    lib = kvcache.load()
    P, I, F, Z, L = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64)
    lib.spec_kv_append.argtypes = [P, P, P, P, P, P, P, I, P, P, P, I, I, I, P, P, P]
    lib.spec_kv_attention.argtypes = [P, P, P, I, P, P, P, F, I, I, I, P, P, Z, P, P]
    lib.spec_kv_commit.argtypes = [P, I, L, P, P, P, I, I, P, P, P]
    return kvcache


class Strides(ctypes.Structure):
    """sv_strides."""
    _fields_ = [("batch", ctypes.c_int64), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


P = 4096  # a 16-byte-aligned fake address: never dereferenced on these paths


def cache_struct(kv, **kw):
    from speculative_decoding_verification_18_gb300 import specverify as sv
    a = dict(k=P, v=P, table=P, k_scale=None, v_scale=None, page_stride=16 * 2 * 64,
             slot_stride=2 * 64, head_stride=64, num_pages=10, page_size=16, table_width=5,
             heads=2, dim=64, dtype=sv.SV_BF16)
    a.update(kw)
    return kv._Cache(*a.values())


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1), (dict(k=P + 8), 1),
              (dict(dtype=1), 1), (dict(dtype=9), 1), (dict(k_scale=P), 1),
              (dict(dtype=3), 1), (dict(dtype=3, k_scale=P), 1), (dict(num_pages=0), 1),
              (dict(page_size=0), 1), (dict(page_size=12), 3), (dict(dim=72), 3),
              (dict(dim=144, head_stride=144, slot_stride=288), 3), (dict(dim=0), 1),
              (dict(head_stride=68), 1), (dict(head_stride=32), 1), (dict(slot_stride=-64), 1),
              (dict(heads=0), 1), (dict(page_size=1 << 20, table_width=1 << 11), 3),
              (dict(table_width=0), 1)]


def test_every_declared_symbol_is_exported(kv):
    text = open(os.path.join(ROOT, "include", "specverify_kv.h")).read()
    names = set(re.findall(r"\b(spec_kv_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(kv.EXPORTS)
    for n in names:
        assert hasattr(kv.load(), n)


def test_workspace_size(kv):
    size = kv.spec_kv_attention_workspace_size
    assert size(1, 1, 8, 2, 64) > 0 and size(0, 65, 32, 32, 128) > 0
    for bad in ((-1, 1, 8, 2, 64), (1, 0, 8, 2, 64), (1, 66, 8, 2, 64), (1, 1, 9, 2, 64),
                (1, 1, 8, 0, 64), (1, 1, 8, 2, 72), (1, 1, 8, 2, 144), (65536, 1, 8, 2, 64),
                (1, 1, 1025, 1, 64), (1, 1, 0, 2, 64)):
        assert size(*bad) == 0, bad


def test_append_argument_errors(kv):
    from speculative_decoding_verification_18_gb300 import specverify as sv
    st = Strides(64 * 6, 64 * 6, 64)

    def call(cache=None, rope=None, q=P, qs=st, k=P, v=P, ks=st, dtype=sv.SV_BF16, kv_len=P,
             num_new=None, parents=None, B=2, N=3, hq=4, out=2 * P, status=None):
        c = cache or cache_struct(kv)
        ref = lambda x: None if x is None else ctypes.byref(x)
        return kv.load().spec_kv_append(ref(c), ref(rope), q, ref(qs), k, v, ref(ks), dtype, kv_len,
                                        num_new, parents, B, N, hq, out, status, None)

    for bad, code in BAD_CACHES:
        assert call(cache=cache_struct(kv, **bad)) == code, bad
    for bad, code in ((dict(k=None), 1), (dict(v=None), 1), (dict(kv_len=None), 1),
                      (dict(out=None), 1), (dict(qs=None), 1), (dict(ks=None), 1),
                      (dict(dtype=1), 1), (dict(dtype=3), 1), (dict(dtype=2), 1), (dict(B=-1), 1),
                      (dict(B=65536), 3), (dict(N=0), 1), (dict(N=66), 3), (dict(hq=3), 1),
                      (dict(hq=0), 1), (dict(hq=1026), 3), (dict(k=P + 2), 1), (dict(q=P + 2), 1),
                      (dict(out=P + 2), 1), (dict(kv_len=P + 4), 1), (dict(num_new=P + 4), 1),
                      (dict(parents=P + 4), 1), (dict(status=P + 4), 1), (dict(out=P), 1),
                      (dict(qs=Strides(64, 64, 4)), 1), (dict(ks=Strides(64, -64, 64)), 1),
                      (dict(rope=kv._Rope(None, 64, 0, 1.0)), 1),
                      (dict(rope=kv._Rope(P, 63, 0, 1.0)), 1),
                      (dict(rope=kv._Rope(P, 66, 0, 1.0)), 1),
                      (dict(rope=kv._Rope(P, 0, 0, 1.0)), 1),
                      (dict(rope=kv._Rope(P, 64, 2, 1.0)), 1),
                      (dict(rope=kv._Rope(P, 64, 0, math.nan)), 1)):
        assert call(**bad) == code, bad
    assert kv.load().spec_kv_append(None, None, P, ctypes.byref(st), P, P, ctypes.byref(st), 0, P,
                                    None, None, 2, 3, 4, P, None, None) == 1
    assert call(B=0) == 0 and call(B=0, cache=cache_struct(kv, table=None)) == 0  # no launch


def test_attention_argument_errors(kv):
    from speculative_decoding_verification_18_gb300 import specverify as sv
    st = Strides(64 * 12, 64 * 4, 64)
    need = kv.spec_kv_attention_workspace_size(2, 3, 4, 2, 64)

    def call(cache=None, q=P, qs=st, dtype=sv.SV_BF16, kv_len=P, num_new=None, parents=None,
             scale=0.1, B=2, N=3, hq=4, out=P, ws=P, wsb=need, status=None):
        ref = lambda x: None if x is None else ctypes.byref(x)
        return kv.load().spec_kv_attention(ref(cache or cache_struct(kv)), q, ref(qs), dtype,
                                           kv_len, num_new, parents, scale, B, N, hq, out, ws, wsb,
                                           status, None)

    for bad, code in BAD_CACHES:
        assert call(cache=cache_struct(kv, **bad)) == code, bad
    for bad, code in ((dict(q=None), 1), (dict(out=None), 1), (dict(qs=None), 1),
                      (dict(kv_len=None), 1), (dict(dtype=1), 1), (dict(dtype=3), 1),
                      (dict(dtype=2), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
                      (dict(B=-1), 1), (dict(N=0), 1), (dict(N=66), 3), (dict(hq=5), 1),
                      (dict(q=P + 8), 1), (dict(out=P + 8), 1), (dict(ws=P + 8), 1),
                      (dict(ws=None), 2), (dict(wsb=need - 1), 2), (dict(num_new=P + 4), 1),
                      (dict(status=P + 4), 1), (dict(parents=P + 4), 1),
                      (dict(qs=Strides(64, 64, 4)), 1)):
        assert call(**bad) == code, bad
    assert call(B=0) == 0 and call(B=0, cache=cache_struct(kv, table=None)) == 0


def test_commit_argument_errors(kv):
    def call(cache=None, layers=2, stride=16 * 2 * 64 * 10, kv_len=P, nodes=P, acc=P, B=2, N=3,
             out=2 * P, status=None):
        return kv.load().spec_kv_commit(ctypes.byref(cache or cache_struct(kv)), layers, stride,
                                        kv_len, nodes, acc, B, N, out, status, None)

    for bad, code in BAD_CACHES:
        if "k_scale" in bad or "dtype" in bad and bad["dtype"] == 3:
            continue  # scales are not looked at
        assert call(cache=cache_struct(kv, **bad)) == code, bad
    for bad, code in ((dict(layers=0), 1), (dict(layers=40000), 3), (dict(stride=8), 1),
                      (dict(stride=65), 1), (dict(kv_len=None), 1), (dict(acc=None), 1),
                      (dict(out=None), 1), (dict(out=P), 1), (dict(out=P + 16, B=9), 1),
                      (dict(acc=2 * P, out=2 * P + 16, B=9), 1),
                      (dict(B=-1), 1), (dict(N=0), 1), (dict(N=66), 3), (dict(nodes=P + 4), 1), (dict(acc=P + 4), 1),
                      (dict(out=P + 4), 1), (dict(status=P + 4), 1)):
        assert call(**bad) == code, bad
    assert call(B=0) == 0 and call(B=0, cache=cache_struct(kv, table=None)) == 0


def test_logits_calls_refuse_the_cache_types(kv):
    from speculative_decoding_verification_18_gb300 import specverify as sv
    for t in (kv.SV_F16, kv.SV_E4M3):
        assert sv.spec_verify_workspace_size(1, 4, 10, t) == 0
        assert sv.load().spec_verify_greedy(P, t, P, 2, 3, 100, P, P, P, 1 << 20, None) == 1


def turns_of(kv, rot, **kw):
    a = dict(base=10000.0, factor=1.0, original=0.0, low=1.0, high=32.0)
    a.update(kw)
    out = (ctypes.c_uint64 * (rot // 2))()
    st = kv.load().spec_kv_rope_turns(rot, a["base"], a["factor"], a["original"], a["low"],
                                      a["high"], out)
    return st, list(out)


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0, factor=8.0),
                                dict(base=500000.0, factor=8.0, original=8192),
                                dict(factor=4.0, original=4096, low=1.0, high=4.0)])
def test_rope_turns(kv, rot, kw):
    """Rates as 64-bit fractions of a turn: off by the double's own roundings only (a few 2^-53
    of the rate: pow, products) and half a step of 2^-62."""
    st, got = turns_of(kv, rot, **kw)
    assert st == 0
    want = kv_plain.rates(rot, **dict(dict(base=10000.0), **kw)) / (2 * math.pi)
    for g, w in zip(got, want.tolist()):
        assert abs(g / 2.0 ** 64 - w) <= 16 * 2.0 ** -53 * w + 2.0 ** -62


def test_rope_turns_refusals(kv):
    for rot in (0, 1, 3, 130):
        assert kv.load().spec_kv_rope_turns(rot, 1e4, 1.0, 0.0, 1.0, 32.0,
                                            (ctypes.c_uint64 * 99)()) == 1
    for kw in (dict(base=1.0), dict(base=math.inf), dict(factor=0.5), dict(factor=math.nan),
               dict(original=math.nan), dict(original=10.0, low=4.0, high=4.0),
               dict(high=math.inf)):
        assert turns_of(kv, 64, **kw)[0] == 1, kw
    assert kv.load().spec_kv_rope_turns(64, 1e4, 1.0, 0.0, 1.0, 32.0, None) == 1


def test_binding_refuses_what_it_cannot_pass_on(kv, monkeypatch):
    """Types, shapes and layouts, before the library is called.  CPU tensors stand in for CUDA
    ones where a check behind the device's is meant."""
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kv.PagedCache(k, k.clone(), t)
    monkeypatch.setattr(kv, "_on_device", lambda t, name: None)
    with pytest.raises(TypeError):
        kv.PagedCache(k.float(), k.float(), t)
    with pytest.raises(TypeError):
        kv.PagedCache(k, k.half(), t)
    with pytest.raises(ValueError, match="shape"):
        kv.PagedCache(k, k[:3], t)
    with pytest.raises(ValueError, match="strides"):
        kv.PagedCache(k, torch.zeros(4, 2, 16, 64, dtype=k.dtype).transpose(1, 2), t)
    with pytest.raises(ValueError, match="contiguous"):
        kv.PagedCache(k.transpose(2, 3), k.transpose(2, 3), t)
    with pytest.raises(TypeError):
        kv.PagedCache(k, k, t.long())
    with pytest.raises(ValueError):
        kv.PagedCache(k, k, t[0])
    with pytest.raises(ValueError, match="k_scale"):
        kv.PagedCache(k, k, t, torch.ones(2), torch.ones(2))
    with pytest.raises(ValueError, match="together"):
        kv.PagedCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), t, torch.ones(2))
    with pytest.raises(ValueError, match="needs k_scale"):
        kv.PagedCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), t).layer(0)
    c = kv.PagedCache(k, k.clone(), t)
    with pytest.raises(ValueError, match="layer"):
        c.layer(1)
    n = torch.zeros(3, dtype=torch.int32)
    new = torch.zeros(3, 5, 2, 64, dtype=k.dtype)
    q = torch.zeros(3, 5, 8, 64, dtype=k.dtype)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: kv.spec_kv_append(c, new[:2], new[:2], n[:2]),            # table rows
                 lambda: kv.spec_kv_append(c, new[..., :32], new[..., :32], n),    # dim
                 lambda: kv.spec_kv_append(c, new, new[:, :4], n),
                 lambda: kv.spec_kv_append(c, new, new, n[:2]),
                 lambda: kv.spec_kv_append(c, new, new, n, q=q),                   # no q_out
                 lambda: kv.spec_kv_append(c, new, new, n, q=q, q_out=q[:, :4]),
                 lambda: kv.spec_kv_append(c, new, new, n, parents=n),
                 lambda: kv.spec_kv_append(c, new, new.transpose(0, 1).contiguous().transpose(0, 1),
                                           n),
                 lambda: kv.spec_kv_attention(c, q[0], n, q, ws, 1.0),
                 lambda: kv.spec_kv_attention(c, q, n, q[:, ::2], ws, 1.0),
                 lambda: kv.spec_kv_attention(c, q, n, q.transpose(1, 2), ws, 1.0),
                 lambda: kv.spec_kv_commit(c, n, n[:2], n.clone()),
                 lambda: kv.spec_kv_commit(c, n[:2], n[:2], n[:2].clone())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: kv.spec_kv_append(c, new.float(), new.float(), n),
                 lambda: kv.spec_kv_append(c, new, new.half(), n),
                 lambda: kv.spec_kv_append(c, new, new, n.long()),
                 lambda: kv.spec_kv_attention(c, q.float(), n, q, ws, 1.0),
                 lambda: kv.spec_kv_attention(c, q, n, q.half(), ws, 1.0),
                 lambda: kv.spec_kv_attention(c, q, n, q, ws.int(), 1.0),
                 lambda: kv.spec_kv_commit(c, n, n, n.clone(), status=n.float())):
        with pytest.raises(TypeError):
            call()
