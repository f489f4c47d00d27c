"""Attention through a window without a GPU: argument errors (returned before any launch), the
binding's checks, and the plain implementation's own visible slots."""
import ctypes

import pytest
import torch

import kv_plain
import window_plain
from test_kv_cpu import BAD_CACHES, P, Strides, cache_struct, kv  # noqa: F401


def test_argument_errors(kv):  # noqa: F811
    from speculative_decoding_verification_18_gb300 import specverify as sv
    V, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    f = kv.load().spec_kv_attention_window
    f.argtypes = [V, V, V, I, V, V, V, F, I, I, I, I, I, V, V, Z, V, V]
    st = Strides(64 * 12, 64 * 4, 64)
    need = kv.spec_kv_attention_workspace_size(2, 3, 4, 2, 64)

    def call(cache=None, q=P, qs=st, dtype=sv.SV_BF16, kv_len=P, num_new=None, parents=None,
             scale=0.1, window=5, sinks=0, B=2, N=3, hq=4, out=P, ws=P, wsb=need, status=None):
        ref = lambda x: None if x is None else ctypes.byref(x)
        return f(ref(cache or cache_struct(kv)), q, ref(qs), dtype, kv_len, num_new, parents, scale,
                 window, sinks, B, N, hq, out, ws, wsb, status, None)

    for bad, code in BAD_CACHES:
        assert call(cache=cache_struct(kv, **bad)) == code, bad
    for bad, code in ((dict(window=0), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
                      (dict(window=-2 ** 31), 1), (dict(q=None), 1), (dict(out=None), 1),
                      (dict(qs=None), 1), (dict(kv_len=None), 1), (dict(dtype=1), 1),
                      (dict(scale=float("nan")), 1), (dict(B=-1), 1), (dict(N=0), 1),
                      (dict(N=66), 3), (dict(hq=5), 1), (dict(q=P + 8), 1), (dict(ws=None), 2),
                      (dict(wsb=need - 1), 2), (dict(num_new=P + 4), 1), (dict(parents=P + 4), 1)):
        assert call(**bad) == code, bad
    assert call(B=0) == 0 and call(B=0, window=2 ** 31 - 1, sinks=2 ** 31 - 1) == 0


def test_binding_refusals(kv, monkeypatch):  # noqa: F811
    monkeypatch.setattr(kv, "_on_device", lambda t, name: None)
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    c = kv.PagedCache(k, k.clone(), torch.zeros(3, 2, dtype=torch.int32))
    n, q = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 5, 8, 64, dtype=k.dtype)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for q2, out, window, sinks in ((q[0], q, 4, 0), (q, q[:, ::2], 4, 0), (q[:2], q[:2], 4, 0),
                                   (q, q, 1 << 31, 0), (q, q, 4, 1 << 40)):
        with pytest.raises(ValueError):
            kv.spec_kv_attention_window(c, q2, n, out, ws, 1.0, window, sinks)
    for q2, window in ((q.float(), 4), (q, 4.5), (q, None), (q, "4")):
        with pytest.raises(TypeError):
            kv.spec_kv_attention_window(c, q2, n, q, ws, 1.0, window)
    with pytest.raises(ValueError, match="CUDA"):
        kv.spec_kv_attention_window(c, q, n, q.clone(), ws, 1.0, 4, 1)


def test_visible_slots():
    """By hand: a window of three behind two first slots, a chain and a tree of two branches."""
    chain = kv_plain.paths(None, 4)
    assert window_plain.seen(10, 4, chain, 3, 2) == [[0, 1, 8, 9, 10], [0, 1, 9, 10, 11],
                                                     [0, 1, 10, 11, 12], [0, 1, 11, 12, 13]]
    tree = kv_plain.paths([0, 0, 0, 2], 4)
    assert window_plain.seen(10, 4, tree, 3, 0) == [[8, 9, 10], [9, 10, 11], [9, 10, 12],
                                                    [10, 12, 13]]
    assert window_plain.seen(1, 3, kv_plain.paths(None, 3), 1, 2) == [[0, 1], [0, 1, 2], [0, 1, 3]]
    assert window_plain.seen(3, 1, [[0]], 100, 1) == [[0, 1, 2, 3]]
