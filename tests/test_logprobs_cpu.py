"""The log-probability calls without a GPU: declared symbols, argument errors (returned before any
launch), the binding's checks, and the plain implementation against autograd."""
import ctypes
import math
import os
import re

import pytest
import torch

import logprobs_plain as plain
from conftest import ROOT

P = 4096  # a 16-byte-aligned fake address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lp():
    from speculative_decoding_verification_18_gb300 import build, logprobs
    build.build()
    lib = logprobs.load()
    V, I, F, Z, L = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64)
    lib.spec_logprobs.argtypes = [V, I, L, V, F, I, I, I, I, V, V, V, V, V, V, Z, V, V]
    lib.spec_logprobs_grad.argtypes = [V, I, L, V, V, V, V, V, F, I, I, I, V, L, V, V]
    return logprobs


def test_every_declared_symbol_is_exported(lp):
    text = open(os.path.join(ROOT, "include", "specverify_logprobs.h")).read()
    names = set(re.findall(r"\b(spec_logprobs\w*)\s*\(", re.sub(r"/\*.*?\*/", "", text,
                                                                flags=re.S)))
    assert names == set(lp.EXPORTS)
    for n in names:
        assert hasattr(lp.load(), n)


def test_workspace_size(lp):
    size = lp.spec_logprobs_workspace_size
    assert size(0, 1) > 0 and size(1, 1 << 21, 1, 64, 64) > 0 and size((1 << 27) - 1, 5) > 0
    for bad in ((-1, 5), (1 << 27, 5), (1, 0), (1, (1 << 21) + 1), (1, 5, 2), (1, 5, 0, 0),
                (1, 5, 0, 65), (1, 5, 0, 1, -1), (1, 5, 0, 1, 65)):
        assert size(*bad) == 0, bad


def test_argument_errors(lp):
    need = lp.spec_logprobs_workspace_size(4, 100, 0, 2, 5)

    def call(l=P, dt=0, stride=100, tok=P, T=1.0, rows=4, V=100, given=2, top=5, out=P, norm=P,
             ent=P, tt=P, tl=P, ws=P, wsb=need, status=None):
        return lp.load().spec_logprobs(l, dt, stride, tok, T, rows, V, given, top, out, norm, ent,
                                       tt, tl, ws, wsb, status, None)

    for bad, code in ((dict(l=None), 1), (dict(tok=None), 1), (dict(out=None), 1), (dict(tt=None), 1),
                      (dict(tl=None), 1), (dict(dt=2), 1), (dict(dt=3), 1), (dict(stride=99), 1),
                      (dict(T=0.0), 1), (dict(T=-1.0), 1), (dict(T=math.nan), 1),
                      (dict(T=math.inf), 1), (dict(rows=-1), 1), (dict(V=0), 1), (dict(given=0), 1),
                      (dict(top=-1), 1), (dict(given=65), 3), (dict(top=65), 3),
                      (dict(V=(1 << 21) + 1, stride=1 << 22), 3), (dict(rows=1 << 27), 3),
                      (dict(stride=1 << 39), 3), (dict(stride=1 << 40), 3), (dict(l=P + 8), 1),
                      (dict(tok=P + 4), 1), (dict(out=P + 4), 1), (dict(norm=P + 4), 1),
                      (dict(ent=P + 4), 1), (dict(tt=P + 4), 1), (dict(tl=P + 4), 1),
                      (dict(ws=P + 4), 1), (dict(status=P + 4), 1), (dict(ws=None), 2),
                      (dict(wsb=need - 1), 2)):
        assert call(**bad) == code, bad
    assert call(rows=0) == 0 and call(rows=0, l=None, tok=None, out=None, tt=None, tl=None) == 0


def test_gradient_argument_errors(lp):
    def call(l=P, dt=1, stride=100, tok=P, norm=P, ent=P, g=P, gh=P, T=1.0, rows=4, V=100, given=2,
             out=2 * P, ostride=100, status=None):
        return lp.load().spec_logprobs_grad(l, dt, stride, tok, norm, ent, g, gh, T, rows, V, given,
                                            out, ostride, status, None)

    for bad, code in ((dict(l=None), 1), (dict(tok=None), 1), (dict(norm=None), 1), (dict(g=None), 1),
                      (dict(out=None), 1), (dict(ent=None), 1), (dict(dt=2), 1), (dict(stride=99), 1),
                      (dict(ostride=99), 1), (dict(T=0.0), 1), (dict(T=math.nan), 1),
                      (dict(rows=-1), 1), (dict(V=0), 1), (dict(given=0), 1), (dict(given=65), 3),
                      (dict(V=(1 << 21) + 1, stride=1 << 22, ostride=1 << 22), 3),
                      (dict(rows=1 << 27), 3), (dict(ostride=1 << 40), 3), (dict(l=P + 8), 1),
                      (dict(tok=P + 4), 1), (dict(norm=P + 4), 1), (dict(ent=P + 4), 1),
                      (dict(g=P + 4), 1), (dict(gh=P + 4), 1), (dict(out=P + 4), 1),
                      (dict(status=P + 4), 1), (dict(out=P, ostride=104), 1)):
        assert call(**bad) == code, bad
    assert call(rows=0) == 0


def test_binding_refusals(lp):
    """Types, shapes and layouts, before the library is called."""
    x = torch.zeros(3, 4, 50)
    t = torch.zeros(3, 4, dtype=torch.int32)
    o, ws = torch.zeros(3, 4), torch.zeros(4096, dtype=torch.uint8)
    two = torch.zeros(3, 4, 2)
    for call in (lambda: lp.spec_logprobs(x[0, 0], t[0, 0], o, ws),             # one dimension
                 lambda: lp.spec_logprobs(x[:, ::2].transpose(1, 2), t, o, ws),  # V not contiguous
                 lambda: lp.spec_logprobs(x[:, :3], t[:, :3].contiguous(), o[:, :3].contiguous(),
                                          ws),                                  # rows unevenly apart
                 lambda: lp.spec_logprobs(x, t[:2], o, ws),
                 lambda: lp.spec_logprobs(x, t, o[:2], ws),
                 lambda: lp.spec_logprobs(x, t[:, ::2], o[:, ::2], ws),
                 lambda: lp.spec_logprobs(x, t, o, ws, entropy=o[0]),
                 lambda: lp.spec_logprobs(x, t, o, ws, normalizer=o),
                 lambda: lp.spec_logprobs(x, t, o, ws, top_tokens=two.int()),    # no top_logprobs
                 lambda: lp.spec_logprobs(x, t, o, ws, top_tokens=two.int(), top_logprobs=o),
                 lambda: lp.spec_logprobs(x, t, o, ws, status=t[0]),
                 lambda: lp.spec_logprobs_grad(x, t, two, o, x[:2]),
                 lambda: lp.spec_logprobs_grad(x, t, two, o, x.transpose(0, 1)),
                 lambda: lp.spec_logprobs_grad(x, t, o, o, x),
                 lambda: lp.spec_logprobs_grad(x, t, two, two, x),
                 lambda: lp.spec_logprobs_grad(x, t, two, o, x, grad_entropy=o)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lp.spec_logprobs(x.half(), t, o, ws),
                 lambda: lp.spec_logprobs(x, t.long(), o, ws),
                 lambda: lp.spec_logprobs(x, t, o.bfloat16(), ws),
                 lambda: lp.spec_logprobs(x, t, o, ws.int()),
                 lambda: lp.spec_logprobs(x, None, o, ws),
                 lambda: lp.spec_logprobs(x, t, None, ws),
                 lambda: lp.spec_logprobs(x, t, o, ws, T="hot"),
                 lambda: lp.spec_logprobs(x, t, o, ws, status=o),
                 lambda: lp.spec_logprobs_grad(x, t, two, o, x.bfloat16()),
                 lambda: lp.spec_logprobs_grad(x, t, None, o, x),
                 lambda: lp.spec_logprobs_grad(x, t, two, None, x)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="CUDA"):
        lp.spec_logprobs(x, t, o, ws)
    with pytest.raises(ValueError, match="CUDA"):
        lp.spec_logprobs_grad(x, t, two, o, x)


def test_plain_gradient_is_autograds():
    """The formula of the gradient against autograd of the definitions, in 64 bits, and against
    differences of the plain forward values."""
    g = torch.Generator().manual_seed(0)
    R, V, K, T = 4, 30, 3, 0.7
    l = torch.randn(R, V, generator=g, dtype=torch.float64).requires_grad_()
    tokens = torch.tensor([[1, 5, 1], [0, 29, 3], [7, -1, 7], [-1, -1, 2]], dtype=torch.int32)
    gl, gh = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((R, K), (R,)))
    lp = torch.log_softmax(l / T, 1)
    H = -(lp.exp() * lp).sum(1)
    told = lp.gather(1, tokens.clamp(min=0).long()) * (tokens >= 0)
    ((told * gl).sum() + (H * gh).sum()).backward()
    x = l.detach()
    want = plain.forward(x, tokens, T, 0)
    assert float((want["entropy"][0] - H.detach()).abs().max()) < 1e-12
    y, _ = plain.gradient(x, tokens, want["normalizer"][0], want["entropy"][0], gl, gh, T,
                          torch.float32)
    assert float((y - l.grad).abs().max()) < 1e-12
    h = 1e-5

    def value(z):
        f = plain.forward(z, tokens, T, 0)
        return (torch.where(tokens >= 0, f["logprobs"][0], 0.0) * gl).sum(1) + f["entropy"][0] * gh
    for v in (0, 1, 7, 12):
        step = torch.zeros(V, dtype=torch.float64)
        step[v] = h
        d = (value(x + step) - value(x - step)) / (2 * h)
        assert float((d - y[:, v]).abs().max()) < 1e-8


def test_temperatures_out_of_range(lp):
    """Beyond 2^-100 to 2^100 a gradient's factor, or the entropy of a row whose masks are its
    type's lowest value, would leave fp32."""
    for T, code in ((2.0**-101, 3), (1e-45, 3), (2.0**101, 3), (3e38, 3), (2.0**-100, 0), (2.0**100, 0)):
        assert lp.load().spec_logprobs(P, 1, 100, P, T, 0, 100, 1, 0, P, None, None, None, None, P,
                                       256, None, None) == code
        assert lp.load().spec_logprobs_grad(P, 1, 100, P, P, None, P, None, T, 0, 100, 1, 2 * P, 100,
                                            None, None) == code
