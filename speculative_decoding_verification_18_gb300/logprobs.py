"""Thin binding of the log-probability calls (include/specverify_logprobs.h):
``spec_logprobs`` and its gradient ``spec_logprobs_grad``.

Like specverify.py it only marshals arguments: torch CUDA tensors on the current
device, launches on the current torch stream unless ``stream`` is given, no CPU
fallback.  Shapes, types and layouts are checked on the way, in csrc/lpbind.cpp
(ValueError / TypeError); everything else by the library (SpecVerifyError).

What a server tells beside a round's tokens::

    specverify.spec_verify_sample(logits, ..., out_tokens, num_accepted, ws)
    spec_logprobs(logits, out_tokens, logprobs, lws, T=T, entropy=entropy,
                  top_tokens=top_tokens, top_logprobs=top_logprobs)

and a step of a draft's training towards the target's alternatives (a loss that is
minus the sum of p log q over them)::

    spec_logprobs(draft_logits, top_tokens, draft_logprobs, lws, normalizer=normalizer)
    spec_logprobs_grad(draft_logits, top_tokens, normalizer, -top_logprobs.exp(), grad_logits)
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import specverify as sv

SV_LOGPROBS_MAX_GIVEN = SV_LOGPROBS_MAX_TOP = 64

EXPORTS = ("spec_logprobs_workspace_size", "spec_logprobs", "spec_logprobs_grad")

BIND = os.path.join(sv.HERE, "_lpbind.so")
_lib = _bind = None


def load():
    """The library with the log-probability calls declared (raises if it has not been built)."""
    global _lib, _bind
    if _lib is not None:
        return _lib
    lib = sv.load()
    I, Z = ctypes.c_int, ctypes.c_size_t
    lib.spec_logprobs_workspace_size.argtypes = [I, I, I, I, I]
    lib.spec_logprobs_workspace_size.restype = Z
    if not os.path.exists(BIND):
        raise ImportError(f"_lpbind.so is not built ({BIND}); run "
                          "speculative_decoding_verification_18_gb300.build.build() first")
    loader = importlib.machinery.ExtensionFileLoader("_lpbind", BIND)
    bind = importlib.util.module_from_spec(importlib.util.spec_from_loader("_lpbind", loader))
    loader.exec_module(bind)
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    bind.bind(address(lib.spec_logprobs), address(lib.spec_logprobs_grad))
    _lib, _bind = lib, bind
    return lib


def spec_logprobs_workspace_size(rows, V, dtype=sv.SV_BF16, given=1, top=0) -> int:
    return int(load().spec_logprobs_workspace_size(rows, V, dtype, given, top))


def logprobs_workspace(logits, given=1, top=0):
    """A workspace tensor of the required size (bytes, uint8) for rows like these; calls that overlap
    may share it."""
    V = logits.shape[-1]
    n = spec_logprobs_workspace_size(logits.numel() // max(V, 1), V, sv._dtype(logits), given, top)
    if n == 0:
        raise sv.SpecVerifyError(sv.SV_ERR_INVALID_ARG, "spec_logprobs_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=logits.device)


def spec_logprobs(logits, tokens, logprobs, ws, T=1.0, entropy=None, normalizer=None,
                  top_tokens=None, top_logprobs=None, status=None, stream=None):
    """logits [..., V] bf16/fp32 (rows equally far apart), tokens [...] or [..., given] int32 (-1:
    none) -> logprobs like tokens, and where given entropy [...], normalizer [..., 2], top_tokens
    and top_logprobs [..., top].  ws: logprobs_workspace(...)."""
    if _bind is None:
        load()
    st = _bind.logprobs(logits, tokens, logprobs, ws, T, entropy, normalizer, top_tokens,
                        top_logprobs, status, None if stream is None else sv._stream(stream))
    if st:
        sv._check(st, "spec_logprobs")


def spec_logprobs_grad(logits, tokens, normalizer, grad_logprobs, grad_logits, T=1.0, entropy=None,
                       grad_entropy=None, status=None, stream=None):
    """Gradient of sum(grad_logprobs * logprobs) + sum(grad_entropy * entropy) to the logits ->
    grad_logits (like logits, or logits itself); normalizer and entropy from spec_logprobs."""
    if _bind is None:
        load()
    st = _bind.grad(logits, tokens, normalizer, grad_logprobs, grad_logits, T, entropy,
                    grad_entropy, status, None if stream is None else sv._stream(stream))
    if st:
        sv._check(st, "spec_logprobs_grad")
