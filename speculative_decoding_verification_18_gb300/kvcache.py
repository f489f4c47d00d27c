"""Thin binding of the paged key-value cache calls (include/specverify_kv.h):
``spec_kv_append``, ``spec_kv_attention`` and ``spec_kv_commit``.

Like specverify.py it only marshals arguments: torch CUDA tensors on the current
device, launches on the current torch stream unless ``stream`` is given, no CPU
fallback.  Shapes, types and layouts are checked on the way, in csrc/kvbind.cpp
(ValueError / TypeError); everything else by the library (SpecVerifyError).

One round of a layer, and the commit of all layers after the verdict::

    cache = PagedCache(k[layer], v[layer], table)
    spec_kv_append(cache, k_new, v_new, kv_len, q=q, q_out=q, rope=rope, parents=parents)
    spec_kv_attention(cache, q, kv_len, out, ws, dim ** -0.5, parents=parents)
    ...
    specverify.spec_verify_tree(..., out_nodes, num_accepted, ...)
    spec_kv_commit(PagedCache(k, v, table), kv_len, num_accepted, kv_len_out, out_nodes)
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import specverify as sv

SV_F16, SV_E4M3 = 2, 3
SV_DEV_BAD_PAGE, SV_DEV_BAD_LENGTH, SV_DEV_TIMEOUT = 0x80, 0x100, 0x200

EXPORTS = ("spec_kv_rope_turns", "spec_kv_append", "spec_kv_attention_workspace_size",
           "spec_kv_attention", "spec_kv_commit")

_TYPES = {torch.bfloat16: sv.SV_BF16, torch.float16: SV_F16, torch.float8_e4m3fn: SV_E4M3}


class _Cache(ctypes.Structure):
    """sv_kv_cache."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "table", "k_scale", "v_scale")]
                + [(n, ctypes.c_int64) for n in ("page_stride", "slot_stride", "head_stride")]
                + [(n, ctypes.c_int) for n in ("num_pages", "page_size", "table_width", "heads",
                                               "dim", "dtype")])


class _Rope(ctypes.Structure):
    """sv_rope."""
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("magnitude", ctypes.c_float)]


BIND = os.path.join(sv.HERE, "_kvbind.so")
_lib = _bind = None


def load():
    """The library with the cache calls declared (raises if it has not been built)."""
    global _lib, _bind
    if _lib is not None:
        return _lib
    lib = sv.load()
    P, I, Z, D = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
    lib.spec_kv_rope_turns.argtypes = [I, D, D, D, D, D, P]
    lib.spec_kv_attention_workspace_size.argtypes = [I, I, I, I, I]
    lib.spec_kv_attention_workspace_size.restype = Z
    lib.spec_kv_rope_turns.restype = I
    if not os.path.exists(BIND):
        raise ImportError(f"_kvbind.so is not built ({BIND}); run "
                          "speculative_decoding_verification_18_gb300.build.build() first")
    loader = importlib.machinery.ExtensionFileLoader("_kvbind", BIND)
    bind = importlib.util.module_from_spec(importlib.util.spec_from_loader("_kvbind", loader))
    loader.exec_module(bind)
    address = lambda f: ctypes.cast(f, P).value
    bind.bind(address(lib.spec_kv_append), address(lib.spec_kv_attention),
              address(lib.spec_kv_commit))
    _lib, _bind = lib, bind
    return lib


def _on_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")


def _vector(t, name, shape, dtype=torch.int32):
    """Pointer of a contiguous tensor of this shape and type (None: NULL)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _on_device(t, name)
    return t.data_ptr()


class PagedCache:
    """A paged cache: keys and values [pages, page_size, heads, dim], or [layers,
    pages, page_size, heads, dim], in bfloat16, float16 or float8_e4m3fn, any
    strides with contiguous dim (a cache stored as [pages, heads, page_size, dim]
    is passed transposed), and the page table [B, width] int32.  float8 caches
    have k_scale and v_scale [heads] (with layers: [layers, heads]) float32: an
    entry stands for its stored value times its head's scale; a cache that is only
    committed needs none.  Keeps the tensors."""

    def __init__(self, k, v, table, k_scale=None, v_scale=None):
        if k.dtype not in _TYPES:
            raise TypeError(f"caches are bfloat16, float16 or float8_e4m3fn, not {k.dtype}")
        if v.dtype != k.dtype:
            raise TypeError(f"v is {v.dtype} and k {k.dtype}")
        if k.dim() not in (4, 5) or v.shape != k.shape or min(k.shape) < 1:
            raise ValueError("k and v must have one shape, [layers,] pages, page_size, heads, dim")
        if v.stride() != k.stride():
            raise ValueError("k and v must have the same strides")
        if k.stride(-1) != 1:
            raise ValueError("the last dimension of k and v must be contiguous")
        if table.dim() != 2:
            raise ValueError("table must be [B, width]")
        for t, name in ((k, "k"), (v, "v")):
            _on_device(t, name)
        self.k, self.v, self.table, self.k_scale, self.v_scale = k, v, table, k_scale, v_scale
        self.layers = k.shape[0] if k.dim() == 5 else 1
        pages, page_size, heads, dim = k.shape[-4:]
        self.heads, self.dim, self.dtype = heads, dim, k.dtype
        if (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale come together")
        if k_scale is not None and k.dtype != torch.float8_e4m3fn:
            raise ValueError("k_scale and v_scale belong to float8_e4m3fn caches only")
        sp, ss, sh = k.stride()[-4:-1]
        sh = sh if heads > 1 else dim  # the stride of a dimension of one entry means nothing
        ss = ss if page_size > 1 else heads * sh
        sp = sp if pages > 1 else page_size * ss
        self.layer_stride = k.stride(0) if self.layers > 1 else 0
        lead = (self.layers, heads) if k.dim() == 5 else (heads,)
        self._scales = [_vector(t, n, lead, torch.float32)
                        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale"))]
        tp = _vector(table, "table", table.shape)
        self._layers = []
        for i in range(self.layers):
            at = i * self.layer_stride * k.element_size()
            scales = [p and p + 4 * heads * i for p in self._scales]
            self._layers.append(_Cache(k.data_ptr() + at, v.data_ptr() + at, tp, *scales, sp, ss,
                                       sh, pages, page_size, table.shape[1], heads, dim,
                                       _TYPES[k.dtype]))
        load()
        self._addresses = [ctypes.addressof(c) for c in self._layers]
        self._rows, self._device = table.shape[0], k.get_device()
        self._held = (k, v, table, k_scale, v_scale)  # whatever becomes of the attributes

    def layer(self, i):
        """Address of the sv_kv_cache of layer i."""
        if not 0 <= i < self.layers:
            raise ValueError(f"layer {i} of {self.layers}")
        if self.k_scale is None and self.dtype == torch.float8_e4m3fn:
            raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale here")
        return self._addresses[i]


class Rope:
    """Rates and layout of a rotation of the first rot_dim elements of each head
    (sv_rope, spec_kv_rope_turns); its table lives on the device."""

    def __init__(self, rot_dim, base=10000.0, interleaved=False, factor=1.0, original_length=0,
                 low=1.0, high=32.0, magnitude=1.0, device=None):
        turns = (ctypes.c_uint64 * max(1, rot_dim // 2))()
        sv._check(load().spec_kv_rope_turns(int(rot_dim), float(base), float(factor),
                                            float(original_length), float(low), float(high),
                                            turns), "spec_kv_rope_turns")
        host = torch.frombuffer(turns, dtype=torch.int64).clone()
        self.turns = host.to(device or "cuda")
        self.rot_dim, self.interleaved, self.magnitude = rot_dim, bool(interleaved), magnitude
        self._c = _Rope(self.turns.data_ptr(), rot_dim, int(self.interleaved), float(magnitude))
        self._address = ctypes.addressof(self._c)
        self._held = self.turns


def spec_kv_append(cache, k, v, kv_len, q=None, q_out=None, rope=None, parents=None, num_new=None,
                   status=None, layer=0, stream=None):
    """Rotate the new tokens' q and k [B, N, heads, dim] by `rope` (None: not at all) and write
    k and v behind the kv_len[b] cached entries; q_out (contiguous, may be q) gets the queries."""
    if rope is not None:
        _on_device(rope.turns, "rope")
    st = _bind.append(cache.layer(layer), cache._rows, cache._device, k, v, kv_len, q, q_out,
                      None if rope is None else rope._address, parents, num_new, status,
                      None if stream is None else sv._stream(stream))
    if st:
        sv._check(st, "spec_kv_append")


def spec_kv_attention_workspace_size(B, N, q_heads, heads, dim) -> int:
    return int(load().spec_kv_attention_workspace_size(B, N, q_heads, heads, dim))


def attention_workspace(cache, B, N, q_heads, device=None):
    """A workspace tensor of the required size (bytes, uint8)."""
    n = spec_kv_attention_workspace_size(B, N, q_heads, cache.heads, cache.dim)
    if n == 0:
        raise sv.SpecVerifyError(sv.SV_ERR_INVALID_ARG, "spec_kv_attention_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or cache.k.device)


def spec_kv_attention(cache, q, kv_len, out, ws, scale, parents=None, num_new=None, status=None,
                      layer=0, stream=None):
    """Attention of the new tokens' q [B, N, q_heads, dim] over the kv_len[b] cached entries and
    their own ancestors' -> out (contiguous).  ws: attention_workspace(...)."""
    st = _bind.attention(cache.layer(layer), cache._rows, cache._device, q, kv_len, out, ws, scale,
                         parents, num_new, status, None if stream is None else sv._stream(stream))
    if st:
        sv._check(st, "spec_kv_attention")


def spec_kv_commit(cache, kv_len, num_accepted, kv_len_out, out_nodes=None, status=None,
                   stream=None):
    """Move the accepted nodes' entries of every layer behind the committed ones;
    kv_len_out = kv_len + num_accepted + 1.  out_nodes [B, N] as spec_verify_tree writes it;
    None for a chain."""
    st = _bind.commit(cache._addresses[0], cache._rows, cache._device, cache.layers,
                      cache.layer_stride, kv_len, num_accepted, kv_len_out, out_nodes, status,
                      None if stream is None else sv._stream(stream))
    if st:
        sv._check(st, "spec_kv_commit")
