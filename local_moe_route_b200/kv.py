"""Binding of the speculative-decoding entry points (``include/strata_kv.h``):
the 8-bit paged KV cache, attention of a draft tree over it, and the
verification of drafts.

The functions forward to the C entry points of the same names and return
their status codes.  The descriptors ``KvCache`` and ``KvSeqs`` are built once
per set of tensors and kept; they hold references to the tensors whose
pointers they carry.  Torch tensors are checked before a call: one of another
type, on another device than the current one, or with elements that do not lie
the way the entry point reads them gives ``STRATA_ERR_INVALID_ARG`` and
nothing is launched.  Raw integer pointers pass unchecked.
"""

from __future__ import annotations

import ctypes
from typing import Any, Optional

from . import STRATA_ERR_INVALID_ARG, StrataError, _nbytes, _stream, lib

__all__ = [
    "STRATA_TREE_MAX_NODES", "STRATA_VERIFY_MAX_VOCAB", "KvCache", "KvSeqs", "VerifyDims",
    "strata_kv_append", "strata_kv_read", "strata_kv_commit", "strata_tree_attention",
    "strata_tree_attention_workspace_bytes", "tree_attention_workspace", "strata_verify_drafts",
]

STRATA_TREE_MAX_NODES = 64
STRATA_VERIFY_MAX_VOCAB = 800000


class _Refused(Exception):
    """A tensor argument the entry point would misread."""


_torch = None      # torch, imported with the first tensor that is checked


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _dev(t: Any, dtype: str, elements: Optional[int] = None) -> Optional[int]:
    """Pointer of a dense tensor of the current device with the given type (and
    number of elements); None and raw pointers pass."""
    if t is None or isinstance(t, int):
        return t
    torch = _torch or _load_torch()
    if t.dtype is not getattr(torch, dtype) or not t.is_contiguous() \
            or (elements is not None and t.numel() != elements) \
            or t.get_device() != _device():
        raise _Refused
    return t.data_ptr()


def _device() -> int:
    """Index of the current CUDA device; -2 without one (a host tensor's is -1)."""
    return _torch._C._cuda_getDevice() if _torch.cuda.is_initialized() else -2


def _rows(t: Any, B: int, N: int, heads: int, D: int):
    """Pointer and token stride of [B][N][heads][D] bf16 rows: the values of a
    token are dense, the tokens follow each other at one stride."""
    if t is None or isinstance(t, int):
        return t, 0
    torch = _torch or _load_torch()
    if t.dtype is not torch.bfloat16 or t.shape != (B, N, heads, D) \
            or t.get_device() != _device():
        raise _Refused
    if t.is_contiguous():
        return t.data_ptr(), 0
    sb, sn, sh, sd = t.stride()
    if sd != 1 or (heads > 1 and sh != D):
        raise _Refused
    step = sn if N > 1 else sb if B > 1 else 0
    if (N > 1 and B > 1 and sb != N * sn) or (step < heads * D and B * N > 1):
        raise _Refused
    return t.data_ptr(), step


def _here(*descriptors: Any) -> None:
    """Refuses descriptors whose tensors are not on the current device."""
    for d in descriptors:
        if d.device is not None and d.device != _device():
            raise _Refused


def _on(stream: Any) -> Optional[int]:
    """The stream's handle; None = the current stream of the current device."""
    if stream is None and _torch is not None and _torch.cuda.is_initialized():
        return _torch._C._cuda_getCurrentRawStream(_torch._C._cuda_getDevice())
    return _stream(stream)


class KvCache(ctypes.Structure):
    """strata_kv_cache_t: k, v [pages][Hkv][page][D] uint8 (e4m3 codes), k_exp,
    v_exp [pages][Hkv][page] uint8 (biased exponents)."""
    _fields_ = [("pages", ctypes.c_int32), ("page", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p)]
    device = None      # of the tensors; None: raw pointers

    @classmethod
    def of(cls, k: Any, v: Any, k_exp: Any, v_exp: Any) -> "KvCache":
        pages, Hkv, page, D = (int(n) for n in k.shape)
        rows = pages * Hkv * page
        try:
            c = cls(pages, page, Hkv, D, _dev(k, "uint8"), _dev(v, "uint8", rows * D),
                    _dev(k_exp, "uint8", rows), _dev(v_exp, "uint8", rows))
        except _Refused:
            raise StrataError(STRATA_ERR_INVALID_ARG, "KvCache") from None
        c.tensors, c.device = (k, v, k_exp, v_exp), k.get_device()
        return c

    @classmethod
    def empty(cls, pages: int, page: int, Hkv: int, D: int, device="cuda") -> "KvCache":
        """A cache that holds nothing yet (codes and exponents 0)."""
        import torch
        z = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=device)  # noqa: E731
        return cls.of(z(pages, Hkv, page, D), z(pages, Hkv, page, D), z(pages, Hkv, page),
                      z(pages, Hkv, page))


class KvSeqs(ctypes.Structure):
    """strata_kv_seqs_t: table [B][max_pages] int32, pos [B] int32, count [B]
    int32 or None (N)."""
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("table", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("count", ctypes.c_void_p)]
    device = None

    @classmethod
    def of(cls, table: Any, pos: Any, count: Any = None, N: int = 1) -> "KvSeqs":
        B, max_pages = (int(n) for n in table.shape)
        try:
            s = cls(B, int(N), max_pages, _dev(table, "int32"), _dev(pos, "int32", B),
                    _dev(count, "int32", B))
        except _Refused:
            raise StrataError(STRATA_ERR_INVALID_ARG, "KvSeqs") from None
        s.tensors, s.device = (table, pos, count), table.get_device()
        return s


class VerifyDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("V", ctypes.c_int32)]

    @classmethod
    def of(cls, dims: Any) -> "VerifyDims":
        if isinstance(dims, cls):
            return dims
        if isinstance(dims, dict):
            return cls(*[int(dims[k]) for k in ("B", "N", "V")])
        return cls(*[int(v) for v in dims])


_bound = None


def _lib() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        L = lib()
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        for name, args in (
                ("strata_kv_append", [KvCache, KvSeqs, vp, vp, i64, vp]),
                ("strata_kv_read", [KvCache, KvSeqs, vp, vp, vp]),
                ("strata_kv_commit", [KvCache, KvSeqs, vp, vp, vp, vp]),
                ("strata_tree_attention_workspace_bytes", [KvCache, KvSeqs, i32]),
                ("strata_tree_attention", [KvCache, KvSeqs, vp, vp, i64, i32, ctypes.c_float, vp,
                                           vp, sz, vp]),
                ("strata_verify_drafts", [vp, vp, vp, vp, vp, vp, vp, VerifyDims, vp, vp, vp,
                                          vp])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_int
        L.strata_tree_attention_workspace_bytes.restype = sz
        _bound = L
    return _bound


def strata_kv_append(cache: KvCache, seqs: KvSeqs, k, v, stride: int = 0, stream=None) -> int:
    """k, v [B][N][Hkv][D] bf16; tensors may be parts of wider rows (their token
    stride is taken from them, `stride` is for raw pointers)."""
    try:
        _here(cache, seqs)
        kp, ks = _rows(k, seqs.B, seqs.N, cache.Hkv, cache.D)
        vp, vs = _rows(v, seqs.B, seqs.N, cache.Hkv, cache.D)
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    if ks != vs:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_kv_append(cache, seqs, kp, vp, ks or int(stride), _on(stream))


def strata_kv_read(cache: KvCache, seqs: KvSeqs, k_out, v_out, stream=None) -> int:
    n = seqs.B * seqs.N * cache.Hkv * cache.D
    try:
        _here(cache, seqs)
        kp, vp = _dev(k_out, "bfloat16", n), _dev(v_out, "bfloat16", n)
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_kv_read(cache, seqs, kp, vp, _on(stream))


def strata_kv_commit(cache: KvCache, seqs: KvSeqs, path, path_len, pos_out, stream=None) -> int:
    try:
        _here(cache, seqs)
        a = (_dev(path, "int32", seqs.B * seqs.N), _dev(path_len, "int32", seqs.B),
             _dev(pos_out, "int32", seqs.B))
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_kv_commit(cache, seqs, *a, _on(stream))


def strata_tree_attention_workspace_bytes(cache: KvCache, seqs: KvSeqs, Hq: int) -> int:
    return int(_lib().strata_tree_attention_workspace_bytes(cache, seqs, int(Hq)))


def tree_attention_workspace(cache: KvCache, seqs: KvSeqs, Hq: int, device="cuda"):
    """A torch uint8 buffer of strata_tree_attention_workspace_bytes() bytes."""
    import torch
    n = strata_tree_attention_workspace_bytes(cache, seqs, Hq)
    if n == 0:
        raise StrataError(STRATA_ERR_INVALID_ARG, "tree attention workspace")
    return torch.empty(n, dtype=torch.uint8, device=device)


def strata_tree_attention(cache: KvCache, seqs: KvSeqs, parent, q, scale, out, ws,
                          ws_bytes: Optional[int] = None, Hq: Optional[int] = None,
                          q_stride: int = 0, stream=None) -> int:
    """q, out [B][N][Hq][D] bf16, parent [B][N] int32 or None; a q tensor may be a
    part of wider rows.  Hq and q_stride are for raw pointers."""
    B, N, D = seqs.B, seqs.N, cache.D
    try:
        _here(cache, seqs)
        if not isinstance(q, int) and q is not None:
            Hq = int(q.shape[2]) if q.dim() == 4 else 0
        heads = int(Hq or 0)
        qp, qs = _rows(q, B, N, heads, D)
        op, pp = _dev(out, "bfloat16", B * N * heads * D), _dev(parent, "int32", B * N)
        wp = _dev(ws, "uint8")
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_tree_attention(
        cache, seqs, pp, qp, qs or int(q_stride), heads, float(scale), op, wp,
        _nbytes(ws) if ws_bytes is None else int(ws_bytes), _on(stream))


def strata_verify_drafts(tokens, parent, count, p, q, u_accept, u_sample, dims, path, path_len,
                         out_tokens, stream=None) -> int:
    d = VerifyDims.of(dims)
    nodes, probs = d.B * d.N, d.B * d.N * d.V
    try:
        a = [_dev(tokens, "int32", nodes), _dev(parent, "int32", nodes), _dev(count, "int32", d.B),
             _dev(p, "float32", probs), _dev(q, "float32", probs),
             _dev(u_accept, "float32", nodes), _dev(u_sample, "float32", d.B)]
        o = [_dev(path, "int32", nodes), _dev(path_len, "int32", d.B),
             _dev(out_tokens, "int32", nodes)]
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_verify_drafts(*a, d, *o, _on(stream))
