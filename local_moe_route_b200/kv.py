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


# torch and what is used of it, looked up with the first call: these calls take a
# few microseconds on the device, so the host's part of them counts
_torch = _bf16 = _i32 = _f32 = _u8 = _current = _raw_stream = None


def _device() -> int:
    """Index of the current CUDA device; -2 without one (a host tensor's is -1)."""
    global _torch, _bf16, _i32, _f32, _u8, _current, _raw_stream
    if _torch is None:
        import torch
        _bf16, _i32, _f32, _u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
        if torch.cuda.is_available():
            torch.cuda.init()
            _current = torch._C._cuda_getDevice
            _raw_stream = torch._C._cuda_getCurrentRawStream
        _torch = torch
    return _current() if _current else -2


def _here(dev: int, *descriptors: Any) -> None:
    """Refuses descriptors whose tensors are not on the current device."""
    for d in descriptors:
        if d.device is not None and d.device != dev:
            raise _Refused


def _dev(t: Any, dtype: Any, dev: int, elements: Optional[int] = None) -> Optional[int]:
    """Pointer of a dense tensor of the current device with the given type (and
    number of elements); None and raw pointers pass."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev \
            or (elements is not None and t.numel() != elements):
        raise _Refused
    return t.data_ptr()


def _rows(t: Any, dev: int, B: int, N: int, heads: int, D: int):
    """Pointer and token stride of [B][N][heads][D] bf16 rows: the values of a
    token are dense, the tokens follow each other at one stride."""
    if t is None or t.__class__ is int:
        return t, 0
    if t.dtype is not _bf16 or t.shape != (B, N, heads, D) or t.get_device() != dev:
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


def _step(given: int, dense: int, *rows: Any) -> int:
    """The token stride given with raw pointers.  Beside a dense tensor any other than
    its own would lead past its end."""
    if given != dense and any(t is not None and t.__class__ is not int for t in rows):
        raise _Refused
    return given


def _ws_bytes(ws: Any, given: int) -> int:
    """The workspace's size as it is given, and no more than a tensor has."""
    n = max(int(given), 0)               # (it travels as a size without a sign)
    return n if ws is None or ws.__class__ is int else min(n, _nbytes(ws))


def _on(stream: Any, dev: int) -> Optional[int]:
    """The stream's handle; None = the current stream of the current device."""
    return _raw_stream(dev) if stream is None and dev >= 0 else _stream(stream)


class KvCache(ctypes.Structure):
    """strata_kv_cache_t: k, v [pages][Hkv][page][D] uint8 (e4m3 codes), k_exp,
    v_exp [pages][Hkv][page] uint8 (biased exponents)."""
    _fields_ = [("pages", ctypes.c_int32), ("page", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p)]
    device = None      # of the tensors; None: raw pointers

    @classmethod
    def of(cls, k: Any, v: Any, k_exp: Any, v_exp: Any) -> "KvCache":
        if k.dim() != 4:
            raise StrataError(STRATA_ERR_INVALID_ARG, "KvCache")
        pages, Hkv, page, D = (int(n) for n in k.shape)
        rows = pages * Hkv * page
        dev = _device()
        try:
            c = cls(pages, page, Hkv, D, _dev(k, _u8, dev), _dev(v, _u8, dev, rows * D),
                    _dev(k_exp, _u8, dev, rows), _dev(v_exp, _u8, dev, rows))
        except _Refused:
            raise StrataError(STRATA_ERR_INVALID_ARG, "KvCache") from None
        c.tensors, c.device = (k, v, k_exp, v_exp), dev
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
        if table.dim() != 2:
            raise StrataError(STRATA_ERR_INVALID_ARG, "KvSeqs")
        B, max_pages = (int(n) for n in table.shape)
        dev = _device()
        try:
            s = cls(B, int(N), max_pages, _dev(table, _i32, dev), _dev(pos, _i32, dev, B),
                    _dev(count, _i32, dev, B))
        except _Refused:
            raise StrataError(STRATA_ERR_INVALID_ARG, "KvSeqs") from None
        s.tensors, s.device = (table, pos, count), dev
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
    stride is taken from them, `stride` is for raw pointers: beside dense tensors another
    than theirs is refused)."""
    dev = _device()
    try:
        _here(dev, cache, seqs)
        kp, ks = _rows(k, dev, seqs.B, seqs.N, cache.Hkv, cache.D)
        vp, vs = _rows(v, dev, seqs.B, seqs.N, cache.Hkv, cache.D)
        if ks != vs:
            raise _Refused
        step = ks or stride and _step(stride, cache.Hkv * cache.D, k, v)
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_kv_append(cache, seqs, kp, vp, step, _on(stream, dev))


def strata_kv_read(cache: KvCache, seqs: KvSeqs, k_out, v_out, stream=None) -> int:
    dev = _device()
    n = seqs.B * seqs.N * cache.Hkv * cache.D
    try:
        _here(dev, cache, seqs)
        kp, vp = _dev(k_out, _bf16, dev, n), _dev(v_out, _bf16, dev, n)
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_kv_read(cache, seqs, kp, vp, _on(stream, dev))


def strata_kv_commit(cache: KvCache, seqs: KvSeqs, path, path_len, pos_out, stream=None) -> int:
    dev = _device()
    try:
        _here(dev, cache, seqs)
        a = (_dev(path, _i32, dev, seqs.B * seqs.N), _dev(path_len, _i32, dev, seqs.B),
             _dev(pos_out, _i32, dev, seqs.B))
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_kv_commit(cache, seqs, *a, _on(stream, dev))


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
    part of wider rows.  Hq and q_stride are for raw pointers; beside a dense q tensor
    another q_stride than its own is refused."""
    dev = _device()
    B, N, D = seqs.B, seqs.N, cache.D
    try:
        _here(dev, cache, seqs)
        if q is not None and q.__class__ is not int:
            Hq = q.shape[2] if q.dim() == 4 else 0
        heads = int(Hq or 0)
        qp, qs = _rows(q, dev, B, N, heads, D)
        step = qs or q_stride and _step(q_stride, heads * D, q)
        op, pp = _dev(out, _bf16, dev, B * N * heads * D), _dev(parent, _i32, dev, B * N)
        wp = _dev(ws, _u8, dev)
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_tree_attention(
        cache, seqs, pp, qp, step, heads, scale, op, wp,
        _nbytes(ws) if ws_bytes is None else _ws_bytes(ws, ws_bytes), _on(stream, dev))


def strata_verify_drafts(tokens, parent, count, p, q, u_accept, u_sample, dims, path, path_len,
                         out_tokens, stream=None) -> int:
    dev = _device()
    d = VerifyDims.of(dims)
    B = d.B
    nodes = B * d.N
    probs = nodes * d.V
    try:
        a = (_dev(tokens, _i32, dev, nodes), _dev(parent, _i32, dev, nodes),
             _dev(count, _i32, dev, B), _dev(p, _f32, dev, probs), _dev(q, _f32, dev, probs),
             _dev(u_accept, _f32, dev, nodes), _dev(u_sample, _f32, dev, B), d,
             _dev(path, _i32, dev, nodes), _dev(path_len, _i32, dev, B),
             _dev(out_tokens, _i32, dev, nodes))
    except _Refused:
        return STRATA_ERR_INVALID_ARG
    return (_bound or _lib()).strata_verify_drafts(*a, _on(stream, dev))
