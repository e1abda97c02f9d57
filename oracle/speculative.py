"""fp64 oracle for a speculative-decoding step over an 8-bit paged KV cache --
TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): it never calls the CUDA
library and the library never calls it.

Plain definitions, one loop per sequence, of the five entry points of
``include/strata_kv.h``.  bf16 tensors are bit patterns (uint16), caches are
dicts of uint8 arrays ``k``, ``v`` [pages][Hkv][page][D] and ``k_exp``, ``v_exp``
[pages][Hkv][page].
"""

from __future__ import annotations

from typing import Dict, Optional

import numpy as np


def _table() -> np.ndarray:
    """The values of the 256 e4m3 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits, subnormals at exponent 0, 0x7F and 0xFF NaN, no infinity."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if e == 15 and m == 7 else -x if c & 0x80 else x
    return v


E4M3 = _table()


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32) \
        .astype(np.float64)


def e4m3_code(y: float) -> int:
    """The code nearest to y, ties to the even code, magnitudes above 448 to 448."""
    if not np.isfinite(y):
        return 0x7F
    mag = E4M3[:0x7F]
    a = min(abs(y), 448.0)
    i = int(np.searchsorted(mag, a))
    if i > 0 and (a - mag[i - 1] < mag[i] - a or (a - mag[i - 1] == mag[i] - a and i % 2)):
        i -= 1
    return i | (0x80 if np.signbit(y) else 0)


def row_exponent(x: np.ndarray) -> int:
    """Smallest e in [-126, 119] with max|x| <= 448 * 2^e over the finite values."""
    top = np.max(np.abs(x[np.isfinite(x)]), initial=0.0)
    e = -126
    while e < 119 and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def quantise_row(x: np.ndarray):
    e = row_exponent(x)
    return np.array([e4m3_code(v / 2.0 ** e) for v in x], np.uint8), e + 127


def _at(cache, table, b, t):
    page = cache["k"].shape[2]
    if t // page >= table.shape[1]:
        return None
    pg = int(table[b, t // page])
    return (pg, t % page) if 0 <= pg < cache["k"].shape[0] else None


def _ranges(table, pos, count, N):
    for b in range(table.shape[0]):
        n = N if count is None else int(count[b])
        if int(pos[b]) >= 0 and 0 <= n <= N:
            yield b, int(pos[b]), n


def append(cache: Dict[str, np.ndarray], table, pos, count, k, v) -> None:
    """k, v [B][N][Hkv][D] bf16 bits, written into `cache` in place."""
    B, N, Hkv, _ = k.shape
    for b, p, n in _ranges(table, pos, count, N):
        for i in range(n):
            at = _at(cache, table, b, p + i)
            if at is None:
                continue
            for name, x in (("k", k), ("v", v)):
                for h in range(Hkv):
                    codes, e = quantise_row(bf16_values(x[b, i, h]))
                    cache[name][at[0], h, at[1]] = codes
                    cache[name + "_exp"][at[0], h, at[1]] = e


def row(cache, name, at, h) -> Optional[np.ndarray]:
    e = int(cache[name + "_exp"][at[0], h, at[1]])
    return None if e == 0 else E4M3[cache[name][at[0], h, at[1]]] * 2.0 ** (e - 127)


def read(cache, table, pos, count, N):
    """fp64 values [B][N][Hkv][D] of K and V; NaN-filled where nothing is read."""
    Hkv, D = cache["k"].shape[1], cache["k"].shape[3]
    out = [np.full((table.shape[0], N, Hkv, D), np.nan) for _ in range(2)]
    for b, p, n in _ranges(table, pos, count, N):
        for i in range(n):
            at = _at(cache, table, b, p + i)
            for o, name in zip(out, ("k", "v")):
                for h in range(Hkv):
                    r = None if at is None else row(cache, name, at, h)
                    o[b, i, h] = 0.0 if r is None else r
    return out


def ancestors(parent: Optional[np.ndarray], n: int) -> np.ndarray:
    """[n][n] truth values: node i sees node j."""
    sees = np.eye(n, dtype=bool)
    for i in range(n):
        up = i - 1 if parent is None else int(parent[i])
        if 0 <= up < i:
            sees[i] |= sees[up]
    return sees


def tree_attention(cache, table, pos, count, parent, q, scale=None) -> np.ndarray:
    """q [B][N][Hq][D] bf16 bits -> fp64 [B][N][Hq][D]; rows of slots behind a
    sequence's count are NaN, a node that sees nothing gets zeros."""
    B, N, Hq, D = q.shape
    Hkv = cache["k"].shape[1]
    sc = 1.0 / np.sqrt(D) if scale is None else float(scale)
    qf = bf16_values(q)
    out = np.full((B, N, Hq, D), np.nan)
    for b, p, n in _ranges(table, pos, count, N):
        sees = ancestors(None if parent is None else parent[b], n)
        for hk in range(Hkv):
            ts, ks, vs = [], [], []
            for t in range(p + n):
                at = _at(cache, table, b, t)
                if at is None or cache["k_exp"][at[0], hk, at[1]] == 0:
                    continue
                ts.append(t)
                ks.append(row(cache, "k", at, hk))
                r = row(cache, "v", at, hk)
                vs.append(np.zeros(D) if r is None else r)
            ts = np.array(ts, np.int64)
            ks, vs = np.array(ks).reshape(-1, D), np.array(vs).reshape(-1, D)
            for i in range(n):
                vis = np.array([t < p or sees[i, t - p] for t in ts], bool)
                for h in range(hk * (Hq // Hkv), (hk + 1) * (Hq // Hkv)):
                    if not vis.any():
                        out[b, i, h] = 0.0
                        continue
                    with np.errstate(invalid="ignore"):
                        s = sc * (ks[vis] @ qf[b, i, h])
                        w = np.exp(s - np.max(s))
                        out[b, i, h] = (w @ vs[vis]) / np.sum(w)
    return out


def verify(tokens, parent, count, p, q, u_accept, u_sample):
    """Rejection sampling down the tree, the row of the remaining target kept and
    normalised step by step.  Returns path, path_len, out_tokens."""
    B, N = tokens.shape
    V = p.shape[2]
    path = np.full((B, N), -1, np.int32)
    toks = np.full((B, N), -1, np.int32)
    length = np.zeros(B, np.int32)
    for b in range(B):
        n = N if count is None else int(count[b])
        if n <= 0 or n > N:
            continue
        cur, nodes = 0, [0]
        r = p[b, 0].astype(np.float64)
        for i in range(1, n):
            up = i - 1 if parent is None else int(parent[b, i])
            x = int(tokens[b, i])
            if up != cur or not 0 <= x < V:
                continue
            if q is None:
                qr = np.zeros(V)
                qr[x] = 1.0
            else:
                qr = q[b, cur].astype(np.float64)
            if float(u_accept[b, i]) * qr[x] < r[x]:
                cur = i
                nodes.append(i)
                r = p[b, i].astype(np.float64)
            else:
                r = np.maximum(r - qr, 0.0) if q is not None else np.where(qr > 0, 0.0, r)
                total = r.sum()
                r = r / total if total > 0 else r
        run = np.cumsum(r)
        over = np.nonzero(run > float(u_sample[b]) * run[-1])[0]
        some = np.nonzero(r > 0)[0]
        nxt = int(over[0]) if over.size else int(some[-1]) if some.size else 0
        length[b] = len(nodes)
        path[b, :len(nodes)] = nodes
        toks[b, :len(nodes)] = [int(tokens[b, i]) for i in nodes[1:]] + [nxt]
    return path, length, toks


def commit(cache, table, pos, path, path_len) -> np.ndarray:
    """Moves the path's rows in place; returns the new positions."""
    old = {n: x.copy() for n, x in cache.items()}
    out = np.array(pos, np.int32).copy()
    B, N = path.shape
    for b in range(B):
        n = int(path_len[b])
        if not 0 <= n <= N or int(pos[b]) < 0:
            continue
        for i in range(n):
            src = int(path[b, i])
            if not i <= src < N:
                continue
            a, z = _at(cache, table, b, int(pos[b]) + src), _at(cache, table, b, int(pos[b]) + i)
            if a is None or z is None:
                continue
            for name in cache:
                cache[name][z[0], :, z[1]] = old[name][a[0], :, a[1]]
        out[b] += n
    return out
