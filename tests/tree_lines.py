"""Cases of the tree attention whose work fills the GPU several times over: every CTA
works through many tiles and units.  Pages are shared between sequences, so the caches
stay small; NumPy only, the same on the host and for the GPU."""

import numpy as np

from moe_inputs import bf16_bits
from oracle import speculative as osp

#  name: B, N, Hq, Hkv, D, page, shortest and longest length, kind
# One block of up to 16 rows per unit, or blocks of 32, at either head size; from 2
# tiles per CTA (296 CTAs) to 18, from one unit per CTA to 10, units cut anywhere.
CASES = {
    "decode_D128": (32, 1, 32, 4, 128, 64, 2, 10000, "chain"),
    "decode_long_D128": (48, 1, 32, 4, 128, 16, 3000, 10300, "chain"),
    "chain4_D128": (44, 4, 32, 4, 128, 64, 8000, 12000, "chain"),
    "tree24_D128": (8, 24, 8, 2, 128, 32, 500, 5500, "tree"),
    "tree24_D64": (16, 24, 16, 2, 64, 32, 10, 8200, "tree"),
    "tree64_D64": (24, 64, 16, 2, 64, 128, 2500, 4600, "tree"),
    "pairs_long_D64": (32, 2, 9, 3, 64, 16, 9000, 33000, "chain"),
    "many_chain4_D128": (700, 4, 16, 2, 128, 16, 0, 600, "chain"),
    "many_decode_D128": (2000, 1, 8, 2, 128, 32, 0, 520, "chain"),
    "many_forest_D64": (500, 6, 24, 3, 64, 64, 0, 700, "forest"),
    "few_long_D128": (2, 3, 9, 3, 128, 128, 20000, 45000, "tree"),
}


def tiles(name, pos, count):
    B, N, Hq, Hkv, D = CASES[name][:5]
    rows = N * Hq // Hkv
    R = 16 if rows <= 16 else 32
    return sum(Hkv * -(-c * (Hq // Hkv) // R) * -(-(p + c) // 256) for p, c in zip(pos, count) if c)


class Line:
    """A pool of pages, tables into it in rising, falling or no order of the scores that
    their rows get; a few rows that hold no K or (even seeds) no V, and page numbers
    out of range."""

    def __init__(self, name, seed=0):
        B, self.N, self.Hq, Hkv, D, page, low, high, kind = CASES[name]
        N = self.N
        rng = np.random.default_rng([seed, list(CASES).index(name)])
        pool = max(64, 4096 // page)
        self.page = page
        e4 = osp.E4M3
        c = {n: rng.integers(0, 256, (pool, Hkv, page, D)).astype(np.uint8) for n in "kv"}
        for x in c.values():
            x[(x & 0x7F) >= 0x78] ^= 0x40                  # below 256, and no NaN
        # what a page's rows score: eight dimensions in which every query is positive
        level = rng.integers(-4, 5, pool) * 56.0
        code = np.array([int(np.nanargmin(np.abs(e4 - v))) for v in level], np.uint8)
        c["k"][..., :8] = code[:, None, None, None]
        self.cache = dict(c, k_exp=np.full((pool, Hkv, page), 127 - 8, np.uint8),
                          v_exp=(127 - 8 - rng.integers(0, 6, (pool, Hkv, page))).astype(np.uint8))
        self.cache["k_exp"][rng.random((pool, Hkv, page)) < 0.01] = 0
        if seed % 2 == 0:        # (a tile with such a row takes a reference of its own for
            self.cache["v_exp"][rng.random((pool, Hkv, page)) < 0.01] = 0   # the scores)
        self.pos = rng.integers(low, high + 1, B).astype(np.int32)
        self.pos[0] = high
        self.count = rng.integers(0, N + 1, B).astype(np.int32) if N > 1 \
            else (rng.random(B) < 0.95).astype(np.int32)
        self.count[0] = N
        cols = -(-(high + N) // page) + 1
        self.table = rng.integers(0, pool, (B, cols)).astype(np.int32)
        for b in range(B):
            if b % 3 < 2:
                used = -(-(int(self.pos[b]) + N) // page)
                self.table[b, :used] = sorted(self.table[b, :used],
                                              key=lambda p: level[p] * (1 if b % 3 else -1))
        self.bad_pages = False
        if high > 2000:
            self.bad_pages = True
            for b in range(1, B, 5):
                at = int(self.pos[b]) // page
                self.table[b, at // 2] = -1
                self.table[b, at - 2] = pool
        q = 0.7 * rng.standard_normal((B, N, self.Hq, D)).astype(np.float32)
        q[..., :8] = 6.0 / np.sqrt(8) * rng.random((B, N, self.Hq, 1))
        self.q = bf16_bits(q)
        self.parent = None
        if kind != "chain":
            self.parent = np.full((B, N), -1, np.int32)
            if kind == "tree":
                for i in range(1, N):
                    self.parent[:, i] = rng.integers(max(0, i - 5), i, B)
            else:
                self.parent[:, 1::2] = np.arange(0, N, 2)[:N // 2]
