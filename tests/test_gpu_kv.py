"""The 8-bit paged KV cache and the tree attention on the GPU, through the
public binding, against the fp64 oracle (oracle/speculative.py).

Bars.  Codes and exponents are whole numbers with one right answer: compared
exactly.  A read is exact up to the rounding to bf16 (none in bf16's normal
range).  Attention, per value, with A = sum_j p_j |v_j| / sum p:
  * the output's rounding, half a bf16 step: 2^-8 |o|;
  * the weights' rounding for the product with V, 2^-9, before it to fp16,
    2^-11, and their floor: a tile's largest weight is scaled to 224 .. 448,
    e4m3's smallest step is 2^-9, so a weight is off by 2^-10 / 224 = 2^-17.8 of the
    tile's largest at most, in units of the tile's largest V scale, whose codes
    reach 448 where its row may hold 224: over the 256 positions of a tile 256 *
    2^-17.8 * 2 = 2^-8.8 of the largest |V| value;
  * the scores: q is split into two e4m3 values, exact down to 2^-17 of the
    row's largest, and D products are summed in fp32 (2^-24 each): an error ds of
    a score changes a weight by about ds, numerator and denominator each.
Every bar is the sum of these bounds; nothing in it was fitted."""

import numpy as np
import pytest
import torch

import local_moe_route_b200 as sm
from gpu_helpers import assert_device_ok, bf16_host, bf16_to_f64
from moe_inputs import bf16_bits
from oracle import speculative as osp

pytestmark = pytest.mark.gpu
NAMES = ("k", "v", "k_exp", "v_exp")


@pytest.fixture(scope="module")
def dev(cuda_dev):
    from local_moe_route_b200 import build
    build.build()
    return cuda_dev


def up(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def up_bf16(bits, dev):
    return up(bits.view(np.int16), dev).view(torch.bfloat16)


class Setup:
    """A cache of random codes (NaN codes everywhere no position lies), a page
    table in no order, and the tensors of one call."""

    def __init__(self, rng, dev, pos, count, N, Hkv, D, page, spare=2, spread=3, slack=0):
        self.pos = np.array(pos, np.int32)
        self.N, self.Hkv, self.D, self.page = N, Hkv, D, page
        self.count = None if count is None else np.array(count, np.int32)
        B = len(pos)
        n = np.full(B, N) if count is None else np.array(count)
        self.end = np.maximum(self.pos, 0) + n
        cols = max(1, int(-(-self.end.max() // page))) + slack
        pages = B * cols + spare
        self.table = rng.permutation(pages)[:B * cols].reshape(B, cols).astype(np.int32)
        self.cache = {}
        for nm in ("k", "v"):
            self.cache[nm] = np.full((pages, Hkv, page, D), 0x7F, np.uint8)
            self.cache[nm + "_exp"] = rng.integers(0, 256, (pages, Hkv, page)).astype(np.uint8)
        for b in range(B):
            for t in range(int(self.end[b])):
                pg, o = self.table[b, t // page], t % page
                for nm in ("k", "v"):
                    c = rng.integers(0, 256, (Hkv, D)).astype(np.uint8)
                    c[(c & 0x7F) >= 0x78] ^= 0x40       # below 256, and no NaN
                    self.cache[nm][pg, :, o] = c
                    # largest code values near 240: exponents around -8 give values near 1
                    e = -8 + rng.integers(-spread, 1, Hkv)
                    self.cache[nm + "_exp"][pg, :, o] = (e + 127).astype(np.uint8)
        self.upload(dev)

    def upload(self, dev):
        self.t = {n: up(self.cache[n], dev) for n in NAMES}
        self.c = sm.KvCache.of(*[self.t[n] for n in NAMES])
        self.s = sm.KvSeqs.of(up(self.table, dev), up(self.pos, dev),
                              None if self.count is None else up(self.count, dev), N=self.N)

    def held(self):
        return {n: self.t[n].cpu().numpy() for n in NAMES}


def same_cache(got, want):
    for n in NAMES:
        if n.endswith("exp"):
            assert np.array_equal(got[n], want[n]), n
        else:
            a, b = osp.E4M3[got[n]], osp.E4M3[want[n]]
            assert np.array_equal(np.isnan(a), np.isnan(b)), n
            assert np.array_equal(got[n][~np.isnan(a)], want[n][~np.isnan(b)]), n


# ---------------------------------------------------------------------------
# append / read / commit
APPENDS = [  # pos, count, N, Hkv, D, page
    ([0], None, 1, 1, 64, 16), ([5], [1], 1, 2, 128, 16), ([15, 0, 31], [3, 0, 2], 3, 3, 64, 16),
    ([0, 127], None, 37, 2, 128, 128), ([63, 64, 65, 1], [4, 1, 4, 0], 4, 4, 128, 64),
    ([7], None, 300, 5, 64, 32)]


def rows_for(rng, shape):
    """Rows of very different magnitudes, with zeros, tiny and huge values,
    values on rounding ties, infinities and NaN."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-20, 20, shape[:-1] + (1,))
    bits = bf16_bits(x.astype(np.float32)).reshape(-1, shape[-1])
    n = len(bits)
    bits[0, :] = 0                                                  # a zero row
    bits[1 % n, :4] = [0x7F80, 0xFF80, 0x7FC0, 0x8000]              # inf, -inf, NaN, -0
    bits[2 % n, :] = bf16_bits(np.full(shape[-1], 1e-39, np.float32))    # subnormal
    bits[3 % n, 0] = 0x7F7F                                         # the largest bf16
    # ties of the grid: 1.0625 = halfway between the codes 1.0 and 1.125
    tie = np.array([448.0, 1.0625, 1.1875, -1.0625, 17.0, 2.0 ** -10, 3 * 2.0 ** -10])
    bits[4 % n, :7] = bf16_bits(tie.astype(np.float32))
    bits[5 % n, :] = 0x7FC0                                         # all NaN
    return bits.reshape(shape)


@pytest.mark.parametrize("pos,count,N,Hkv,D,page", APPENDS)
@pytest.mark.parametrize("fused", [False, True])
def test_append_then_read(pos, count, N, Hkv, D, page, fused, dev):
    rng = np.random.default_rng(100 + N)
    a = Setup(rng, dev, pos, count, N, Hkv, D, page, slack=1)
    B = len(pos)
    k, v = rows_for(rng, (B, N, Hkv, D)), rows_for(rng, (B, N, Hkv, D))
    if fused:    # parts of wider rows
        qkv = up_bf16(np.concatenate([k, v, k[:, :, :1]], 2), dev)
        kd, vd = qkv[:, :, :Hkv], qkv[:, :, Hkv:2 * Hkv]
    else:
        kd, vd = up_bf16(k, dev), up_bf16(v, dev)
    assert sm.strata_kv_append(a.c, a.s, kd, vd) == sm.STRATA_OK
    assert_device_ok()
    want = {n: x.copy() for n, x in a.cache.items()}
    osp.append(want, a.table, a.pos, a.count, k, v)
    got = a.held()
    same_cache(got, want)
    out = [torch.full((B, N, Hkv, D), -7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    assert sm.strata_kv_read(a.c, a.s, out[0], out[1]) == sm.STRATA_OK
    assert_device_ok()
    ref = osp.read(want, a.table, a.pos, a.count, N)
    n = np.full(B, N) if count is None else np.array(count)
    for o, r in zip(out, ref):
        o = bf16_to_f64(bf16_host(o))
        for b in range(B):
            assert np.all(o[b, n[b]:] == -7.0)            # slots behind the count are left alone
            x, y = o[b, :n[b]], r[b, :n[b]]
            assert np.array_equal(np.isnan(x), np.isnan(y))
            fine = ~np.isnan(y)
            # exact in bf16's normal range, half of its smallest step (2^-134) below it
            assert np.all(np.abs(x[fine] - y[fine]) <= 2.0 ** -134)


def test_read_of_one_side_and_of_empty_rows(dev):
    rng = np.random.default_rng(7)
    a = Setup(rng, dev, [3], None, 20, 2, 64, 16)
    a.cache["v_exp"][a.table[0, 1], 1, 2] = 0               # position 18, head 1 holds nothing
    a.upload(dev)
    v = torch.full((1, 20, 2, 64), -7.0, dtype=torch.bfloat16, device=dev)
    assert sm.strata_kv_read(a.c, a.s, None, v) == sm.STRATA_OK
    assert_device_ok()
    got = bf16_to_f64(bf16_host(v))
    assert np.array_equal(got, osp.read(a.cache, a.table, a.pos, None, 20)[1])
    assert np.all(got[0, 15, 1] == 0) and np.any(got[0, 15, 0] != 0)


@pytest.mark.parametrize("B,N,Hkv,D", [(3, 2, 32, 128), (2, 9, 33, 64), (2, 100, 31, 128),
                                       (1, 700, 9, 128), (1, 640, 17, 64)])
def test_append_and_read_of_many_heads(B, N, Hkv, D, dev):
    """A token's rows over one warp, or over as many as there are steps, or between."""
    rng = np.random.default_rng(Hkv)
    a = Setup(rng, dev, rng.integers(0, 40, B), rng.integers(0, N + 1, B), N, Hkv, D, 32)
    k, v = (bf16_bits(rng.standard_normal((B, N, Hkv, D)).astype(np.float32)) for _ in "kv")
    sm.check(sm.strata_kv_append(a.c, a.s, up_bf16(k, dev), up_bf16(v, dev)))
    out = [torch.full((B, N, Hkv, D), -7.0, dtype=torch.bfloat16, device=dev) for _ in "kv"]
    sm.check(sm.strata_kv_read(a.c, a.s, *out))
    assert_device_ok()
    osp.append(a.cache, a.table, a.pos, a.count, k, v)
    same_cache(a.held(), a.cache)
    for o, r in zip(out, osp.read(a.cache, a.table, a.pos, a.count, N)):
        o = bf16_to_f64(bf16_host(o))
        for b, n in enumerate(a.count):
            assert np.all(o[b, n:] == -7.0) and np.array_equal(o[b, :n], r[b, :n])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("off_k,off_v", [(0, 0), (8, 0), (0, 8), (24, 40)])
def test_read_to_outputs_on_16_byte_boundaries(D, off_k, off_v, dev):
    """Outputs that start 16 bytes behind a 32-byte boundary, and what lies
    around them is left alone."""
    a = Setup(np.random.default_rng(17), dev, [3, 40, 0], [9, 20, 0], 20, 3, D, 32)
    n = 3 * 20 * 3 * D
    flat = [torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device=dev) for _ in "kv"]
    outs = [f[o:o + n].view(3, 20, 3, D) for f, o in zip(flat, (off_k, off_v))]
    assert [o.data_ptr() % 32 for o in outs] == [2 * off_k % 32, 2 * off_v % 32]
    plain = [torch.full((3, 20, 3, D), 7.0, dtype=torch.bfloat16, device=dev) for _ in "kv"]
    sm.check(sm.strata_kv_read(a.c, a.s, *outs))
    sm.check(sm.strata_kv_read(a.c, a.s, *plain))
    assert_device_ok()
    want = osp.read(a.cache, a.table, a.pos, a.count, 20)
    for f, o, out, p, w in zip(flat, (off_k, off_v), outs, plain, want):
        assert torch.equal(out.view(torch.int16), p.view(torch.int16))
        got = bf16_to_f64(bf16_host(out))
        for b, k in enumerate(a.count):
            assert np.all(got[b, k:] == 7.0)
            assert np.array_equal(got[b, :k], np.asarray(w, np.float64)[b, :k])
        assert bool((f[:o] == 7.0).all()) and bool((f[o + n:] == 7.0).all())


def test_bad_pages_and_ranges_are_reported_and_skipped(dev):
    rng = np.random.default_rng(8)
    a = Setup(rng, dev, [10, 0, 20, -1], [8, 4, 99, 2], 8, 2, 64, 16)
    a.table[0, 1] = a.cache["k"].shape[0]                   # page out of range
    a.table[1, 0] = -1
    a.upload(dev)
    k = rows_for(rng, (4, 8, 2, 64))
    assert sm.strata_kv_append(a.c, a.s, up_bf16(k, dev), up_bf16(k, dev)) == sm.STRATA_OK
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    want = {n: x.copy() for n, x in a.cache.items()}
    osp.append(want, a.table, a.pos, a.count, k, k)
    same_cache(a.held(), want)
    # positions behind the table
    b = Setup(rng, dev, [30], None, 8, 2, 64, 16)
    b.table = b.table[:, :2].copy()
    b.upload(dev)
    k = k[:1]
    assert sm.strata_kv_append(b.c, b.s, up_bf16(k, dev), up_bf16(k, dev)) == sm.STRATA_OK
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    want = {n: x.copy() for n, x in b.cache.items()}
    osp.append(want, b.table, b.pos, None, k, k)
    same_cache(b.held(), want)
    assert sm.strata_moe_device_status() == sm.STRATA_OK


@pytest.mark.parametrize("Hkv,D,page,N", [(1, 64, 16, 1), (2, 128, 16, 8), (3, 64, 128, 64),
                                          (9, 128, 32, 33)])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(Hkv, D, page, N, in_place, dev):
    rng = np.random.default_rng(9 + N)
    pos = [0, 15, 31, 100, 7]
    a = Setup(rng, dev, pos, None, N, Hkv, D, page)
    path = np.full((5, N), -1, np.int32)
    n = np.zeros(5, np.int32)
    for b in range(5):
        keep = [0] + sorted(rng.permutation(np.arange(1, N))[:int(rng.integers(0, N))].tolist())
        if b == 1:
            keep = list(range(N))                           # nothing moves
        if b == 2:
            keep = []
        n[b] = len(keep)
        path[b, :len(keep)] = keep
    out = a.s.tensors[1] if in_place else torch.full((5,), -9, dtype=torch.int32, device=dev)
    assert sm.strata_kv_commit(a.c, a.s, up(path, dev), up(n, dev), out) == sm.STRATA_OK
    assert_device_ok()
    want = {m: x.copy() for m, x in a.cache.items()}
    new = osp.commit(want, a.table, a.pos, path, n)
    same_cache(a.held(), want)
    assert np.array_equal(out.cpu().numpy(), new)


def test_commit_reports_bad_paths(dev):
    rng = np.random.default_rng(10)
    a = Setup(rng, dev, [5, 5, 5], None, 6, 2, 64, 16)
    path = np.array([[0, 0, 5, -1, -1, -1], [0, 6, 3, -1, -1, -1], [0, 1, 2, 3, 4, 5]], np.int32)
    n = np.array([3, 3, 7], np.int32)
    out = torch.empty(3, dtype=torch.int32, device=dev)
    assert sm.strata_kv_commit(a.c, a.s, up(path, dev), up(n, dev), out) == sm.STRATA_OK
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    want = {m: x.copy() for m, x in a.cache.items()}
    new = osp.commit(want, a.table, a.pos, path, n)
    same_cache(a.held(), want)
    assert np.array_equal(out.cpu().numpy(), new)


# ---------------------------------------------------------------------------
# attention
def tree(rng, B, N, kind):
    if kind == "chain":
        return None
    p = np.full((B, N), -1, np.int32)
    for b in range(B):
        for i in range(1, N):
            p[b, i] = {"star": 0, "forest": -1}.get(kind, int(rng.integers(max(0, i - 5), i)))
    return p


def attention_bound(a, parent, q, scale):
    """(reference, bound per value), see the top of the file."""
    ref = osp.tree_attention(a.cache, a.table, a.pos, a.count, parent, q, scale)
    sc = 1.0 / np.sqrt(a.D) if scale is None else scale
    B, N, Hq, D = q.shape
    qf = np.abs(bf16_to_f64(q))
    bound = np.zeros_like(ref)
    for b, p, n in osp._ranges(a.table, a.pos, a.count, N):
        for hk in range(a.Hkv):
            ats = [osp._at(a.cache, a.table, b, t) for t in range(p + n)]
            ks = [osp.row(a.cache, "k", t, hk) for t in ats if t is not None]
            vs = [osp.row(a.cache, "v", t, hk) for t in ats if t is not None]
            ks = np.nan_to_num(np.abs([x for x in ks if x is not None])).reshape(-1, D)
            vs = np.nan_to_num(np.abs([x for x in vs if x is not None])).reshape(-1, D)
            if not len(ks):
                continue
            for h in range(hk * (Hq // a.Hkv), (hk + 1) * (Hq // a.Hkv)):
                x = qf[b, :n, h]
                ds = sc * np.max(D * 2.0 ** -24 * (x @ ks.T)
                                 + 2.0 ** -17 * x.max(-1)[:, None] * ks.sum(-1), axis=-1)
                A = vs.max(0)[None, :]                       # at least sum p |v| / sum p
                bound[b, :n, h] = (2.0 ** -8 * np.abs(np.nan_to_num(ref[b, :n, h]))
                                   + A * (2.0 ** -9 + 2.0 ** -11 + 2.5 * ds[:, None])
                                   + 2.0 ** -8.8 * vs.max(initial=0.0))
    return ref, bound


def run_attention(a, parent, q, dev, scale=None, fill=-7.0, stream=None, out=None):
    B, N, Hq, D = q.shape
    out = torch.full((B, N, Hq, D), fill, dtype=torch.bfloat16, device=dev) if out is None else out
    ws = sm.tree_attention_workspace(a.c, a.s, Hq, dev)
    ws.fill_(0xFF)                    # what a workspace held before does not matter
    st = sm.strata_tree_attention(a.c, a.s, None if parent is None else up(parent, dev),
                                  up_bf16(q, dev), 0.0 if scale is None else scale, out, ws,
                                  stream=stream)
    assert st == sm.STRATA_OK
    return out


def check_attention(a, parent, q, out, scale=None):
    ref, bound = attention_bound(a, parent, q, scale)
    got = bf16_to_f64(bf16_host(out))
    unread = np.isnan(ref).all(-1) & (got == -7.0).all(-1)
    B, N = q.shape[:2]
    n = np.full(B, N) if a.count is None else a.count
    for b in range(B):
        live = max(0, min(int(n[b]), N)) if 0 <= n[b] <= N and a.pos[b] >= 0 else 0
        assert unread[b, live:].all(), "a slot behind the count was written"
        x, y, e = got[b, :live], ref[b, :live], bound[b, :live]
        assert np.array_equal(np.isnan(x), np.isnan(y)), f"sequence {b}"
        fine = ~np.isnan(y)
        off = np.abs(x[fine] - y[fine]) - e[fine]
        assert np.all(off <= 0), f"sequence {b}: {np.max(off)} above the bound"
    fine = ~np.isnan(ref)
    if fine.any() and np.linalg.norm(ref[fine]) > 0:
        rel = np.linalg.norm((got - ref)[fine]) / np.linalg.norm(ref[fine])
        print(f"relative error {rel:.2e}")
        # bf16's rounding is 2^-8 at most; the weights' (independent over the
        # positions) adds 2^-9 at most
        assert rel <= 2.0 ** -8 + 2.0 ** -9
    return got


ATTEND = [  # pos, count, N, Hq, Hkv, D, page, kind
    ([0], None, 1, 1, 1, 64, 16, "chain"),
    ([0], None, 1, 4, 2, 128, 16, "chain"),
    ([1, 0, 15, 16, 17], None, 1, 8, 1, 128, 16, "chain"),
    ([126, 127, 128, 129], None, 1, 8, 4, 128, 64, "chain"),
    ([126, 124, 128, 300], None, 4, 8, 1, 128, 32, "chain"),
    ([0, 60, 130], None, 64, 2, 2, 64, 16, "tree"),
    ([100, 3], None, 64, 16, 1, 128, 128, "tree"),
    ([255, 256, 257, 64, 0], [5, 0, 1, 3, 4], 5, 6, 2, 128, 64, "tree"),
    ([40, 700], None, 9, 48, 3, 64, 32, "star"),
    ([513, 1000], None, 3, 64, 1, 128, 16, "forest"),
    ([33], None, 2, 5, 5, 128, 128, "chain"),
    ([1500, 20], None, 7, 7, 1, 64, 64, "tree"),
    ([4000, 10, 0], [16, 16, 2], 16, 16, 2, 128, 64, "tree"),
    ([0, 300, 7], [0, 0, 0], 4, 8, 2, 128, 16, "chain"),                    # nothing to do
    ([300, 40, 0, 511, 512, 513, 9, 70] * 12, [2, 0, 1, 2, 1, 0, 2, 1] * 12, 2, 3, 3, 64, 16,
     "forest"),                                                             # 96 short sequences
    ([2047, 2048, 255, 256, 257, 1], None, 1, 64, 4, 64, 128, "chain"),     # ends at tile edges
    ([190], None, 64, 64, 1, 64, 32, "tree"),                               # 4096 rows
    ([9000, 1], [1, 33], 33, 4, 4, 64, 16, "tree"),                         # one long, one short
]


@pytest.mark.parametrize("pos,count,N,Hq,Hkv,D,page,kind", ATTEND)
def test_attention(pos, count, N, Hq, Hkv, D, page, kind, dev):
    rng = np.random.default_rng(1000 + N + Hq)
    a = Setup(rng, dev, pos, count, N, Hkv, D, page, slack=1)
    q = bf16_bits(rng.standard_normal((len(pos), N, Hq, D)).astype(np.float32))
    parent = tree(rng, len(pos), N, kind)
    out = run_attention(a, parent, q, dev)
    assert_device_ok()
    check_attention(a, parent, q, out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("std,scale", [(30.0, None), (1e-3, None), (1.0, 2.0), (1e20, 1e-21),
                                       (1e-30, 1e30)])
def test_attention_of_sharp_flat_and_extreme_scores(D, std, scale, dev):
    """Scores from nearly one-hot to nearly equal, rows of q whose magnitudes
    differ, values of V of very different scales."""
    rng = np.random.default_rng(77)
    a = Setup(rng, dev, [700, 90], None, 5, 2, D, 32, spread=9)
    q = rng.standard_normal((2, 5, 8, D)) * std * 2.0 ** rng.integers(-6, 1, (2, 5, 8, 1))
    q = bf16_bits(q.astype(np.float32))
    out = run_attention(a, None, q, dev, scale)
    assert_device_ok()
    check_attention(a, None, q, out, scale)


def test_attention_nan_stays_where_it_is_seen(dev):
    """NaN in a sibling's K or V reaches neither the other branches nor the
    positions before it; where it is seen it comes out (V: in its dimension)."""
    rng = np.random.default_rng(78)
    a = Setup(rng, dev, [130, 5, 50], None, 6, 2, 128, 16)
    parent = np.array([[-1, 0, 0, 1, 2, 3]] * 3, np.int32)

    def at(b, i):
        t = int(a.pos[b]) + i
        return a.table[b, t // 16], t % 16
    pg, o = at(0, 1)
    a.cache["v"][pg, 0, o, 7] = 0x7F           # seen by nodes 1, 3, 5 of sequence 0, head 0
    pg, o = at(1, 2)
    a.cache["k"][pg, 1, o, 3] = 0xFF           # seen by nodes 2 and 4 of sequence 1, head 1
    a.cache["v"][a.table[2, 0], 0, 9, 100] = 0xFF     # a committed position: seen by all
    a.upload(dev)
    q = bf16_bits(rng.standard_normal((3, 6, 8, 128)).astype(np.float32))
    out = run_attention(a, parent, q, dev)
    assert_device_ok()
    got = check_attention(a, parent, q, out)
    assert np.isnan(got[0, 1, :4, 7]).all() and not np.isnan(got[0, 2]).any()
    assert np.isnan(got[1, 4, 4:]).all() and not np.isnan(got[1, 3]).any()
    assert np.isnan(got[2, :, :4, 100]).all() and not np.isnan(got[2, :, 4:]).any()


def test_attention_nan_and_infinite_queries_stay_in_their_rows(dev):
    rng = np.random.default_rng(79)
    a = Setup(rng, dev, [200], None, 4, 2, 64, 16)
    q = bf16_bits(rng.standard_normal((1, 4, 8, 64)).astype(np.float32))
    q[0, 1, 2, 5] = 0x7FC0
    q[0, 3, 6, 0] = 0x7F80
    out = bf16_to_f64(bf16_host(run_attention(a, None, q, dev)))
    assert_device_ok()
    assert np.isnan(out[0, 1, 2]).all() and np.isnan(out[0, 3, 6]).all()
    out[0, 1, 2] = out[0, 3, 6] = 0
    assert not np.isnan(out).any()


def test_attention_passes_over_empty_rows_and_bad_pages(dev):
    rng = np.random.default_rng(80)
    a = Setup(rng, dev, [300, 40, 0, 5], None, 3, 2, 128, 32)
    a.cache["k_exp"][a.table[0, 2], 0, 5:20] = 0            # rows that hold nothing
    a.cache["k_exp"][a.table[2, 0], :, :3] = 0              # all that sequence 2 would see
    a.upload(dev)
    q = bf16_bits(rng.standard_normal((4, 3, 4, 128)).astype(np.float32))
    out = run_attention(a, None, q, dev)
    assert_device_ok()
    got = check_attention(a, None, q, out)
    assert np.all(got[2] == 0)
    a.table[0, 4] = a.cache["k"].shape[0] + 5
    a.table[1, 0] = -3
    a.table[3, 0] = 1 << 30                                 # sequence 3 sees nothing
    a.upload(dev)
    out = run_attention(a, None, q, dev)
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    got = check_attention(a, None, q, out)
    assert np.all(got[3] == 0)


def test_attention_reports_bad_parents_counts_and_ends(dev):
    rng = np.random.default_rng(81)
    a = Setup(rng, dev, [30, 30, -2, 30], [4, 4, 4, 5], 4, 2, 64, 16)
    parent = np.array([[-1, 0, 5, 2], [0, -7, 1, 2], [-1, 0, 1, 2], [-1, 0, 1, 2]], np.int32)
    q = bf16_bits(rng.standard_normal((4, 4, 4, 64)).astype(np.float32))
    out = run_attention(a, parent, q, dev)
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    fixed = parent.copy()
    fixed[0, 2] = fixed[1, 0] = fixed[1, 1] = -1
    check_attention(a, fixed, q, out)
    # more positions than the table has columns for
    b = Setup(rng, dev, [30], None, 4, 2, 64, 16)
    b.table = b.table[:, :2].copy()
    b.upload(dev)
    out = run_attention(b, None, q[:1], dev)
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    check_attention(b, None, q[:1], out)


def test_attention_is_the_same_every_time_on_any_stream_and_replayed(dev):
    """Bit-identical over repeats, two calls at once on two streams, and a
    captured call replayed after the lengths and the cache changed."""
    rng = np.random.default_rng(82)
    a = Setup(rng, dev, [900, 333], None, 4, 2, 128, 64)
    b = Setup(rng, dev, [50, 777], None, 4, 2, 128, 64)
    q = bf16_bits(rng.standard_normal((2, 4, 16, 128)).astype(np.float32))
    first = {id(x): run_attention(x, None, q, dev) for x in (a, b)}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    outs = []
    for _ in range(5):
        for x, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                outs.append((id(x), run_attention(x, None, q, dev)))
    torch.cuda.synchronize()
    for key, o in outs:
        assert torch.equal(o, first[key])
    # captured
    ws = sm.tree_attention_workspace(a.c, a.s, 16, dev)
    out = torch.zeros((2, 4, 16, 128), dtype=torch.bfloat16, device=dev)
    qd = up_bf16(q, dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sm.check(sm.strata_tree_attention(a.c, a.s, None, qd, 0.0, out, ws))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[id(a)])
    a.pos[:] = [17, 620]
    a.s.tensors[1].copy_(up(a.pos, dev))
    out.fill_(-7.0)
    g.replay()
    assert_device_ok()
    check_attention(a, None, q, out)


def test_attention_takes_parts_of_wider_query_rows(dev):
    rng = np.random.default_rng(83)
    a = Setup(rng, dev, [70, 3], None, 3, 2, 64, 16)
    q = bf16_bits(rng.standard_normal((2, 3, 6, 64)).astype(np.float32))
    wide = up_bf16(np.concatenate([q[:, :, :2], q], 2), dev)
    out = torch.full((2, 3, 6, 64), -7.0, dtype=torch.bfloat16, device=dev)
    ws = sm.tree_attention_workspace(a.c, a.s, 6, dev)
    assert sm.strata_tree_attention(a.c, a.s, None, wide[:, :, 2:], 0.0, out, ws) == sm.STRATA_OK
    assert_device_ok()
    check_attention(a, None, q, out)


def test_binding_refuses_other_types_shapes_and_layouts(dev):
    rng = np.random.default_rng(84)
    a = Setup(rng, dev, [7, 3], None, 3, 2, 64, 16)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device=dev)
    ws = sm.tree_attention_workspace(a.c, a.s, 4, dev)
    par = torch.full((2, 3), -1, dtype=torch.int32, device=dev)
    call = lambda **k: sm.strata_tree_attention(  # noqa: E731
        a.c, a.s, k.get("parent", par), k.get("q", q), 0.0, k.get("out", q.clone()),
        k.get("ws", ws))
    assert call() == sm.STRATA_OK
    for bad in (dict(q=q.half()), dict(q=q[:, :2]), dict(q=q.transpose(1, 2)),
                dict(q=q[..., :32]), dict(out=q.float()), dict(out=q[:, :, :2]),
                dict(parent=par.long()), dict(parent=par[:, :2]), dict(out=q.transpose(2, 3)),
                dict(q=q[0])):
        assert call(**bad) == sm.STRATA_ERR_INVALID_ARG, list(bad)
    assert call(ws=ws[:-16]) == sm.STRATA_ERR_WORKSPACE
    x = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16, device=dev)
    wide = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device=dev)
    assert sm.strata_kv_append(a.c, a.s, x, x.float()) == sm.STRATA_ERR_INVALID_ARG
    assert sm.strata_kv_append(a.c, a.s, x, wide[:, :, :2]) == sm.STRATA_ERR_INVALID_ARG
    assert sm.strata_kv_append(a.c, a.s, wide[:, :, ::2], wide[:, :, ::2]) \
        == sm.STRATA_ERR_INVALID_ARG
    assert sm.strata_kv_read(a.c, a.s, x, wide) == sm.STRATA_ERR_INVALID_ARG
    with pytest.raises(sm.StrataError):
        sm.KvCache.of(a.t["k"], a.t["v"][:1], a.t["k_exp"], a.t["v_exp"])
    assert_device_ok()


def test_cache_of_more_than_four_gib(dev):
    """Rows past 2^32 bytes of codes: appended, read, attended to and moved."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of free device memory")
    pages, page, Hkv, D = 40000, 128, 8, 128                       # 5.2 GB of K, and of V
    c = sm.KvCache.empty(pages, page, Hkv, D, dev)
    rng = np.random.default_rng(90)
    table = np.array([[39999, 5, 39000], [33000, 39998, 7]], np.int32)
    pos, N, Hq = np.array([0, 0], np.int32), 300, 8
    s = sm.KvSeqs.of(up(table, dev), up(pos, dev), N=N)
    k, v = (bf16_bits(rng.standard_normal((2, N, Hkv, D)).astype(np.float32)) for _ in "kv")
    sm.check(sm.strata_kv_append(c, s, up_bf16(k, dev), up_bf16(v, dev)))
    out = [torch.empty((2, N, Hkv, D), dtype=torch.bfloat16, device=dev) for _ in "kv"]
    sm.check(sm.strata_kv_read(c, s, *out))
    assert_device_ok()
    # the same through a small cache
    small = Setup(rng, dev, pos, None, N, Hkv, D, page)
    osp.append(small.cache, small.table, pos, None, k, v)
    ref = osp.read(small.cache, small.table, pos, None, N)
    for o, r in zip(out, ref):
        assert np.array_equal(bf16_to_f64(bf16_host(o)), r)
    n = 8
    at = np.array([N - n, N - n - 40], np.int32)
    q = bf16_bits(rng.standard_normal((2, n, Hq, D)).astype(np.float32))
    small.pos, small.N = at, n
    small.count = None
    small.upload(dev)
    t = sm.KvSeqs.of(up(table, dev), up(at, dev), N=n)
    big = torch.full((2, n, Hq, D), -7.0, dtype=torch.bfloat16, device=dev)
    ws = sm.tree_attention_workspace(c, t, Hq, dev)
    sm.check(sm.strata_tree_attention(c, t, None, up_bf16(q, dev), 0.0, big, ws))
    assert_device_ok()
    check_attention(small, None, q, big)
    path = np.array([[0, 3, 4, 7, -1, -1, -1, -1], [0, 1, 2, 6, -1, -1, -1, -1]], np.int32)
    new = torch.zeros(2, dtype=torch.int32, device=dev)
    sm.check(sm.strata_kv_commit(c, t, up(path, dev), up(np.array([4, 4], np.int32), dev), new))
    osp.commit(small.cache, small.table, at, path, np.array([4, 4]))
    sm.check(sm.strata_kv_read(c, s, *out))
    assert_device_ok()
    for o, r in zip(out, osp.read(small.cache, small.table, pos, None, N)):
        assert np.array_equal(bf16_to_f64(bf16_host(o)), r)
    assert new.cpu().tolist() == (at + 4).tolist()


def test_attention_with_a_huge_value_at_a_hidden_sibling(dev):
    """A sibling's V far larger than all others takes nothing from the rows that
    do not see it; a large committed value beside small ones keeps the bound."""
    rng = np.random.default_rng(91)
    a = Setup(rng, dev, [200], None, 6, 2, 128, 16)
    parent = np.array([[-1, 0, 0, 1, 2, 3]], np.int32)
    t = 201                                          # node 1: not seen by 0, 2 and 4
    a.cache["v_exp"][a.table[0, t // 16], :, t % 16] = 127 + 90
    a.upload(dev)
    q = bf16_bits(rng.standard_normal((1, 6, 8, 128)).astype(np.float32))
    out = run_attention(a, parent, q, dev)
    assert_device_ok()
    got = bf16_to_f64(bf16_host(out))
    ref, bound = attention_bound(a, parent, q, None)
    for i in (0, 2, 4):                              # the bound without the sibling's V
        keep = a.cache["v_exp"].copy()
        a.cache["v_exp"][a.table[0, t // 16], :, t % 16] = 119
        _, fine = attention_bound(a, parent, q, None)
        a.cache["v_exp"] = keep
        assert np.all(np.abs(got[0, i] - ref[0, i]) <= fine[0, i])
    assert np.all(np.abs(got - ref) <= bound)


def test_attention_keeps_a_sink_and_a_long_tail_apart(dev):
    """One position with almost all the weight and thousands of small equal ones: the
    tail's share of the output (about a quarter) is not lost to the weights' floor."""
    D, n = 64, 6000
    c = sm.KvCache.empty(400, 16, 1, D, dev)
    k = np.zeros((1, n, 1, D), np.float32)
    v = np.zeros((1, n, 1, D), np.float32)
    k[0, 0, 0, 0] = 1.0
    v[0, 0, 0, 0] = 1.0
    v[0, 1:, 0, 1] = 1.0
    s = sm.KvSeqs.of(torch.arange(400, dtype=torch.int32, device=dev).view(1, 400),
                     torch.zeros(1, dtype=torch.int32, device=dev), N=n)
    sm.check(sm.strata_kv_append(c, s, up_bf16(bf16_bits(k), dev), up_bf16(bf16_bits(v), dev)))
    t = sm.KvSeqs.of(s.tensors[0], torch.full((1,), n - 1, dtype=torch.int32, device=dev), N=1)
    q = np.zeros((1, 1, 1, D), np.float32)
    q[..., 0] = 1.0
    out = torch.zeros((1, 1, 1, D), dtype=torch.bfloat16, device=dev)
    ws = sm.tree_attention_workspace(c, t, 1, dev)
    scale = float(np.log(3.0 * (n - 1)))             # the sink weighs three times the tail
    sm.check(sm.strata_tree_attention(c, t, None, up_bf16(bf16_bits(q), dev), scale, out, ws))
    assert_device_ok()
    got = bf16_to_f64(bf16_host(out))[0, 0, 0]
    # every weight is off by 2^-9 at most (a tail tile's own largest is the tail's
    # weight; beside the sink 255 tail positions keep 2^-17.8 of it each), bf16 2^-8
    off = 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -11 + 255 * 2.0 ** -17.8
    assert abs(got[0] - 0.75) <= 0.75 * off and abs(got[1] - 0.25) <= 0.25 * (2.0 ** -8 + 2.0 ** -9
                                                                          + 2.0 ** -11) + 255 * 2.0 ** -17.8


def test_attention_of_positions_behind_the_page_table(dev):
    """A committed length past the table's room: what has a column is attended to,
    the rest (the nodes too) reported and passed over."""
    rng = np.random.default_rng(92)
    a = Setup(rng, dev, [48, 512, 300], None, 2, 2, 64, 16)
    a.table = a.table[:, :3].copy()                  # room for 48 positions
    a.pos = np.array([48, 1000, 40], np.int32)
    a.upload(dev)
    q = bf16_bits(rng.standard_normal((3, 2, 4, 64)).astype(np.float32))
    out = run_attention(a, None, q, dev)
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    check_attention(a, None, q, out)


def test_attention_of_thousands_of_short_sequences(dev):
    rng = np.random.default_rng(93)
    B = 3000
    pos = rng.integers(0, 3, B)
    count = rng.integers(0, 3, B)
    a = Setup(rng, dev, pos, count, 2, 1, 64, 16)
    q = bf16_bits(rng.standard_normal((B, 2, 2, 64)).astype(np.float32))
    out = run_attention(a, None, q, dev)
    assert_device_ok()
    check_attention(a, None, q, out)


def test_attention_in_place_and_with_shared_pages(dev):
    """Two sequences that share their first pages, and the output written over the
    queries."""
    rng = np.random.default_rng(94)
    a = Setup(rng, dev, [600, 600], None, 4, 2, 128, 32)
    a.table[1, :18] = a.table[0, :18]                # positions below 576 are the same
    a.upload(dev)
    q = bf16_bits(rng.standard_normal((2, 4, 8, 128)).astype(np.float32))
    out = run_attention(a, None, q, dev)
    same = up_bf16(q, dev)
    ws = sm.tree_attention_workspace(a.c, a.s, 8, dev)
    sm.check(sm.strata_tree_attention(a.c, a.s, None, same, 0.0, same, ws))
    assert_device_ok()
    check_attention(a, None, q, out)
    assert torch.equal(same, out)


def test_one_workspace_for_two_captured_calls(dev):
    rng = np.random.default_rng(95)
    a = Setup(rng, dev, [700, 10], None, 3, 2, 64, 16)
    b = Setup(rng, dev, [5, 1200], None, 3, 2, 64, 16)
    q = bf16_bits(rng.standard_normal((2, 3, 8, 64)).astype(np.float32))
    want = [run_attention(x, None, q, dev) for x in (a, b)]
    ws = torch.empty(max(sm.strata_tree_attention_workspace_bytes(x.c, x.s, 8) for x in (a, b)),
                     dtype=torch.uint8, device=dev)
    qd, outs, graphs = up_bf16(q, dev), [torch.zeros_like(w) for w in want], []
    for x, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sm.check(sm.strata_tree_attention(x.c, x.s, None, qd, 0.0, o, ws))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])
