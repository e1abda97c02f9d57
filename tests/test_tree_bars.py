"""The bars of the tree attention (tree_bars.py) let the exact result through, rounded
as the kernel may round it, and notice results that are wrong: a sequence of zeros, a
tile or a page that is left out or counts twice, half of the positions lost."""

import numpy as np
import pytest
import torch

from moe_inputs import bf16_bits
from oracle import speculative as osp
from tree_bars import Bars
from tree_lines import CASES, Line, tiles

CTAS = 296


def test_the_cases_fill_the_gpu():
    """More than four and more than sixteen tiles per CTA in every kind of kernel (blocks
    of 16 or 32 rows, D = 64 or 128), and more than four units per CTA."""
    most = {}
    for name, (B, N, Hq, Hkv, D, *_) in CASES.items():
        a = Line(name)
        n = tiles(name, a.pos, a.count)
        assert n > CTAS, name
        kind = (D, 16 if N * Hq // Hkv <= 16 else 32)
        most.setdefault(kind, []).append(n / CTAS)
    assert sorted(most) == [(64, 16), (64, 32), (128, 16), (128, 32)]
    for kind, n in most.items():
        assert max(n) > 16, (kind, n)
    assert any(4 < x < 16 for n in most.values() for x in n)


def live(a):
    return [b for b in range(len(a.pos)) if a.count[b] > 0]


@pytest.mark.parametrize("name", list(CASES))
def test_lines(name):
    a = Line(name)
    alive = live(a)
    longest = max(alive, key=lambda b: int(a.pos[b]))
    some = [longest] + [b for b in alive if b != longest][:2]
    for b in some:
        args = (a.cache, a.table, a.pos, a.count, a.parent, a.q)
        bars = Bars(*args, only=[b])
        exact = bars.ref
        assert not bars.faults(exact.bfloat16().double())
        end = int(a.pos[b] + a.count[b])
        bad = exact.clone()
        bad[b] = 0
        assert bars.faults(bad)
        lost = {"half": range(0, end, 2)}
        # the tile and the page with the most weight on them: its values say so, the
        # output moves most without them
        for what, size in (("tile", 256), ("page", a.page)):
            starts = list(range(0, end, size))
            if len(starts) < 2:
                continue
            step = max(1, len(starts) // 8)
            far = [(float((Bars(*args, only=[b], drop={b: list(range(s, s + size))}).ref
                           - exact)[b].nan_to_num().norm()), s) for s in starts[::step]]
            s = max(far)[1]
            lost[what] = range(s, s + size)
        for what, ts in lost.items():
            ts = list(ts)
            assert bars.faults(Bars(*args, only=[b], drop={b: ts}).ref), (b, what)
            if what != "half":
                assert bars.faults(Bars(*args, only=[b], twice={b: ts}).ref), (b, what)


def test_the_reference_is_the_oracles():
    rng = np.random.default_rng(3)
    for D, parent in ((64, None), (128, np.array([[-1, 0, 0, 1]] * 2, np.int32))):
        cache = {n: rng.integers(0, 0x77, (6, 2, 16, D)).astype(np.uint8) for n in "kv"}
        for n in "kv":
            cache[n + "_exp"] = rng.integers(110, 121, (6, 2, 16)).astype(np.uint8)
        cache["k_exp"][1, 0, 3:9] = 0
        cache["v_exp"][2, 1, 3:9] = 0
        table = np.array([[0, 1, 2], [4, -1, 5]], np.int32)
        pos, count = np.array([30, 40], np.int32), np.array([4, 3], np.int32)
        q = bf16_bits(rng.standard_normal((2, 4, 6, D)).astype(np.float32))
        bars = Bars(cache, table, pos, count, parent, q)
        ref = osp.tree_attention(cache, table, pos, count, parent, q)
        got = bars.ref.numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        fine = ~np.isnan(ref)
        assert np.allclose(got[fine], ref[fine], rtol=1e-12, atol=1e-15)
        assert not bars.faults(torch.from_numpy(ref).bfloat16().double())
