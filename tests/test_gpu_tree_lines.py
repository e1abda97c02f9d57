"""The tree attention where every CTA works through many tiles and units (rings that
wrap, running maxima that move, units cut in two by the runs), for every block size
and head size, against fp64 with the bars of tree_bars.py: per sequence and per row."""

import numpy as np
import pytest
import torch

import local_moe_route_b200 as sm
from gpu_helpers import assert_device_ok
from moe_inputs import bf16_bits
from test_gpu_kv import ATTEND, NAMES, Setup, run_attention, tree, up
from tree_bars import Bars
from tree_lines import CASES, Line

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_dev):
    from local_moe_route_b200 import build
    build.build()
    return cuda_dev


def upload(a, dev):
    a.c = sm.KvCache.of(*[up(a.cache[n], dev) for n in NAMES])
    a.s = sm.KvSeqs.of(up(a.table, dev), up(a.pos, dev), up(a.count, dev), N=a.N)


def check(a, parent, q, out, dev):
    bars = Bars(a.cache, a.table, a.pos, a.count, parent, q, None, dev)
    faults = bars.faults(out.double())
    assert not faults, faults
    unread = bars.ref.isnan()
    assert bool((out[unread] == -7.0).all()), "a slot behind the count was written"
    if not bool(unread.all()):
        print(f"largest row error {bars.share(out.double()):.2f} of its bound")


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("name", list(CASES))
def test_lines(name, seed, dev):
    a = Line(name, seed)
    upload(a, dev)
    out = run_attention(a, a.parent, a.q, dev)
    bad = a.bad_pages and any(a.count[1::5] > 0)
    assert sm.strata_moe_device_status() == (sm.STRATA_ERR_DEVICE_CHECK if bad else sm.STRATA_OK)
    check(a, a.parent, a.q, out, dev)
    again = run_attention(a, a.parent, a.q, dev)
    torch.cuda.synchronize()
    sm.strata_moe_device_status()
    assert torch.equal(out, again)


@pytest.mark.parametrize("name", ["chain4_D128", "many_forest_D64"])
def test_lines_of_changing_lengths_from_one_graph(name, dev):
    """One captured call replayed over lengths, counts and tables that change between
    the replays: another cut of the line every time, the workspace left as it was."""
    a = Line(name)
    upload(a, dev)
    ws = sm.tree_attention_workspace(a.c, a.s, a.Hq, dev)
    q = up(a.q.view(np.int16), dev).view(torch.bfloat16)
    par = None if a.parent is None else up(a.parent, dev)
    out = torch.full(a.q.shape, -7.0, dtype=torch.bfloat16, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sm.check(sm.strata_tree_attention(a.c, a.s, par, q, 0.0, out, ws))
    rng = np.random.default_rng(40)
    most = int(a.pos.max())
    for step in range(4):
        if step:
            a.pos[:] = rng.integers(0, [most + 1, 40, 700][step - 1], len(a.pos))
            a.count[:] = rng.integers(0, a.N + 1, len(a.pos))
            a.table[:] = rng.permuted(a.table, axis=1)
            for t, x in zip(a.s.tensors, (a.table, a.pos, a.count)):
                t.copy_(up(x, dev))
        out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        sm.strata_moe_device_status()
        check(a, a.parent, a.q, out, dev)


@pytest.mark.parametrize("pos,count,N,Hq,Hkv,D,page,kind", ATTEND)
def test_small_cases_sequence_by_sequence(pos, count, N, Hq, Hkv, D, page, kind, dev):
    rng = np.random.default_rng(1000 + N + Hq)
    a = Setup(rng, dev, pos, count, N, Hkv, D, page, slack=1)
    q = bf16_bits(rng.standard_normal((len(pos), N, Hq, D)).astype(np.float32))
    parent = tree(rng, len(pos), N, kind)
    out = run_attention(a, parent, q, dev)
    assert_device_ok()
    check(a, parent, q, out, dev)
