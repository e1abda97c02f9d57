"""Tree attention at the edges of what its inputs may hold, against the fp64 oracle
(the bars are those of test_gpu_kv.py unless a test says otherwise)."""

import numpy as np
import pytest

import local_moe_route_b200 as sm
from gpu_helpers import assert_device_ok, bf16_host, bf16_to_f64
from moe_inputs import bf16_bits
from oracle import speculative as osp
from test_gpu_kv import Setup, check_attention, run_attention
from tree_bars import Bars

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_dev):
    from local_moe_route_b200 import build
    build.build()
    return cuda_dev


@pytest.mark.parametrize("D,G", [(64, 1), (64, 8), (128, 2), (128, 9)])
def test_a_node_that_sees_nothing_gets_zeros_whatever_its_query_is(D, G, dev):
    """NaN and infinite queries of nodes that see no row (every page out of range, or
    every row empty, over one tile and over several), beside ones that see some."""
    rng = np.random.default_rng(200 + D + G)
    a = Setup(rng, dev, [700, 5, 900, 40, 600], None, 4, 2, D, 32)
    a.table[0, :] = -1                                       # nothing, over three tiles
    a.table[1, :] = a.cache["k"].shape[0]                    # nothing, in one
    for pg in a.table[3]:
        a.cache["k_exp"][pg] = 0                             # rows that hold nothing
    a.table[4, :18] = -1                                     # a few positions at the end
    a.upload(dev)
    q = bf16_bits(rng.standard_normal((5, 4, 2 * G, D)).astype(np.float32))
    q[:, 0, 0, 3] = 0x7FC0
    q[:, 1, -1, D - 1] = 0x7F80
    q[:, 3, 0, :] = 0xFF80
    out = run_attention(a, None, q, dev)
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    got = check_attention(a, None, q, out)
    for b in (0, 1, 3):
        assert np.all(got[b] == 0)
    for b in (2, 4):
        assert np.isnan(got[b, 0, 0]).all() and np.isnan(got[b, 1, -1]).all()
        assert not np.isnan(got[b, 2]).any()


def check_bars(a, parent, q, out, dev, scale=None):
    bars = Bars(a.cache, a.table, a.pos, a.count, parent, q, scale, dev)
    assert not bars.faults(out.double()), bars.faults(out.double())
    print(f"largest row error {bars.share(out.double()):.2f} of its bound")


def far_away(a, q, b, ts):
    """Makes positions ts of sequence b ones that no query gives weight to: K far from
    every query in dimension 0, where q is positive and the other K rows are 0."""
    q[b, ..., 0] = bf16_bits(np.full(q.shape[1:3], 8.0, np.float32))
    for pg in a.table[b]:
        a.cache["k"][pg, :, :, 0] = 0
    for t in ts:
        pg, o = a.table[b, t // a.page], t % a.page
        a.cache["k"][pg, :, o, 0] = 0xFE                 # -448
        a.cache["k_exp"][pg, :, o] = 127 - 3             # -56: scores around -40 (D = 128)


@pytest.mark.parametrize("ratio", [0, 6, 10, 14, 18, 29, 30, 31, 40, 80])
@pytest.mark.parametrize("D,Hq", [(128, 4), (64, 16)])
def test_a_large_value_without_weight_takes_nothing_from_the_others(D, Hq, ratio, dev):
    """One committed V row 2^ratio above the others which every row sees and none gives
    weight to (2^-58 and less): the others keep their precision.  (Above 2^30 the sum of
    the weights has a reference of its own.)"""
    rng = np.random.default_rng(300 + ratio)
    a = Setup(rng, dev, [250, 1000], None, 2, 2, D, 32, spread=1)
    q = bf16_bits(rng.standard_normal((2, 2, Hq, D)).astype(np.float32))
    for b, ts in ((0, [77]), (1, [300, 999])):
        far_away(a, q, b, ts)
        for t in ts:
            a.cache["v_exp"][a.table[b, t // 32], :, t % 32] = 127 - 8 + ratio
    a.upload(dev)
    out = run_attention(a, None, q, dev)
    assert_device_ok()
    if ratio <= 40:                     # (2^-58 of 2^80 is what the output consists of)
        got, ref = bf16_to_f64(bf16_host(out)), osp.tree_attention(a.cache, a.table, a.pos, None,
                                                                   None, q)
        assert np.linalg.norm(got - ref) <= (2.0 ** -8 + 2.0 ** -9) * np.linalg.norm(ref)
    check_bars(a, None, q, out, dev)


@pytest.mark.parametrize("small", [4, 12, 24, 40, 90])
@pytest.mark.parametrize("D", [64, 128])
def test_a_sink_with_small_values_leaves_the_tail_its_weights(D, small, dev):
    """A position with nearly all the weight and V rows 2^-small of the others (0: V
    rows of zeros, as appended), beside positions of the same tile that carry the output."""
    rng = np.random.default_rng(310 + small)
    a = Setup(rng, dev, [400, 40], None, 3, 2, D, 16, spread=2)
    q = rng.standard_normal((2, 3, 8, D)).astype(np.float32)
    q[..., 0] = 6.0
    q = bf16_bits(q)
    for b in range(2):
        for pg in a.table[b]:
            a.cache["k"][pg, :, :, 0] = 0
        pg = a.table[b, 0]
        a.cache["k"][pg, :, 1, 0] = 0x7E                 # 448 * 2^-4: score 21 at D = 64
        a.cache["k_exp"][pg, :, 1] = 127 - 4
        a.cache["v_exp"][pg, :, 1] = 127 - 8 - small
        if small == 90:
            a.cache["v"][pg, :, 1] = 0                   # as a row of zeros is appended
            a.cache["v_exp"][pg, :, 1] = 1
    a.upload(dev)
    out = run_attention(a, None, q, dev)
    assert_device_ok()
    check_bars(a, None, q, out, dev)


def test_values_of_every_magnitude(dev):
    """V rows from 2^-60 to 2^60 in one tile, huge ones at siblings, empty V rows."""
    rng = np.random.default_rng(320)
    a = Setup(rng, dev, [500, 20], None, 6, 2, 128, 16)
    parent = np.array([[-1, 0, 0, 1, 2, 3]] * 2, np.int32)
    e = a.cache["v_exp"]
    e[:] = rng.integers(127 - 60, 127 + 61, e.shape)
    e[a.table[0, 0], :, 3] = 0                               # no V, but a K
    for b in range(2):
        t = int(a.pos[b]) + 1
        e[a.table[b, t // 16], :, t % 16] = 127 + 85         # node 1: 0, 2 and 4 do not see it
    a.upload(dev)
    q = bf16_bits((3 * rng.standard_normal((2, 6, 8, 128))).astype(np.float32))
    out = run_attention(a, parent, q, dev)
    assert_device_ok()
    check_bars(a, parent, q, out, dev)


@pytest.mark.parametrize("ratio", [0, 8, 11, 13, 16])
@pytest.mark.parametrize("D,Hq", [(64, 16), (128, 6)])
def test_a_large_query_channel_leaves_the_others_their_precision(D, Hq, ratio, dev):
    """Queries with one channel 2^ratio above the others where K is zero, and the others
    scaled so that the scores are as spread as ever."""
    rng = np.random.default_rng(330 + ratio)
    a = Setup(rng, dev, [600, 90], None, 2, 2, D, 32)
    a.cache["k"][:, :, :, 5] = 0
    a.upload(dev)
    q = rng.standard_normal((2, 2, Hq, D)) * 2.0 ** -ratio
    q[..., 5] = 3.7
    q = bf16_bits(q.astype(np.float32))
    scale = 2.0 ** (ratio - 3)
    out = run_attention(a, None, q, dev, scale)
    assert_device_ok()
    got, ref = bf16_to_f64(bf16_host(out)), osp.tree_attention(a.cache, a.table, a.pos, None, None,
                                                               q, scale)
    assert np.linalg.norm(got - ref) <= (2.0 ** -8 + 2.0 ** -9) * np.linalg.norm(ref)
    check_bars(a, None, q, out, dev, scale)


@pytest.mark.parametrize("ratio", [0, 4, 8, 12, 15])
@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 24)])
def test_scores_that_differ_little_from_a_large_common_part(D, Hq, ratio, dev):
    """A channel with the same large K at every position: the sums of products keep what
    the other channels add to it."""
    rng = np.random.default_rng(340 + ratio)
    a = Setup(rng, dev, [520, 33], None, 3, 2, D, 64)
    a.cache["k"][:, :, :, 9] = 0x7E                      # 448, the others below 256
    a.cache["k_exp"][:] = 127 - 8
    a.upload(dev)
    q = rng.standard_normal((2, 3, Hq, D))
    q[..., 9] = 0.83 * 2.0 ** ratio
    q = bf16_bits(q.astype(np.float32))
    out = run_attention(a, None, q, dev)
    assert_device_ok()
    check_bars(a, None, q, out, dev)
