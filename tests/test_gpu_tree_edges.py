"""Tree attention at the edges of what its inputs may hold, against the fp64 oracle
(the bars are those of test_gpu_kv.py unless a test says otherwise)."""

import numpy as np
import pytest

import local_moe_route_b200 as sm
from moe_inputs import bf16_bits
from test_gpu_kv import Setup, check_attention, run_attention

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
