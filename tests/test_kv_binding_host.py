"""What the binding of the speculative-decoding calls lets through to the library,
looked at with a recorder in the library's place (nothing is launched, so it runs
with and without a GPU)."""

import pytest
import torch

import local_moe_route_b200 as sm
from local_moe_route_b200 import KvCache, KvSeqs, kv

FAKE = 1 << 40
OK, INVALID = sm.STRATA_OK, sm.STRATA_ERR_INVALID_ARG
B, N, HKV, HQ, D = 2, 3, 2, 6, 64


class Rows:
    """A dense or strided tensor of the current device, by its shape alone."""

    def __init__(self, shape, dtype, strides=None):
        self.shape, self.dtype = torch.Size(shape), dtype
        dense = [1]
        for n in reversed(shape[1:]):
            dense.insert(0, dense[0] * n)
        self.strides = tuple(strides or dense)
        self.contiguous = self.strides == tuple(dense)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    def is_contiguous(self):
        return self.contiguous

    def stride(self):
        return self.strides

    def get_device(self):
        return kv._device()

    def data_ptr(self):
        return FAKE


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return OK
        return call


@pytest.fixture
def library(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(kv, "_bound", r)
    return r


def cache():
    return KvCache(8, 16, HKV, D, FAKE, FAKE, FAKE, FAKE)


def seqs():
    return KvSeqs(B, N, 3, FAKE, FAKE, None)


def bf16(heads, wide=0):
    token = (heads + wide) * D
    return Rows((B, N, heads, D), torch.bfloat16, (N * token, token, D, 1))


def append(k, v, **kw):
    return sm.strata_kv_append(cache(), seqs(), k, v, stream=0, **kw)


def attend(q, ws=None, **kw):
    ws = Rows((1 << 20,), torch.uint8) if ws is None else ws
    return sm.strata_tree_attention(cache(), seqs(), None, q, 0.0, Rows((B, N, HQ, D), torch.bfloat16),
                                    ws, stream=0, **kw)


def test_a_stride_beside_dense_tensors_is_refused_unless_it_is_theirs(library):
    dense, wide = HKV * D, (HKV + 4) * D
    for k, v in ((bf16(HKV), bf16(HKV)), (bf16(HKV), FAKE), (FAKE, bf16(HKV))):
        for stride in (8, wide, 2 * wide, 1 << 30, -dense):
            assert append(k, v, stride=stride) == INVALID and not library.calls, stride
        for stride in (0, dense):
            assert append(k, v, stride=stride) == OK and library.calls.pop()[1][4] == stride
    # parts of wider rows bring their own, raw pointers the caller's
    for stride in (0, wide, 2 * wide):
        assert append(bf16(HKV, 4), bf16(HKV, 4), stride=stride) == OK
        assert library.calls.pop()[1][4] == wide
        assert append(FAKE, FAKE, stride=stride) == OK and library.calls.pop()[1][4] == stride


def test_a_query_stride_beside_a_dense_tensor_is_refused_unless_it_is_its_own(library):
    dense, wide = HQ * D, (HQ + 2) * D
    for stride in (8, wide, 1 << 30, -dense):
        assert attend(bf16(HQ), q_stride=stride) == INVALID and not library.calls, stride
    for stride in (0, dense):
        assert attend(bf16(HQ), q_stride=stride) == OK
        assert library.calls.pop()[1][4:6] == (stride, HQ)
    for stride in (0, wide, 2 * wide):
        assert attend(bf16(HQ, 2), q_stride=stride) == OK
        assert library.calls.pop()[1][4:6] == (wide, HQ)
        assert attend(FAKE, Hq=HQ, q_stride=stride) == OK
        assert library.calls.pop()[1][4:6] == (stride, HQ)


def test_a_workspace_tensor_counts_as_what_it_has(library):
    ws = Rows((4096,), torch.uint8)
    for given, got in ((None, 4096), (4096, 4096), (100, 100), (4097, 4096), (1 << 40, 4096)):
        assert attend(bf16(HQ), ws=ws, ws_bytes=given) == OK
        assert library.calls.pop()[1][9] == got
    assert attend(bf16(HQ), ws=FAKE, ws_bytes=1 << 30) == OK
    assert library.calls.pop()[1][9] == 1 << 30


def test_a_negative_workspace_size_is_none_at_all(library):
    for ws in (Rows((4096,), torch.uint8), FAKE):
        for given in (-1, -4096, -(1 << 40)):
            assert attend(bf16(HQ), ws=ws, ws_bytes=given) == OK
            assert library.calls.pop()[1][9] == 0
