"""Host-side checks of the speculative-decoding entry points (no GPU needed):
the library exports what strata_kv.h declares, every refusal comes before a
launch, the binding refuses tensors the entry points would misread; and pins
of the fp64 oracle."""

import os
import re
import subprocess

import numpy as np
import pytest
import torch

import local_moe_route_b200 as sm
from local_moe_route_b200 import KvCache, KvSeqs, VerifyDims
from oracle import speculative as osp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "strata_kv.h")
FAKE = 1 << 40          # 16-byte aligned, never dereferenced (validation fails first)
OK, INVALID, UNSUPPORTED, WORKSPACE = (sm.STRATA_OK, sm.STRATA_ERR_INVALID_ARG,
                                       sm.STRATA_ERR_UNSUPPORTED, sm.STRATA_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from local_moe_route_b200 import build
    build.build()
    return sm.lib()


def test_header_exports_and_binding():
    names = re.findall(r"STRATA_API\s+[\w\s\*]+?\b(strata_\w+)\s*\(", open(HEADER).read())
    assert set(names) == {"strata_kv_append", "strata_kv_read", "strata_kv_commit",
                          "strata_tree_attention", "strata_tree_attention_workspace_bytes",
                          "strata_verify_drafts"}
    out = subprocess.run(["nm", "-D", "--defined-only", sm.lib_path()], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    for n in names:
        assert n in exported and hasattr(sm, n) and n in sm.__all__


def cache(**kw):
    d = dict(pages=8, page=16, Hkv=2, D=64, k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE)
    d.update(kw)
    return KvCache(*[d[n] for n, _ in KvCache._fields_])


def seqs(**kw):
    d = dict(B=2, N=4, max_pages=3, table=FAKE, pos=FAKE, count=None)
    d.update(kw)
    return KvSeqs(*[d[n] for n, _ in KvSeqs._fields_])


def append(c=None, s=None, k=FAKE, v=FAKE, stride=0):
    return sm.strata_kv_append(c or cache(), s or seqs(), k, v, stride, stream=0)


def attend(c=None, s=None, parent=None, q=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40, Hq=4,
           q_stride=0):
    return sm.strata_tree_attention(c or cache(), s or seqs(), parent, q, 0.0, out, ws, ws_bytes,
                                    Hq=Hq, q_stride=q_stride, stream=0)


BAD_CACHE = [(dict(pages=0), INVALID), (dict(Hkv=-1), INVALID), (dict(D=96), UNSUPPORTED),
             (dict(page=24), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
             (dict(pages=1 << 27), UNSUPPORTED), (dict(k=None), INVALID),
             (dict(v=FAKE + 8), INVALID), (dict(k_exp=None), INVALID), (dict(v_exp=FAKE + 1), INVALID)]
BAD_SEQS = [(dict(B=-1), INVALID), (dict(N=0), INVALID), (dict(max_pages=0), INVALID),
            (dict(B=1 << 22), UNSUPPORTED), (dict(max_pages=1 << 28), UNSUPPORTED),
            (dict(table=None), INVALID), (dict(pos=FAKE + 4), INVALID),
            (dict(count=FAKE + 4), INVALID)]


def calls(c, s):
    return {"append": lambda: append(c, s),
            "read": lambda: sm.strata_kv_read(c or cache(), s or seqs(), FAKE, FAKE, stream=0),
            "commit": lambda: sm.strata_kv_commit(c or cache(), s or seqs(), FAKE, FAKE, FAKE,
                                                  stream=0),
            "attend": lambda: attend(c, s)}


@pytest.mark.parametrize("op", ["append", "read", "commit", "attend"])
def test_bad_caches_and_sequences_are_refused(op):
    for kw, want in BAD_CACHE:
        assert calls(cache(**kw), None)[op]() == want, kw
    for kw, want in BAD_SEQS:
        assert calls(None, seqs(**kw))[op]() == want, kw


@pytest.mark.parametrize("op", ["append", "read", "commit", "attend"])
def test_no_sequences_is_a_no_op(op):
    assert calls(cache(k=None, v=None, k_exp=None, v_exp=None),
                 seqs(B=0, table=None, pos=None))[op]() == OK


def test_append_refusals():
    assert append(k=None) == INVALID
    assert append(v=FAKE + 2) == INVALID
    for stride in (127, 120, 132, -128, 1 << 40):
        assert append(stride=stride) == INVALID, stride
    assert append(cache(Hkv=64, pages=1), seqs(B=1 << 10, N=1 << 13)) == UNSUPPORTED


def test_read_refusals():
    assert sm.strata_kv_read(cache(), seqs(), FAKE + 2, FAKE, stream=0) == INVALID
    assert sm.strata_kv_read(cache(), seqs(), None, None, stream=0) == OK


def test_commit_refusals():
    c, s = cache(), seqs()
    assert sm.strata_kv_commit(c, s, None, FAKE, FAKE, stream=0) == INVALID
    assert sm.strata_kv_commit(c, s, FAKE, FAKE + 4, FAKE, stream=0) == INVALID
    assert sm.strata_kv_commit(c, s, FAKE, FAKE, None, stream=0) == INVALID
    assert sm.strata_kv_commit(c, seqs(N=65), FAKE, FAKE, FAKE, stream=0) == UNSUPPORTED


def test_attention_refusals():
    assert attend(Hq=3) == INVALID
    assert attend(Hq=0) == INVALID
    assert attend(Hq=2 * 65) == UNSUPPORTED
    assert attend(s=seqs(N=65)) == UNSUPPORTED
    assert attend(parent=FAKE + 4) == INVALID
    assert attend(q=None) == INVALID
    assert attend(out=FAKE + 8) == INVALID
    assert attend(ws=None) == WORKSPACE
    n = sm.strata_tree_attention_workspace_bytes(cache(), seqs(), 4)
    assert n > 0 and attend(ws_bytes=n - 1) == WORKSPACE
    assert attend(q_stride=4 * 64 - 8) == INVALID
    assert attend(q_stride=4 * 64 + 4) == INVALID
    for bad in (lambda: sm.strata_tree_attention_workspace_bytes(cache(D=32), seqs(), 4),
                lambda: sm.strata_tree_attention_workspace_bytes(cache(), seqs(N=65), 4),
                lambda: sm.strata_tree_attention_workspace_bytes(cache(), seqs(), 5)):
        assert bad() == 0


def verify(dims=(2, 4, 100), **kw):
    a = dict(tokens=FAKE, parent=None, count=None, p=FAKE, q=None, u_accept=FAKE, u_sample=FAKE,
             path=FAKE, path_len=FAKE, out_tokens=FAKE)
    a.update(kw)
    return sm.strata_verify_drafts(a["tokens"], a["parent"], a["count"], a["p"], a["q"],
                                   a["u_accept"], a["u_sample"], VerifyDims(*dims), a["path"],
                                   a["path_len"], a["out_tokens"], stream=0)


def test_verify_refusals():
    for dims, want in (((-1, 4, 9), INVALID), ((1, 0, 9), INVALID), ((1, 4, 0), INVALID),
                       ((1, 65, 9), UNSUPPORTED), ((1 << 20, 64, 9), UNSUPPORTED),
                       ((1, 4, 800001), UNSUPPORTED), ((0, 4, 9), OK)):
        assert verify(dims) == want, dims
    for name in ("tokens", "p", "u_accept", "u_sample", "path", "path_len", "out_tokens"):
        assert verify(**{name: None}) == INVALID, name
        assert verify(**{name: FAKE + 4}) == INVALID, name
    for name in ("parent", "count", "q"):
        assert verify(**{name: FAKE + 4}) == INVALID, name


def test_binding_refuses_host_tensors_and_other_layouts():
    z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t)  # noqa: E731
    with pytest.raises(sm.StrataError):
        KvCache.of(z(2, 2, 16, 64), z(2, 2, 16, 64), z(2, 2, 16), z(2, 2, 16))
    with pytest.raises(sm.StrataError):
        KvSeqs.of(z(2, 3, t=torch.int32), z(2, t=torch.int32))
    with pytest.raises(sm.StrataError):
        KvCache.of(z(2, 2, 64), z(2, 2, 64), z(2, 2, 16), z(2, 2, 16))
    with pytest.raises(sm.StrataError):
        KvSeqs.of(z(6, t=torch.int32), z(2, t=torch.int32))
    x = z(2, 4, 2, 64, t=torch.bfloat16)
    assert append(k=x, v=x) == INVALID
    assert sm.strata_kv_read(cache(), seqs(), x, x, stream=0) == INVALID
    assert attend(q=z(2, 4, 4, 64, t=torch.bfloat16)) == INVALID
    assert verify(tokens=z(2, 4, t=torch.int32)) == INVALID


# ---------------------------------------------------------------------------
# Oracle pins
def test_oracle_e4m3_codes():
    # the values of the codes, against torch's type
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    assert np.array_equal(osp.E4M3, want.numpy(), equal_nan=True)
    # rounding to nearest even, against torch's cast (exact inputs)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(300) * 2.0 ** rng.integers(-12, 9, 300),
                        (osp.E4M3[:126] + osp.E4M3[1:127]) / 2, osp.E4M3[:127], [448.0, -448.0]])
    x = x.astype(np.float32).clip(-448, 448)
    got = np.array([osp.e4m3_code(float(v)) for v in x], np.uint8)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, ref)


def test_oracle_row_exponent():
    for top, e in ((448.0, 0), (448.0001, 1), (1.0, -8), (1.75, -8), (1.76, -7), (0.0, -126),
                   (2.0 ** -130, -126), (3.3e38, 119)):
        assert osp.row_exponent(np.array([top, -top / 2, np.inf, np.nan])) == e, top


def test_oracle_verify_preserves_the_target():
    """Over all random numbers the first new token is distributed as the target
    row: a grid over u_accept and u_sample, one draft of each token."""
    p0 = np.array([0.5, 0.3, 0.2], np.float32)
    q0 = np.array([0.2, 0.2, 0.6], np.float32)
    K = 60
    got = np.zeros(3)
    p = np.stack([p0, p0])[None]
    q = np.stack([q0, q0])[None]
    for x in range(3):
        for i in range(K):
            for j in range(K):
                _, _, t = osp.verify(np.array([[0, x]]), None, None, p, q,
                                     np.array([[0, (i + 0.5) / K]]), np.array([(j + 0.5) / K]))
                got[t[0, 0]] += q0[x] / K ** 2
    assert np.max(np.abs(got - p0)) < 2.0 / K


def test_oracle_ancestors():
    a = osp.ancestors(np.array([-1, 0, 0, 1, -1, 4]), 6)
    assert [list(np.nonzero(r)[0]) for r in a] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [4, 5]]
