"""Verification of drafted tokens on the GPU against the fp64 oracle: whole
numbers with one right answer, compared exactly, and a whole speculative step
with all five entry points."""

import threading

import numpy as np
import pytest
import torch

import local_moe_route_b200 as sm
from gpu_helpers import assert_device_ok, bf16_host, bf16_to_f64
from moe_inputs import bf16_bits
from oracle import speculative as osp
from test_gpu_kv import Setup, check_attention, run_attention, same_cache, tree, up, up_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_dev):
    from local_moe_route_b200 import build
    build.build()
    return cuda_dev


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def make(rng, B, N, V, kind, sharp=1.5):
    """Target and draft rows, drafts drawn from their parents' draft rows."""
    z = rng.standard_normal((B, N, V)) * sharp
    p, q = softmax(z), softmax(z + 0.7 * rng.standard_normal((B, N, V)))
    parent = tree(rng, B, N, kind)
    tokens = np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(1, N):
            up_ = i - 1 if parent is None else max(0, parent[b, i])
            r = q[b, up_].astype(np.float64)
            tokens[b, i] = rng.choice(V, p=r / r.sum())
    return dict(tokens=tokens, parent=parent, p=p, q=q,
                u_accept=rng.random((B, N)).astype(np.float32),
                u_sample=rng.random(B).astype(np.float32), count=None)


def run(a, dev, out=None, stream=None):
    B, N = a["tokens"].shape
    V = a["p"].shape[2]
    t = {k: None if x is None else up(x, dev) for k, x in a.items()}
    out = out or [torch.full(s, -9, dtype=torch.int32, device=dev) for s in ((B, N), (B,), (B, N))]
    sm.check(sm.strata_verify_drafts(t["tokens"], t["parent"], t["count"], t["p"], t["q"],
                                     t["u_accept"], t["u_sample"], dict(B=B, N=N, V=V), *out,
                                     stream=stream))
    return out


def check(a, out):
    want = osp.verify(a["tokens"], a["parent"], a["count"], a["p"], a["q"], a["u_accept"],
                      a["u_sample"])
    for name, x, y in zip(("path", "path_len", "out_tokens"), out, want):
        assert np.array_equal(x.cpu().numpy(), y), name
    return want


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 127, 128, 1000, 4097, 32000, 100003])
@pytest.mark.parametrize("kind,draft", [("chain", True), ("tree", True), ("star", True),
                                        ("chain", False), ("star", False)])
def test_verify(V, kind, draft, dev):
    rng = np.random.default_rng(V)
    B, N = (6, 9) if V < 5000 else (2, 5)
    a = make(rng, B, N, V, kind)
    if not draft:
        a["q"] = None
    out = run(a, dev)
    assert_device_ok()
    check(a, out)


@pytest.mark.parametrize("V", [180000, 181300, 190001, 196600, 230000, 800000])
def test_verify_vocabularies_whose_sums_need_large_shared_memory(V, dev):
    """Around the size from which a kernel's shared memory (the sums of four
    probabilities and what is there for every V) has to be asked for."""
    rng = np.random.default_rng(V)
    a = make(rng, 1, 3, V, "star")
    out = run(a, dev)
    assert_device_ok()
    check(a, out)


def test_verify_from_two_threads_with_different_vocabularies(dev):
    """Calls of two host threads, one with a far larger vocabulary: neither takes
    away the shared memory the other's launch needs."""
    jobs = []
    for V in (210000, 790000):
        a = make(np.random.default_rng(V), 1, 2, V, "chain")
        jobs.append((a, [up(a[n], dev) for n in ("tokens", "p", "q", "u_accept", "u_sample")],
                     [torch.zeros(s, dtype=torch.int32, device=dev) for s in ((1, 2), (1,), (1, 2))],
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    status = []

    def work(job):
        a, (tok, p, q, ua, us), out, stream = job
        dims = sm.VerifyDims.of((1, 2, p.shape[2]))
        for _ in range(1500):
            status.append(sm.strata_verify_drafts(tok, None, None, p, q, ua, us, dims, *out,
                                                  stream=stream))

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(status) == 3000 and set(status) == {sm.STRATA_OK}
    assert_device_ok()
    for a, _, out, _ in jobs:
        check(a, out)


def test_verify_sizes_counts_and_many_rejections(dev):
    rng = np.random.default_rng(5)
    a = make(rng, 9, 64, 700, "star")
    a["count"] = np.array([64, 0, 1, 2, 33, 64, 5, 0, 64], np.int32)
    a["u_accept"][:] = 0.999            # most of a star's children are rejected
    out = run(a, dev)
    assert_device_ok()
    _, n, _ = check(a, out)
    assert n[1] == 0 and n[7] == 0 and n[2] == 1
    a["q"] = None
    check(a, run(a, dev))
    b = make(rng, 1, 1, 333, "chain")   # no drafts: plain sampling
    check(b, run(b, dev))
    c = make(rng, 300, 3, 64, "chain")
    check(c, run(c, dev))
    d = make(rng, 1, 3, sm.STRATA_VERIFY_MAX_VOCAB, "star")
    check(d, run(d, dev))
    d["q"] = None
    check(d, run(d, dev))


def test_verify_past_two_to_the_31_values(dev):
    """Rows whose offsets pass 32 bits."""
    B, N, V = 65, 64, 600001
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of free device memory")
    rng = np.random.default_rng(12)
    a = make(rng, 1, 5, V, "star")
    p = torch.zeros((B, N, V), device=dev)
    p[-1, :5] = up(a["p"][0], dev)
    t = {k: np.zeros((B, N), x.dtype) for k, x in a.items() if k in ("tokens", "u_accept")}
    for k in t:
        t[k][-1, :5] = a[k][0]
    parent = np.full((B, N), -1, np.int32)
    parent[-1, :5] = a["parent"][0]
    count = np.zeros(B, np.int32)
    count[-1] = 5
    us = np.zeros(B, np.float32)
    us[-1] = a["u_sample"][0]
    out = [torch.full(s, -9, dtype=torch.int32, device=dev) for s in ((B, N), (B,), (B, N))]
    sm.check(sm.strata_verify_drafts(up(t["tokens"], dev), up(parent, dev), up(count, dev), p, None,
                                     up(t["u_accept"], dev), up(us, dev), (B, N, V), *out))
    assert_device_ok()
    want = osp.verify(a["tokens"], a["parent"], None, a["p"], None, a["u_accept"], a["u_sample"])
    assert np.array_equal(out[0][-1, :5].cpu().numpy(), want[0][0])
    assert out[1].cpu().tolist() == [0] * (B - 1) + [int(want[1][0])]
    assert np.array_equal(out[2][-1, :5].cpu().numpy(), want[2][0])


def test_verify_equal_rows_and_extreme_random_numbers(dev):
    """p = q accepts everything; u_sample 0 takes the lowest token with any
    probability, u_sample next to 1 the highest; sums on exact borders go to the next
    token; one-hot targets."""
    rng = np.random.default_rng(6)
    a = make(rng, 4, 7, 515, "chain")
    a["q"] = a["p"].copy()
    a["u_sample"][:] = [0.0, np.nextafter(np.float32(1), np.float32(0)), 0.5, 0.25]
    _, n, _ = check(a, run(a, dev))
    assert np.all(n == 7)
    b = make(rng, 4, 2, 1024, "chain")
    b["p"][:] = 1.0 / 1024              # running sums are exact: u * sum lies on a border
    b["q"][:] = 1.0 / 1024
    b["u_sample"][:] = [0.0, 0.25, 0.5, 1023.0 / 1024]
    _, _, t = check(b, run(b, dev))
    assert t[:, 1].tolist() == [0, 256, 512, 1023]
    c = make(rng, 2, 3, 97, "chain")
    c["p"][:] = 0.0
    c["p"][:, :, 41] = 1.0
    c["tokens"][:] = [[0, 41, 3], [0, 3, 41]]
    _, n, t = check(c, run(c, dev))
    assert n.tolist() == [2, 1] and t[0, :2].tolist() == [41, 41] and t[1, 0] == 41


def test_verify_reports_bad_tokens_counts_and_rows_without_weight(dev):
    rng = np.random.default_rng(7)
    a = make(rng, 3, 4, 50, "star")
    a["tokens"][0, 1] = 50
    a["tokens"][1, 2] = -1
    a["count"] = np.array([4, 4, 5], np.int32)
    out = run(a, dev)
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    want = dict(a, count=np.array([4, 4, 0], np.int32))
    check(want, out)
    b = make(rng, 2, 2, 50, "chain")
    b["p"][1] = 0.0
    out = run(b, dev)
    assert sm.strata_moe_device_status() == sm.STRATA_ERR_DEVICE_CHECK
    _, _, t = check(b, out)
    assert t[1, 0] == 0
    assert sm.strata_moe_device_status() == sm.STRATA_OK


def test_verify_keeps_the_targets_distribution(dev):
    """First new tokens of 40,000 sequences with the same rows: each token's
    frequency within 5 standard deviations of the target's (fixed seed)."""
    rng = np.random.default_rng(8)
    B, V = 40000, 7
    one = make(rng, 1, 4, V, "star", sharp=1.0)
    a = {k: None if x is None else np.ascontiguousarray(np.broadcast_to(x, (B,) + x.shape[1:]))
         for k, x in one.items()}
    r = one["q"][0, 0].astype(np.float64)
    a["tokens"] = rng.choice(V, p=r / r.sum(), size=(B, 4)).astype(np.int32)
    a["u_accept"] = rng.random((B, 4)).astype(np.float32)
    a["u_sample"] = rng.random(B).astype(np.float32)
    out = run(a, dev)
    assert_device_ok()
    got = np.bincount(out[2][:, 0].cpu().numpy(), minlength=V) / B
    p = one["p"][0, 0].astype(np.float64)
    assert np.all(np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / B))


def test_verify_repeats_streams_and_graphs(dev):
    rng = np.random.default_rng(9)
    a, b = make(rng, 5, 8, 3001, "tree"), make(rng, 5, 8, 3001, "tree")
    wa, wb = run(a, dev), run(b, dev)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = []
    for _ in range(4):
        for x, w, st in zip((a, b), (wa, wb), streams):
            with torch.cuda.stream(st):
                got.append((w, run(x, dev)))
    torch.cuda.synchronize()
    for w, o in got:
        assert all(torch.equal(i, j) for i, j in zip(w, o))
    t = {k: None if x is None else up(x, dev) for k, x in a.items()}
    out = [torch.zeros_like(x) for x in wa]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sm.check(sm.strata_verify_drafts(t["tokens"], t["parent"], None, t["p"], t["q"],
                                         t["u_accept"], t["u_sample"], (5, 8, 3001), *out))
    for x, w in ((a, wa), (b, wb)):
        for k in ("tokens", "parent", "p", "q", "u_accept", "u_sample"):
            t[k].copy_(up(x[k], dev))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(w, out))


def test_binding_refusals(dev):
    rng = np.random.default_rng(10)
    a = make(rng, 2, 3, 40, "chain")
    for k, f in (("p", lambda x: x.astype(np.float64)), ("q", lambda x: x[:, :2]),
                 ("tokens", lambda x: x.astype(np.int64)), ("u_sample", lambda x: x[:1])):
        with pytest.raises(sm.StrataError):
            run(dict(a, **{k: f(a[k])}), dev)
    assert_device_ok()


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_a_decoding_loop(D, page, dev):
    """Six speculative steps as a program runs them: the tree's K and V appended,
    attention from every node, verification, the accepted path committed, the
    lengths fed to the next step; all of it captured once and replayed. The
    cache, the outputs and the tokens against the oracle at every step."""
    rng = np.random.default_rng(11)
    B, N, Hq, Hkv, V = 3, 7, 8, 2, 211
    a = Setup(rng, dev, [page - 3, 0, 2 * page + 5], None, N, Hkv, D, page,
              slack=-(-8 * N // page))
    i32 = dict(dtype=torch.int32, device=dev)
    d = dict(k=torch.empty((B, N, Hkv, D), dtype=torch.bfloat16, device=dev),
             v=torch.empty((B, N, Hkv, D), dtype=torch.bfloat16, device=dev),
             q=torch.empty((B, N, Hq, D), dtype=torch.bfloat16, device=dev),
             p=torch.empty((B, N, V), device=dev), dq=torch.empty((B, N, V), device=dev),
             parent=torch.empty((B, N), **i32), tokens=torch.empty((B, N), **i32),
             ua=torch.empty((B, N), device=dev), us=torch.empty(B, device=dev))
    out = torch.zeros((B, N, Hq, D), dtype=torch.bfloat16, device=dev)
    path, n, toks = torch.zeros((B, N), **i32), torch.zeros(B, **i32), torch.zeros((B, N), **i32)
    ws = sm.tree_attention_workspace(a.c, a.s, Hq, dev)
    pos = a.s.tensors[1]

    def step():
        sm.check(sm.strata_kv_append(a.c, a.s, d["k"], d["v"]))
        sm.check(sm.strata_tree_attention(a.c, a.s, d["parent"], d["q"], 0.0, out, ws))
        sm.check(sm.strata_verify_drafts(d["tokens"], d["parent"], None, d["p"], d["dq"], d["ua"],
                                         d["us"], (B, N, V), path, n, toks))
        sm.check(sm.strata_kv_commit(a.c, a.s, path, n, pos))

    graph = None
    for it in range(6):
        m = make(rng, B, N, V, "tree")
        m["u_accept"] *= 0.3
        k, v = (bf16_bits(rng.standard_normal((B, N, Hkv, D)).astype(np.float32)) for _ in "kv")
        q = bf16_bits(rng.standard_normal((B, N, Hq, D)).astype(np.float32))
        for name, x in (("p", m["p"]), ("dq", m["q"]), ("parent", m["parent"]),
                        ("tokens", m["tokens"]), ("ua", m["u_accept"]), ("us", m["u_sample"])):
            d[name].copy_(up(x, dev))
        for name, x in (("k", k), ("v", v), ("q", q)):
            d[name].copy_(up_bf16(x, dev))
        if it < 2:
            step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        assert_device_ok()
        osp.append(a.cache, a.table, a.pos, None, k, v)
        check_attention(a, m["parent"], q, out)
        wpath, wn, wt = osp.verify(m["tokens"], m["parent"], None, m["p"], m["q"], m["u_accept"],
                                   m["u_sample"])
        assert np.array_equal(path.cpu().numpy(), wpath)
        assert np.array_equal(toks.cpu().numpy(), wt) and np.array_equal(n.cpu().numpy(), wn)
        a.pos = osp.commit(a.cache, a.table, a.pos, wpath, wn)
        same_cache(a.held(), a.cache)
        assert np.array_equal(pos.cpu().numpy(), a.pos)
