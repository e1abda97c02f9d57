"""The speculative-decoding calls in the order of their stream: what runs before a
call (a long kernel, a copy, a memset, another stream's work that an event joins,
the call before) is complete when the call reads, and a call's results are complete
when the next work reads them. The same steps with a synchronisation after
everything are the reference; every result is the same bit for bit."""

import subprocess
import sys

import numpy as np
import pytest
import torch

import local_moe_route_b200 as sm
from gpu_helpers import assert_device_ok

pytestmark = pytest.mark.gpu
STEPS = 5


@pytest.fixture(scope="module")
def dev(cuda_dev):
    from local_moe_route_b200 import build
    build.build()
    return cuda_dev


class Steps:
    """Speculative steps whose inputs are written just before they are read."""

    def __init__(self, dev, B, N, Hkv, D, page, V, start):
        g = torch.Generator(device=dev).manual_seed(23)
        bf = dict(dtype=torch.bfloat16, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        Hq, self.dev, self.dims = 4 * Hkv, dev, (B, N, V)
        cols = -(-(start + STEPS * N + N) // page)

        def draw(*shape):
            return torch.randn(STEPS, *shape, generator=g, device=dev)

        def rows():
            return torch.softmax(2 * draw(B, N, V), -1)

        par = [-1] + [(i - 1) // 2 for i in range(1, N)]
        self.src = dict(k=draw(B, N, Hkv, D).bfloat16(), v=draw(B, N, Hkv, D).bfloat16(),
                        q=draw(B, N, Hq, D).bfloat16(), p=rows(), dq=rows(),
                        tokens=torch.randint(0, V, (STEPS, B, N), generator=g, **i32),
                        ua=0.3 * torch.rand(STEPS, B, N, generator=g, device=dev),
                        us=torch.rand(STEPS, B, generator=g, device=dev),
                        parent=torch.tensor(par, **i32).expand(STEPS, B, N).contiguous())
        self.x = {name: torch.zeros_like(t[0]) for name, t in self.src.items()}
        self.cache = sm.KvCache.empty(B * cols, page, Hkv, D, dev)
        table = torch.randperm(B * cols, generator=g, device=dev).to(torch.int32).view(B, cols)
        self.start = start
        self.pos = torch.full((B,), start, **i32)
        self.seqs = sm.KvSeqs.of(table, self.pos, N=N)
        self.back = sm.KvSeqs.of(table, torch.zeros(B, **i32), N=start + N)
        self.prefix = [draw(B, start + N, Hkv, D)[0].bfloat16() for _ in "kv"]
        self.ws = sm.tree_attention_workspace(self.cache, self.seqs, Hq, dev)
        self.big = torch.zeros(1 << 26, device=dev)      # 256 MB: a pass over it is ~100 us
        self.out = torch.zeros((B, N, Hq, D), **bf)
        self.path, self.toks = torch.zeros((B, N), **i32), torch.zeros((B, N), **i32)
        self.n = torch.zeros(B, **i32)
        self.kv = [torch.zeros((B, start + N, Hkv, D), **bf) for _ in "kv"]
        self.log = {name: torch.zeros((STEPS,) + t.shape, dtype=t.dtype, device=dev)
                    for name, t in self.results().items()}
        self.side = torch.cuda.Stream()

    def results(self):
        return dict(out=self.out, path=self.path, n=self.n, toks=self.toks, pos=self.pos,
                    k=self.kv[0], v=self.kv[1])

    def reset(self):
        for t in (self.cache_tensors() + list(self.x.values()) + list(self.log.values())
                  + list(self.results().values())):
            t.zero_()
        self.pos.fill_(self.start)
        sm.check(sm.strata_kv_append(self.cache, self.back, *self.prefix))
        torch.cuda.synchronize()

    def cache_tensors(self):
        return list(self.cache.tensors)

    def step(self, i, side, sync):
        def then():
            if sync:
                torch.cuda.synchronize()

        def write(*names):
            # after a long kernel, so that a call that did not wait would see
            # the values of the step before
            cur = torch.cuda.current_stream()
            if side:
                self.side.wait_stream(cur)
            with torch.cuda.stream(self.side if side else cur):
                self.big.add_(1)
                for name in names:
                    self.x[name].copy_(self.src[name][i])
            if side:
                cur.wait_stream(self.side)
            then()

        x = self.x
        write("k", "v")
        sm.check(sm.strata_kv_append(self.cache, self.seqs, x["k"], x["v"]))
        then()
        write("q", "parent")
        self.out.zero_()
        sm.check(sm.strata_tree_attention(self.cache, self.seqs, x["parent"], x["q"], 0.0,
                                          self.out, self.ws))
        then()
        write("p", "dq", "tokens", "ua", "us")
        sm.check(sm.strata_verify_drafts(x["tokens"], x["parent"], None, x["p"], x["dq"], x["ua"],
                                         x["us"], self.dims, self.path, self.n, self.toks))
        then()
        sm.check(sm.strata_kv_commit(self.cache, self.seqs, self.path, self.n, self.pos))
        then()
        sm.check(sm.strata_kv_read(self.cache, self.back, *self.kv))
        then()
        # attention of the same tree again, straight behind the read
        sm.check(sm.strata_kv_append(self.cache, self.seqs, x["k"], x["v"]))
        then()
        sm.check(sm.strata_tree_attention(self.cache, self.seqs, x["parent"], x["q"], 0.0,
                                          self.out, self.ws))
        then()
        for name, t in self.results().items():
            self.log[name][i].copy_(t)
        then()


@pytest.mark.parametrize("way", ["stream", "graph"])
@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("B,N,Hkv,D,page,start", [(2, 5, 2, 128, 16, 37), (1, 9, 4, 64, 64, 3000),
                                                  (40, 4, 1, 128, 32, 300)])
def test_calls_wait_for_what_runs_before_them(B, N, Hkv, D, page, start, side, way, dev):
    s = Steps(dev, B, N, Hkv, D, page, 1021, start)
    s.reset()
    for i in range(STEPS):
        s.step(i, False, True)
    want = {name: t.clone() for name, t in s.log.items()}
    assert bool((want["pos"][-1] > start).any()) and bool((want["out"] != 0).any())
    s.reset()
    if way == "graph":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(STEPS):
                s.step(i, side, False)
    for _ in range(3):
        s.reset()
        if way == "graph":
            graph.replay()
        else:
            for i in range(STEPS):
                s.step(i, side, False)
        torch.cuda.synchronize()
        for name, t in s.log.items():
            assert torch.equal(t.view(torch.uint8), want[name].view(torch.uint8)), name
    assert_device_ok()


@pytest.mark.parametrize("D", [64, 128])
def test_calls_of_two_streams_and_one_cache_at_once(D, dev):
    """Two streams attend to the same cache at the same time, each with a workspace
    of its own, again and again: neither changes the other's output."""
    rng = np.random.default_rng(4)
    B, N, Hkv, page, L = 3, 4, 2, 32, 700
    cols = -(-(L + N) // page)
    c = sm.KvCache.empty(B * cols, page, Hkv, D, dev)
    table = torch.from_numpy(rng.permutation(B * cols).reshape(B, cols).astype(np.int32)).to(dev)
    i32 = dict(dtype=torch.int32, device=dev)
    fill = sm.KvSeqs.of(table, torch.zeros(B, **i32), N=L + N)
    kv = [torch.randn(B, L + N, Hkv, D, device=dev).bfloat16() for _ in "kv"]
    sm.check(sm.strata_kv_append(c, fill, *kv))
    parent = torch.tensor([-1, 0, 1, 2], **i32).expand(B, N).contiguous()
    jobs = []
    for _ in range(2):
        s = sm.KvSeqs.of(table, torch.full((B,), L, **i32), N=N)
        q = torch.randn(B, N, 4 * Hkv, D, device=dev).bfloat16()
        jobs.append((s, q, torch.zeros_like(q), sm.tree_attention_workspace(c, s, 4 * Hkv, dev),
                     torch.cuda.Stream()))

    def call(job, stream=None):
        s, q, out, ws, _ = job
        sm.check(sm.strata_tree_attention(c, s, parent, q, 0.0, out, ws, stream=stream))

    want = []
    for job in jobs:
        call(job)
        torch.cuda.synchronize()
        want.append(job[2].clone())
        job[2].zero_()
    torch.cuda.synchronize()
    for _ in range(50):
        for job in jobs:
            call(job, job[4])
    torch.cuda.synchronize()
    for job, w in zip(jobs, want):
        assert torch.equal(job[2], w)
    assert_device_ok()


FIRST = """
import torch
import local_moe_route_b200 as sm
dev = torch.device("cuda", 0)
torch.manual_seed(1)
i32 = dict(dtype=torch.int32, device=dev)
B, N, Hkv, Hq, D, page, V = 2, 3, 2, 8, 128, 16, 200001
c = sm.KvCache.empty(8, page, Hkv, D, dev)
pos = torch.tensor([20, 9], **i32)
s = sm.KvSeqs.of(torch.arange(8, **i32).view(2, 4), pos, N=N)
back = sm.KvSeqs.of(torch.arange(8, **i32).view(2, 4), torch.zeros(2, **i32), N=24)
k, v = (torch.randn(B, N, Hkv, D, device=dev).bfloat16() for _ in "kv")
q = torch.randn(B, N, Hq, D, device=dev).bfloat16()
p = torch.softmax(torch.randn(B, N, V, device=dev), -1)
tok = p.argmax(-1).to(torch.int32).roll(1, 1).contiguous()
ua, us = torch.full((B, N), 1e-9, device=dev), torch.full((B,), 0.5, device=dev)
path, n, toks = torch.zeros(B, N, **i32), torch.zeros(B, **i32), torch.zeros(B, N, **i32)
out, pos_out = torch.zeros_like(q), torch.zeros(B, **i32)
kv = [torch.zeros(B, 24, Hkv, D, dtype=torch.bfloat16, device=dev) for _ in "kv"]
ws = sm.tree_attention_workspace(c, s, Hq, dev)

def step():
    sm.check(sm.strata_kv_append(c, s, k, v))
    sm.check(sm.strata_tree_attention(c, s, None, q, 0.0, out, ws))
    sm.check(sm.strata_verify_drafts(tok, None, None, p, None, ua, us, (B, N, V), path, n, toks))
    sm.check(sm.strata_kv_commit(c, s, path, n, pos_out))
    sm.check(sm.strata_kv_read(c, back, *kv))

def results():
    torch.cuda.synchronize()
    return [t.clone() for t in (out, path, n, toks, pos_out, *kv)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
got = results()
for t in (out, path, n, toks, pos_out, *kv, *c.tensors):
    t.zero_()
step()
want = results()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert bool((want[0] != 0).any()) and bool((want[2] > 0).all())
sm.check(sm.strata_moe_device_status())
print("same")
"""


def test_a_processs_first_calls_may_be_captured(dev):
    """Nothing has to be called before a capture: a process whose first calls of
    the library are captured gets what the same calls give outside a graph."""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr
