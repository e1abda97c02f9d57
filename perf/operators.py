"""What is measured of the speculative-decoding operators: a step over an 8-bit
paged KV cache appends the drafted tokens' K and V (quantised as they are
written), attends from every node of the draft tree, verifies the drafted
tokens against the target's probabilities and keeps the accepted path's rows.

The five operators, by a case's "op":
  append  strata_kv_append       quantise new K and V rows into the cache's pages
  read    strata_kv_read         dequantise a range of positions back to bf16
  attend  strata_tree_attention  a tree (or chain, or single token) over the cache
  verify  strata_verify_drafts   accept drafted tokens, sample the next one
  commit  strata_kv_commit       move the accepted path's rows to their positions

The cache: pages of `page` positions, k and v [pages][Hkv][page][D] e4m3
codes, k_exp and v_exp [pages][Hkv][page] exponents plus 127; a row's value is
code * 2^(exponent), the exponent the smallest that keeps the row's largest
magnitude within 448.  Position t of sequence b lies in page table[b][t // page].
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
def listed():
    return [
        # a verify step of eight sequences (last token + 3 drafts) entering the cache
        dict(name="append_verify4_b8", op="append", B=8, N=4, Hkv=4, D=128, page=64, L=2000),
        # four 6144-token prompt chunks entering the cache
        dict(name="append_chunk6144", op="append", B=4, N=6144, Hkv=4, D=128, page=64, L=0),
        # a short prefix read back for three sequences, small heads and pages
        dict(name="read_prefix517", op="read", B=3, N=517, Hkv=2, D=64, page=16, L=83),
        # a whole 34,000-token prompt read back
        dict(name="read_34000", op="read", B=1, N=34000, Hkv=4, D=128, page=64, L=0),
        # one token of one short conversation: the smallest call
        dict(name="attend_decode1_L300", op="attend", B=1, N=1, Hq=32, Hkv=4, D=128, page=16,
             L=300, tree=False),
        # last token + 3 drafts behind the 34,000-token prompt
        dict(name="attend_verify4_L34000", op="attend", B=1, N=4, Hq=32, Hkv=4, D=128, page=64,
             L=34000, tree=False),
        # a served batch with 24-node trees, ragged contexts up to 8192
        dict(name="attend_tree24_b16", op="attend", B=16, N=24, Hq=16, Hkv=2, D=64, page=32,
             L=8192, tree=True),
        # a large served batch of verify steps, ragged contexts up to 34,000
        dict(name="attend_verify4_b32", op="attend", B=32, N=4, Hq=32, Hkv=4, D=128, page=64,
             L=34000, tree=False),
        # three drafts of one sequence against the target, greedy drafter (no draft rows)
        dict(name="verify_chain4_b1", op="verify", B=1, N=4, V=32000, tree=False, draft=False),
        # 16-node trees of 32 sequences, sampled drafts, an odd vocabulary
        dict(name="verify_tree16_b32", op="verify", B=32, N=16, V=100003, tree=True, draft=True),
        # the accepted path of two 8-node trees
        dict(name="commit_tree8_b2", op="commit", B=2, N=8, Hkv=4, D=128, page=16, L=1000),
        # the accepted paths of 256 trees of 64 nodes
        dict(name="commit_tree64_b256", op="commit", B=256, N=64, Hkv=8, D=128, page=64, L=900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "verify", "commit"])
    heads = dict(Hkv=rng.randint(1, 8), D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    if op in ("append", "read"):
        B = _log(rng, 1, 32)
        return dict(op=op, B=B, N=_log(rng, 1, 34000 // B), L=rng.randint(0, 3000), **heads)
    if op == "attend":
        B = _log(rng, 1, 32)
        return dict(op=op, B=B, N=_log(rng, 1, 64), Hq=heads["Hkv"] * rng.randint(1, 16),
                    L=_log(rng, 1, 60000 // B + 1), tree=rng.random() < 0.6, **heads)
    if op == "verify":
        B = _log(rng, 1, 24)
        return dict(op=op, B=B, N=rng.randint(1, 16), V=_log(rng, 500, 130000),
                    tree=rng.random() < 0.6, draft=rng.random() < 0.6)
    return dict(op=op, B=_log(rng, 1, 256), N=rng.randint(1, 64), L=rng.randint(0, 1500), **heads)


def _pos(case):
    """Positions before the call: the longest first, the others spread below it
    (fixed by the case, so that the work of a case does not change with the seed)."""
    return [int(case["L"] * (1.0 if b == 0 else (b * 0.6180339887) % 1.0)) for b in range(case["B"])]


def _count(case):
    """Tokens of every sequence in this call: ragged, the first one full."""
    return [case["N"] if b % 3 == 0 else 1 + (b * 7 + case["N"] // 2) % case["N"]
            for b in range(case["B"])]


# ---------------------------------------------------------------------------
# Inputs
def _bf16_bits_exp(amax):
    """Smallest e in [-126, 119] with amax <= 448 * 2^e (448 = 1.75 * 2^8)."""
    a = amax.float().view(torch.int32)
    e = (a >> 23) - 127 - 8 + ((a & 0x7FFFFF) > 0x600000).to(torch.int32)
    return e.clamp(-126, 119)


def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """bf16 rows [..., D] -> e4m3 codes as bytes, exponents plus 127 as bytes."""
    e = _bf16_bits_exp(x.abs().amax(-1))
    c = (x.float() * _pow2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return c.view(torch.uint8), (e + 127).to(torch.uint8)


def _rows(g, shape, hot):
    """K- or V-like rows: rows of different magnitude, a few hot channels."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))
    x *= 1 + hot * (torch.rand(shape[-2:], generator=g, device=DEV) < 0.04)
    return x.to(torch.bfloat16)


def _cache(case, g, ends):
    """A cache with room for positions 0..ends[b], pages in no order, filled with
    written rows; what lies behind a sequence's end is any bytes at all."""
    page, Hkv, D, B = case["page"], case["Hkv"], case["D"], case["B"]
    per = max(1, max(-(-e // page) for e in ends))
    used = B * per
    pages = used + 3
    table = torch.randperm(pages, generator=g, device=DEV)[:used].to(torch.int32).view(B, per)
    s = dict(table=table.contiguous(), pages=pages, max_pages=per)
    for n, hot in (("k", 3.0), ("v", 1.0)):
        c = torch.empty((pages, Hkv, page, D), dtype=torch.uint8, device=DEV)
        x = torch.empty((pages, Hkv, page), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 26) // (Hkv * page * D))
        for i in range(0, pages, step):
            n_ = min(step, pages - i)
            c[i:i + n_], x[i:i + n_] = _quantise(_rows(g, (n_, Hkv, page, D), hot))
        s[n], s[n + "_exp"] = c, x
    # behind the ends: bytes that mean nothing, not-a-numbers among them
    t = torch.arange(per * page, device=DEV)
    behind = t[None, :] >= torch.tensor(ends, device=DEV)[:, None]
    b, t = torch.nonzero(behind, as_tuple=True)
    pg, off = table[b, t // page].long(), t % page
    for n in ("k", "v"):
        s[n][pg, :, off] = torch.randint(0, 256, (len(b), Hkv, D), generator=g, device=DEV,
                                         dtype=torch.uint8)
    return s


def _parents(case, g):
    B, N = case["B"], case["N"]
    up = torch.arange(-1, N - 1, device=DEV, dtype=torch.int32).repeat(B, 1)
    if case.get("tree"):   # a node hangs from one of the nodes up to 6 before it
        back = torch.randint(1, 7, (B, N), generator=g, device=DEV, dtype=torch.int32)
        up = torch.maximum(torch.arange(N, device=DEV, dtype=torch.int32) - back,
                           torch.zeros_like(up))
        up[:, 0] = -1
    return up.contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, N = case["B"], case["N"]
    s = dict(case=dict(case))
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "verify":
        V = case["V"]
        s["parent"] = _parents(case, g)
        logits = 2.5 * torch.randn((B, N, V), generator=g, device=DEV)
        near = logits + 0.7 * torch.randn((B, N, V), generator=g, device=DEV)
        s["p"] = torch.softmax(logits, -1)
        q = torch.softmax(near, -1)
        del logits, near
        at = s["parent"].clamp(min=0).long()
        if case["draft"]:
            rows = torch.gather(q, 1, at[..., None].expand(B, N, V)).view(B * N, V)
            s["tokens"] = torch.multinomial(rows, 1, generator=g).view(B, N).to(torch.int32)
            s["q"] = q
        else:   # a greedy drafter: a node's children are its most likely tokens, in order
            rank = ((at[:, :, None] == at[:, None, :]).tril(-1)[..., 1:]).sum(-1).clamp(max=7)
            best = torch.topk(q, 8, -1).indices
            s["tokens"] = best[torch.arange(B, device=DEV)[:, None], at, rank].to(torch.int32)
            s["q"] = None
        s["u_accept"] = torch.rand((B, N), generator=g, device=DEV)
        if not case["draft"]:
            s["u_accept"] *= 0.05   # peaks of these rows are low: let some be accepted
        s["u_sample"] = torch.rand((B,), generator=g, device=DEV)
        s["count"] = torch.tensor(_count(case), **i32)
        s["path"] = torch.empty((B, N), **i32)
        s["path_len"] = torch.empty((B,), **i32)
        s["out_tokens"] = torch.empty((B, N), **i32)
        if own:
            import local_moe_route_b200 as sm
            s["dims"] = sm.VerifyDims.of(dict(B=B, N=N, V=V))
        return s
    pos, count = _pos(case), _count(case)
    Hkv, D = case["Hkv"], case["D"]
    s.update(_cache(case, g, [p + c for p, c in zip(pos, count)]))
    s["pos"], s["count"] = torch.tensor(pos, **i32), torch.tensor(count, **i32)
    if case["op"] == "append":
        # K and V as they leave a fused projection: parts of one row per token
        qkv = _rows(g, (B, N, 2 * Hkv, D), 2.0)
        s["k_new"], s["v_new"] = qkv[:, :, :Hkv], qkv[:, :, Hkv:]
    elif case["op"] == "read":
        for n in ("k_out", "v_out"):
            s[n] = torch.zeros((B, N, Hkv, D), dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "attend":
        Hq = case["Hq"]
        s["parent"] = _parents(case, g) if case["tree"] else None
        s["q"] = torch.randn((B, N, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.zeros((B, N, Hq, D), dtype=torch.bfloat16, device=DEV)
    else:
        # the accepted path: node 0 and some of the nodes after it, ascending
        keep = torch.rand((B, N), generator=g, device=DEV) < 0.4
        keep[:, 0] = True
        keep &= torch.arange(N, device=DEV) < s["count"][:, None]
        s["path_len"] = keep.sum(-1).to(torch.int32)
        first = torch.sort(~keep, dim=-1, stable=True).indices.to(torch.int32)
        s["path"] = torch.where(torch.arange(N, device=DEV) < s["path_len"][:, None], first,
                                torch.full_like(first, -1)).contiguous()
        s["pos_out"] = torch.empty((B,), **i32)
    if own:
        import local_moe_route_b200 as sm
        s["cache"] = sm.KvCache.of(s["k"], s["v"], s["k_exp"], s["v_exp"])
        s["seqs"] = sm.KvSeqs.of(s["table"], s["pos"], s["count"], N=N)
        if case["op"] == "attend":
            s["ws"] = sm.tree_attention_workspace(s["cache"], s["seqs"], case["Hq"], DEV)
    return s


# ---------------------------------------------------------------------------
# The plain forms
def _slots(s):
    """(b, i, page, offset) of every token of the call."""
    page, N = s["case"]["page"], s["case"]["N"]
    b, i = torch.nonzero(torch.arange(N, device=DEV) < s["count"][:, None], as_tuple=True)
    t = s["pos"][b].long() + i
    return b, i, s["table"][b, t // page].long(), t % page


def _held(s):
    """The cache as it is held: codes as the values they stand for, and exponents."""
    return {n: s[n].view(torch.float8_e4m3fn) if n in ("k", "v") else s[n]
            for n in ("k", "v", "k_exp", "v_exp")}


def _append(s):
    b, i, pg, off = _slots(s)
    for n in ("k", "v"):
        codes, exps = _quantise(s[n + "_new"][b, i])
        s[n][pg, :, off] = codes
        s[n + "_exp"][pg, :, off] = exps
    return _held(s)


def _value(codes, exps):
    return codes.view(torch.float8_e4m3fn).float() * _pow2(exps.to(torch.int32) - 127)[..., None]


def _read(s):
    b, i, pg, off = _slots(s)
    for n in ("k", "v"):
        s[n + "_out"][b, i] = _value(s[n][pg, :, off], s[n + "_exp"][pg, :, off]).to(torch.bfloat16)
    return {"k": s["k_out"], "v": s["v_out"]}


def _ancestors(parent, B, N):
    """[B][N][N] truth values: node i sees node j (itself and the nodes above it).
    With A[i][parent(i)] = 1, the sum of A's powers is the inverse of 1 - A."""
    if parent is None:
        return torch.ones((N, N), dtype=torch.bool, device=DEV).tril().expand(B, N, N)
    eye = torch.eye(N, device=DEV)
    a = (parent[..., None] == torch.arange(N, device=DEV)).float()
    return torch.linalg.solve_triangular(eye - a, eye.expand(B, N, N), upper=False) > 0.5


def _attend(s):
    c = s["case"]
    B, N, Hq, Hkv, D, page = (c[n] for n in ("B", "N", "Hq", "Hkv", "D", "page"))
    G, L = Hq // Hkv, s["max_pages"] * page
    t = torch.arange(L, device=DEV)
    there = t < (s["pos"] + s["count"])[:, None]                                # [B][L]

    def take(n):   # [B][Hkv][L][D], zeros behind the ends
        x = _value(s[n][s["table"].long()], s[n + "_exp"][s["table"].long()])
        x = x.transpose(1, 2).reshape(B, Hkv, L, D)
        return torch.where(there[:, None, :, None], x, 0.0)

    q = s["q"].float().view(B, N, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, N * G, D)
    score = (q @ take("k").transpose(-1, -2)) * (1.0 / math.sqrt(D))
    node = (t - s["pos"][:, None]).long()                                       # [B][L]
    among = torch.gather(_ancestors(s["parent"], B, N), 2,
                         node.clamp(0, N - 1)[:, None, :].expand(B, N, L))
    seen = torch.where(node[:, None, :] < 0, True, among & (node < N)[:, None, :])
    seen = seen & there[:, None, :]
    seen = seen[:, None, :, None, :].expand(B, Hkv, N, G, L).reshape(B, Hkv, N * G, L)
    score = torch.where(seen, score, -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    w = torch.where(seen, w, 0.0)
    o = (w @ take("v")) / w.sum(-1, keepdim=True)
    o = o.view(B, Hkv, N, G, D).transpose(1, 2).reshape(B, N, Hq, D).to(torch.bfloat16)
    mine = torch.arange(N, device=DEV) < s["count"][:, None]
    s["out"].copy_(torch.where(mine[..., None, None], o, s["out"]))
    return s["out"]


def _verify(s):
    """Children of a node are tried in ascending order; nodes are numbered after
    their parents, so one pass over the nodes follows the path.  After a rejected
    child the target's row p becomes r = max(p - c q, 0), c grown by the last r's sum;
    a drafter without rows puts all of q on its token.  All in 64 bits."""
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    at = torch.arange(B, device=DEV)
    p64, q64 = s["p"], s["q"]
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    grown = torch.zeros(B, dtype=torch.float64, device=DEV)
    total = torch.ones(B, dtype=torch.float64, device=DEV)
    gone = torch.zeros((B, V), dtype=torch.bool, device=DEV)
    on_path = torch.zeros((B, N), dtype=torch.bool, device=DEV)
    on_path[:, 0] = True

    def rest():
        p = p64[at, cur].double()
        if q64 is None:
            return torch.where(gone, 0.0, p)
        return (p - grown[:, None] * q64[at, cur].double()).clamp(min=0)

    for i in range(1, N):
        asked = (s["parent"][:, i] == cur) & (i < s["count"])
        x = s["tokens"][:, i].long()
        r = rest()
        qx = 1.0 if q64 is None else q64[at, cur, x].double()
        take = asked & (s["u_accept"][:, i].double() * qx * total < r[at, x])
        drop = asked & ~take
        gone[at, x] |= drop
        gone &= ~take[:, None]
        grown = torch.where(take, 0.0, torch.where(drop, grown + total, grown))
        cur = torch.where(take, i, cur)
        total = torch.where(take, 1.0, torch.where(drop, rest().sum(-1), total))
        on_path[:, i] |= take
    r = rest()
    below = torch.cumsum(r, -1)
    more = below > s["u_sample"].double()[:, None] * below[:, -1:]
    last = V - 1 - (r > 0).flip(-1).to(torch.uint8).argmax(-1)
    nxt = torch.where(more.any(-1), more.to(torch.uint8).argmax(-1), last)
    on_path &= (s["count"] > 0)[:, None]
    n = on_path.sum(-1)
    nodes = torch.sort(~on_path, dim=-1, stable=True).indices
    k = torch.arange(N, device=DEV)
    s["path"].copy_(torch.where(k < n[:, None], nodes, -1))
    s["path_len"].copy_(n)
    tok = torch.gather(s["tokens"].long(), 1, nodes.roll(-1, 1))
    tok = torch.where(k < n[:, None] - 1, tok, torch.where(k == n[:, None] - 1, nxt[:, None], -1))
    s["out_tokens"].copy_(tok)
    return {"path": s["path"], "path_len": s["path_len"], "out_tokens": s["out_tokens"]}


def _commit(s):
    page = s["case"]["page"]
    b, i = torch.nonzero(torch.arange(s["case"]["N"], device=DEV) < s["path_len"][:, None],
                         as_tuple=True)
    src, dst = s["pos"][b].long() + s["path"][b, i], s["pos"][b].long() + i
    from_, to = s["table"][b, src // page].long(), s["table"][b, dst // page].long()
    for n in ("k", "v", "k_exp", "v_exp"):
        s[n][to, :, dst % page] = s[n][from_, :, src % page]
    s["pos_out"].copy_(s["pos"] + s["path_len"])
    return _held(s) | {"pos": s["pos_out"]}


# ---------------------------------------------------------------------------
# The framework's calls
def _own(s):
    import local_moe_route_b200 as sm
    op = s["case"]["op"]
    if op == "append":
        sm.check(sm.strata_kv_append(s["cache"], s["seqs"], s["k_new"], s["v_new"]))
        return _held(s)
    if op == "read":
        sm.check(sm.strata_kv_read(s["cache"], s["seqs"], s["k_out"], s["v_out"]))
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attend":
        sm.check(sm.strata_tree_attention(s["cache"], s["seqs"], s["parent"], s["q"], 0.0, s["out"],
                                          s["ws"]))
        return s["out"]
    if op == "verify":
        sm.check(sm.strata_verify_drafts(s["tokens"], s["parent"], s["count"], s["p"], s["q"],
                                         s["u_accept"], s["u_sample"], s["dims"], s["path"],
                                         s["path_len"], s["out_tokens"]))
        return {"path": s["path"], "path_len": s["path_len"], "out_tokens": s["out_tokens"]}
    sm.check(sm.strata_kv_commit(s["cache"], s["seqs"], s["path"], s["path_len"], s["pos_out"]))
    return _held(s) | {"pos": s["pos_out"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "read": _read, "attend": _attend, "verify": _verify,
            "commit": _commit}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
def work(case):
    B, N, op = case["B"], case["N"], case["op"]
    count = _count(case)
    if op == "verify":
        # the row the next token comes from (p, and q where a draft was rejected), and
        # the drafted tokens' own probabilities; of a row's sums one operation a value
        rows = 2 if case["draft"] else 1
        return {"bytes": B * (4 * case["V"] * rows + N * 28 + 12), "flops": B * case["V"] * rows}
    Hkv, D, T = case["Hkv"], case["D"], sum(count)
    row = Hkv * (D + 1)                        # a position's codes and exponents, K or V
    index = B * (8 + 4 * -(-(case["L"] + N) // case["page"]))
    if op in ("append", "read"):
        return {"bytes": T * 2 * (row + Hkv * D * 2) + index, "flops": 2 * T * Hkv * D}
    if op == "commit":
        kept = sum(1 + 0.4 * (c - 1) for c in count)     # rows of the path, the first in place
        return {"bytes": 2 * 2 * row * kept + 4 * B * N + index, "flops": 0}
    ends = [p + c for p, c in zip(_pos(case), count)]
    pairs = sum(e * c for e, c in zip(ends, count))
    return {"bytes": sum(ends) * 2 * row + 2 * T * case["Hq"] * D * 2 + 4 * B * N + index,
            "flops": 4 * pairs * case["Hq"] * D}


# ---------------------------------------------------------------------------
# The same from the definitions in 64 bits, written apart from the plain forms
_E4M3 = [(-1.0) ** (c >> 7) * ((8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10) if (c >> 3) & 15
                               else (c & 7) * 2.0 ** -9) for c in range(256)]
_E4M3[0x7F] = _E4M3[0xFF] = math.nan


def _exact_codes(x):
    """Rows to the nearest e4m3 values (even on ties) of x / 2^e, and e + 127."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448.0) - 1e-12)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top > 0, e, -126.0).clamp(-126, 119)
    y = x / torch.exp2(e)[..., None]
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / unit) * unit).clamp(-448, 448), (e + 127).to(torch.uint8)


def exact(case, seed):
    op = case["op"]
    if op in ("verify", "commit"):
        return None            # whole numbers, and rows moved as they are
    s = prepare(case, seed)
    page, N, D = case["page"], case["N"], case["D"]
    pos, count = s["pos"].tolist(), s["count"].tolist()
    grid = torch.tensor(_E4M3, dtype=torch.float64, device=DEV)

    def rows(n, b, t0, t1):      # [t1 - t0][Hkv][D]
        t = torch.arange(t0, t1, device=DEV)
        pg = s["table"][b, t // page].long()
        return (grid[s[n][pg, :, t % page].long()]
                * torch.exp2(s[n + "_exp"][pg, :, t % page].double() - 127)[..., None])

    if op == "append":
        held = {}
        for n in ("k", "v"):
            code, exps = grid[s[n].long()], s[n + "_exp"].clone()
            for b in range(case["B"]):
                t = torch.arange(pos[b], pos[b] + count[b], device=DEV)
                pg = s["table"][b, t // page].long()
                code[pg, :, t % page], exps[pg, :, t % page] = _exact_codes(s[n + "_new"][b, :count[b]])
            held[n], held[n + "_exp"] = code, exps
        return held
    if op == "read":
        out = {}
        for n in ("k", "v"):
            out[n] = torch.zeros((case["B"], N, case["Hkv"], D), dtype=torch.float64, device=DEV)
            for b in range(case["B"]):
                out[n][b, :count[b]] = rows(n, b, pos[b], pos[b] + count[b])
        return out
    Hq, Hkv = case["Hq"], case["Hkv"]
    out = torch.zeros((case["B"], N, Hq, D), dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        n, end = count[b], pos[b] + count[b]
        up = list(range(-1, n - 1)) if s["parent"] is None else s["parent"][b].tolist()
        seen = np.zeros((n, n), bool)
        for i in range(n):
            if up[i] >= 0:
                seen[i] = seen[up[i]]
            seen[i, i] = True
        hidden = torch.zeros((n, end), dtype=torch.bool, device=DEV)
        hidden[:, pos[b]:] = ~torch.from_numpy(seen).to(DEV)
        k, v = rows("k", b, 0, end), rows("v", b, 0, end)
        for h in range(Hq):
            x = s["q"][b, :n, h].double() @ k[:, h // (Hq // Hkv)].T / math.sqrt(D)
            w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[b, :n, h] = w @ v[:, h // (Hq // Hkv)]
    return out
