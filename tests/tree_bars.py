"""What the tree attention may be off by, from its roundings, and the fp64 result
itself, computed with torch in 64 bits from the weights of every row (the oracle of
oracle/speculative.py is loops; this one serves long lines, on the host or the GPU).

Per (node, query head), with normalised weights p_t over what it sees, values
v_t = code_t * 2^(e_t), the output o = sum p_t v_t:
  * o's rounding to bf16: 2^-8 |o|;
  * a weight's rounding, first to fp16 (2^-11), then to two e4m3 codes (2^-9), of what
    it adds: (2^-9 + 2^-11) p_t |v_t|;
  * the floor of the codes: in a tile of 256 positions the row's largest p_t 2^(e_t)
    is scaled to 224 .. 448, and half of e4m3's smallest step is 2^-10, so a weight is
    off by up to 2^-10 / 224 (2^-17.8) of that, times |code_t|;
  * a score's error ds_t, fp32 sums of D products (D 2^-24 sum |q k|) and the values of
    q that are no multiple of 2^-13 of the row's scale, off by half of that: p_t ds_t
    |v_t| and, through the sum of the weights, max ds_t |o|;
  * fp32 sums over the tiles and the exponential (2^-22): 2^-19 of sum p_t |v_t|.
`bound` is the sum of these for every value: no result of the formula may exceed it.
`row` bounds the 2-norm of a row's error with the roundings of different positions
independent of each other, as they are for values that have nothing to do with one
another: the terms over t then add as squares.  It is what notices a few lost positions
among thousands, where the roundings of every value could, in the worst case, hide
them."""

import numpy as np
import torch

from oracle import speculative as osp

TILE = 256


def _codes(dev):
    return torch.from_numpy(osp.E4M3).to(dev)


def _seen(parent, n, dev):
    return torch.from_numpy(osp.ancestors(parent, n)).to(dev)


class Bars:
    """ref, bound [B][N][Hq][D] and row [B][N][Hq], NaN for slots behind the counts;
    the cache's rows that are seen must hold no NaN.  `only`: the sequences to look at,
    the others stay NaN.  `drop` {b: positions that are left out}, `twice` {b: positions
    that count twice}: wrong results, to see that the bars notice."""

    def __init__(self, cache, table, pos, count, parent, q, scale=None, dev="cpu", only=None,
                 drop=None, twice=None):
        t = {n: torch.as_tensor(x).to(dev) for n, x in cache.items()}
        pages, Hkv, page, D = t["k"].shape
        B, N, Hq, _ = q.shape
        G = Hq // Hkv
        sc = 1.0 / np.sqrt(D) if scale is None else float(scale)
        grid = _codes(dev)
        qd = torch.from_numpy(osp.bf16_values(q)).to(dev)
        tab = torch.as_tensor(np.asarray(table)).to(dev).long()
        f64 = dict(dtype=torch.float64, device=dev)
        self.ref = torch.full((B, N, Hq, D), float("nan"), **f64)
        self.bound, self.row = self.ref.clone(), torch.full((B, N, Hq), float("nan"), **f64)
        for b, p, n in osp._ranges(table, pos, count, N):
            if n == 0 or (only is not None and b not in only):
                continue
            at = torch.arange(min(p + n, tab.shape[1] * page), device=dev)
            pg = tab[b, at // page]
            good = (pg >= 0) & (pg < pages)
            at, pg = at[good], pg[good]
            if len(at) == 0:                 # a sequence without a valid page
                self.ref[b, :n] = self.bound[b, :n] = self.row[b, :n] = 0.0
                continue
            node = at - p
            sees = torch.ones((n, len(at)), dtype=torch.bool, device=dev)
            late = node >= 0
            sees[:, late] = _seen(None if parent is None else parent[b], n, dev)[:, node[late]]
            for hk in range(Hkv):
                ke, ve = (t[m + "_exp"][pg, hk, at % page].double() for m in "kv")
                kc, vc = (grid[t[m][pg, hk, at % page].long()] for m in "kv")
                here = ke > 0
                k = torch.where(here[:, None], kc * torch.exp2(ke - 127)[:, None], 0.0)
                vc = torch.where((here & (ve > 0))[:, None], vc, 0.0)
                v = vc * torch.exp2(ve - 127)[:, None]
                x = qd[b, :n, hk * G:(hk + 1) * G].reshape(n * G, D)
                vis = (sees & here).repeat_interleave(G, 0)
                if drop is not None and b in drop:
                    vis = vis & ~torch.isin(at, torch.as_tensor(drop[b], device=dev))
                s = (sc * (x @ k.T)).masked_fill(~vis, -float("inf"))
                top = s.amax(-1, keepdim=True)
                w = torch.exp(s - torch.where(top > -float("inf"), top, 0.0))
                if twice is not None and b in twice:
                    w = w * (1 + torch.isin(at, torch.as_tensor(twice[b], device=dev)))
                total = w.sum(-1, keepdim=True)
                w = torch.where(total > 0, w / total, 0.0)
                o = w @ v
                # q in units of its row's scale: the smallest 2^e with max|q| <= 448 2^e
                e = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True).clamp(min=1e-300) / 448))
                u = x / torch.exp2(e) * 2.0 ** 13
                dq = torch.where(u == torch.round(u), 0.0, torch.exp2(e - 14))
                ds = sc * (dq @ k.abs().T + D * 2.0 ** -24 * (x.abs() @ k.abs().T))
                ds_top = torch.where(vis, ds, 0.0).amax(-1, keepdim=True)
                a = 2.0 ** -9 + 2.0 ** -11
                # the largest contribution of the row in each tile, at its positions
                c = w * torch.exp2(ve - 127)
                tile = (at // TILE)[None].expand_as(c)
                most = torch.zeros((n * G, int(at[-1]) // TILE + 1 if len(at) else 1), **f64)
                most = most.scatter_reduce(1, tile, c, "amax")
                floor = torch.where(vis, 2.0 ** -10 / 224 * most.gather(1, tile), 0.0)
                bound = (2.0 ** -8 * o.abs() + (w * (a + ds + 2.0 ** -19)) @ v.abs()
                         + ds_top * o.abs() + floor @ vc.abs())
                part = ((w * (a + ds)) ** 2) @ (v ** 2) + (floor ** 2) @ (vc ** 2)
                row = ((2.0 ** -8 + 2.0 ** -19 + ds_top[:, 0]) * o.norm(dim=-1)
                       + part.sum(-1).sqrt())
                to = (b, slice(0, n), slice(hk * G, (hk + 1) * G))
                self.ref[to] = o.view(n, G, D)
                self.bound[to] = bound.view(n, G, D)
                self.row[to] = row.view(n, G)

    def faults(self, got):
        """What exceeds a bar: a text per kind and sequence, none if all is well.  `got`
        [B][N][Hq][D]; slots behind the counts are not looked at."""
        got = torch.as_tensor(got).to(self.ref)
        live = ~self.ref.isnan()
        off = torch.where(live, (got - self.ref).abs(), 0.0)
        out = []
        for b in range(self.ref.shape[0]):
            here = live[b]
            if not bool(here.any()):
                continue
            if not bool(torch.isfinite(got[b][here]).all()):
                out.append(f"sequence {b}: not finite")
                continue
            if bool((off[b][here] > self.bound[b][here]).any()):
                k = (off[b] / self.bound[b])[here & (self.bound[b] > 0)]
                out.append(f"sequence {b}: a value is {float(k.max()):.3g} of its bound")
            rows = here.any(-1)
            r = (off[b].norm(dim=-1) - self.row[b])[rows]
            if bool((r > 0).any()):
                k = (off[b].norm(dim=-1) / self.row[b])[rows & (self.row[b] > 0)]
                out.append(f"sequence {b}: a row is {float(k.max()):.3g} of its bound")
        return out

    def share(self, got):
        """The largest row error over its bound."""
        got = torch.as_tensor(got).to(self.ref)
        r = (got - self.ref).norm(dim=-1) / self.row
        return float(r[torch.isfinite(r)].max())
