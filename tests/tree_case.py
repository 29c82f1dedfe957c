"""A batch's mixed cache with a tree of nodes behind each request, and the 64-bit arithmetic its tests compare with.

Plain numpy in float64, written from the definitions in include/oscar_tree.h.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import int4_case as ic

D = 128


def random_parents(n, rng, near=8):
    """Node 0 is the root; a node's parent is one of the `near` nodes before it."""
    return np.array([-1] + [rng.integers(max(0, j - near), j) for j in range(1, n)], np.int32)


def ancestors(parents):
    """sees[i, j]: node i sees node j, itself and its ancestors."""
    n = len(parents)
    sees = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            sees[i] = sees[p]
        sees[i, i] = True
    return sees


class TreeCache:
    """seq: tokens of each request, nodes: of each tree; every slot of both pools that holds none is rubbish."""

    def __init__(self, seq, nodes, hist=None, n_kv=2, gqa=4, page=16, group=128, sink=64, recent=256, seed=0, chain=False, sees=None,
                 scale_k=1.0, scale_v=1.0, q_size=1.0, extra_rows=0, extra_pages=0, words=None):
        self.rng = rng = np.random.default_rng(seed)
        self.L = ob.Layout(n_kv, gqa, page, group, sink, recent)
        self.seq, self.nodes = np.asarray(seq, np.int64), np.asarray(nodes, np.int64)
        self.hist = np.minimum(self.seq, np.maximum(sink, self.seq - recent)) if hist is None else np.asarray(hist, np.int64)
        self.B, self.most, self.chain = len(seq), max(1, int(self.nodes.max())), chain
        self.begin = np.concatenate([[0], np.cumsum(self.nodes)])
        self.n = int(self.begin[-1]) + extra_rows
        self.parents = [random_parents(n, rng) if n else np.zeros(0, np.int32) for n in self.nodes]
        self.sees = sees if sees is not None else [np.tril(np.ones((n, n), bool)) if chain else ancestors(p) for n, p in zip(self.nodes, self.parents)]
        self.max_pages = -(-int((self.seq + self.nodes).max()) // page) + extra_pages
        self.max_pages = max(1, self.max_pages)
        self.t4, n4 = ic.tables(self.B, [[(sink, int(h))] for h in self.hist], page, self.max_pages, rng)
        self.tb, nb = ic.tables(self.B, [[(0, min(sink, int(t))), (int(h), int(t + n))] for t, h, n in zip(self.seq, self.hist, self.nodes)], page,
                                self.max_pages, rng)
        shp = (n4, n_kv, page)
        self.ck = rng.integers(0, 256, shp + (D // 2,), dtype=np.uint8)
        self.cv = rng.integers(0, 256, shp + (D // 2,), dtype=np.uint8)
        s = rng.uniform(0.1, 0.4, shp + (D // group, 2)) * [scale_k, scale_v]
        z = -s * rng.uniform(5, 10, s.shape)
        self.sz = ic.bf16(np.stack([s[..., 0], z[..., 0], s[..., 1], z[..., 1]], -1))
        bshape = (nb, page, n_kv, D)
        self.bk, self.bv = ic.bf16(rng.normal(0, 1.3 * scale_k, bshape)), ic.bf16(rng.normal(0, 1.3 * scale_v, bshape))
        self.q = ic.bf16(rng.normal(0, q_size, (self.n, n_kv * gqa, D)))
        self.sm_scale = 1 / math.sqrt(D)
        words = words or (self.most + 31) // 32
        bits = np.ones((self.n, words * 32), bool)             # bits beyond a request's nodes are not read
        for b in range(self.B):
            lo, n = int(self.begin[b]), int(self.nodes[b])
            bits[lo:lo + n, :n] = self.sees[b]
        self.mask = np.packbits(bits, axis=1, bitorder="little").view("<i4")
        used4, usedb = np.zeros((n4, page), bool), np.zeros((nb, page), bool)
        for b in range(self.B):
            for p in range(int(self.seq[b] + self.nodes[b])):
                if sink <= p < self.hist[b]:
                    used4[self.t4[b, p // page], p % page] = True
                else:
                    usedb[self.tb[b, p // page], p % page] = True
        self.sz.transpose(0, 2, 1, 3, 4)[~used4] = np.nan
        self.bk[~usedb], self.bv[~usedb] = np.nan, np.inf

    def upload(self, device="cuda"):
        put = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(device=device, dtype=t)  # noqa: E731
        self.int4 = ob.Int4Pool(put(self.ck, torch.uint8), put(self.cv, torch.uint8), put(self.sz, torch.bfloat16))
        self.bfp = ob.Bf16Pool(put(self.bk, torch.bfloat16), put(self.bv, torch.bfloat16))
        self.d4, self.db = put(self.t4, torch.int32), put(self.tb, torch.int32)
        self.dT, self.dh, self.dbegin = put(self.seq, torch.int32), put(self.hist, torch.int32), put(self.begin, torch.int32)
        self.dq, self.dmask = put(self.q, torch.bfloat16), None if self.chain else put(self.mask, torch.int32)
        return self

    def run(self, splits=None, out=None, lse=None, partials=None, stream=None):
        L = self.L
        S = splits or ob.oscar_suggest_splits_tree_int4(L, self.B, self.most, max(1, int(self.seq.max())), 152)
        out = torch.full((self.n, L.n_q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        lse = torch.full((self.n, L.n_q_heads), 7.0, device="cuda") if lse is None else lse
        part = ob.Partials.empty(L, self.n, S) if partials is None else partials
        ob.oscar_tree_attention_int4(L, self.dq, self.dbegin, self.dmask, self.most, self.bfp, self.db, self.int4, self.d4, self.dT, self.dh,
                                     self.sm_scale, part, out, lse, stream=stream)
        return out, lse

    def rows(self, b, h, kind):
        """Rows of every position and node of (request, kv head) in float64."""
        L, T, he, ps = self.L, int(self.seq[b]), int(self.hist[b]), self.L.page_size
        p = np.arange(T + int(self.nodes[b]))
        x = np.empty((len(p), D))
        far = (p >= L.sink) & (p < he)
        pf, pn = p[far], p[~far]
        pg = self.t4[b, pf // ps]
        x[far] = ic.restore((self.ck, self.cv)[kind][pg, h, pf % ps], self.sz[pg, h, pf % ps], kind, L.group)
        x[~far] = (self.bk, self.bv)[kind][self.tb[b, pn // ps], pn % ps, h]
        return x

    def attention(self):
        """Output [n, Hq, 128] and log-sum-exp [n, Hq] in float64; rows without a node are 7, as run() leaves them."""
        out, lse = np.full(self.q.shape, 7.0), np.full(self.q.shape[:2], 7.0)
        G = self.L.gqa
        for b in range(self.B):
            T, lo, n = int(self.seq[b]), int(self.begin[b]), int(self.nodes[b])
            for h in range(self.L.n_kv_heads):
                K, V = self.rows(b, h, 0), self.rows(b, h, 1)
                for i in range(n):
                    on = np.concatenate([np.ones(T, bool), self.sees[b][i]])
                    out[lo + i, h * G:(h + 1) * G], lse[lo + i, h * G:(h + 1) * G] = 0, -np.inf
                    if not on.any():
                        continue
                    z = self.q[lo + i, h * G:(h + 1) * G] @ K[on].T * self.sm_scale
                    m = z.max(1, keepdims=True)
                    p = np.exp(z - m)
                    lse[lo + i, h * G:(h + 1) * G] = (m + np.log(p.sum(1, keepdims=True)))[:, 0]
                    out[lo + i, h * G:(h + 1) * G] = p @ V[on] / p.sum(1, keepdims=True)
        return out, lse

    def logit_error(self):
        """q.k as scale (q.code) + zero sum(q) has |q| (15 scale + |zero|) as the sum of its terms' sizes, in at most 8 accumulation
        steps and 4 further fp32 operations of 2^-23 each (BF16 rows: |q| |k|)."""
        sz, bk = np.abs(np.nan_to_num(self.sz)), np.where(np.isfinite(self.bk), np.abs(self.bk), 0)
        size = max((15 * sz[..., 0] + sz[..., 1]).max(), bk.max())
        return 12 * 2.0 ** -23 * self.sm_scale * np.abs(np.nan_to_num(self.q)).sum(-1).max() * size

    def output_error(self):
        """A probability times its value scale is rounded to fp16, half a step of 2^-10 relative, and meets codes of at most 8 in
        size: 2^-11 8 scale, weighted by probabilities that sum to 1 (a BF16 row's in two bf16 parts: 2^-16 of its value).  A
        logit error e changes a probability by 2 e, which meets the largest value.  The sums: a step of 16 positions cuts off at
        most 2^-23 of what was summed, and twenty fp32 operations of 2^-24 cover the rest."""
        sz = np.abs(np.nan_to_num(self.sz))
        scale = sz[..., 2].max()
        size = max((15 * sz[..., 2] + sz[..., 3]).max(), np.where(np.isfinite(self.bv), np.abs(self.bv), 0).max())
        return 2.0 ** -11 * 8 * scale + (2.0 ** -16 + 2 * self.logit_error() + (20 + self.seq.max() / 16) * 2.0 ** -23) * size

    def check(self, out, lse, ref=None):
        o, e = ref or self.attention()
        got, want = out.double().cpu().numpy(), o
        err = self.output_error()
        bound = err + 2.0 ** -8 * (np.abs(want) + err)
        assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound).max())
        l = lse.double().cpu().numpy()
        assert np.array_equal(np.isinf(l), np.isinf(e))
        on = np.isfinite(e)
        # the log's own error and the sums': 8 operations of 2^-23 on numbers of the result's size
        assert np.all(np.abs(l[on] - e[on]) <= 2 * self.logit_error() + 8 * 2.0 ** -23 * (1 + np.abs(e[on])))
