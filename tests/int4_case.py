"""A batch's cache [BF16 sink | INT4 history | BF16 recent] with the 64-bit arithmetic its tests compare with.

Host plumbing and plain numpy in float64, written from the definitions in include/oscar_int4.h.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from bit_kv_cache_oscar_gb300 import binding as ob

D = 128


def bf16(a) -> np.ndarray:
    """float values rounded to bf16 (from float32), as float64."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def bf16_once(a) -> np.ndarray:
    """float64 values rounded once to bf16 (nearest, ties to even), as float64; magnitudes of normal bf16 numbers."""
    a = np.asarray(a, np.float64)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(a), 2.0 ** -126))) - 7)
    return np.rint(a / step) * step


def quantize(x: np.ndarray, group: int, clip: float):
    """Rows [..., 128] -> codes [..., 128] and (scale, zero) [..., 128 / group] as stored, float64."""
    g = x.reshape(x.shape[:-1] + (D // group, group))
    c = np.float32(clip)
    lo = c * (g.min(-1).astype(np.float32) + np.float32(0))
    hi = c * (g.max(-1).astype(np.float32) + np.float32(0))
    zero, scale = bf16(lo), bf16((hi - lo) / np.float32(15))
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.clip(np.rint((g - zero[..., None]) / scale[..., None]), 0, 15)
    return np.where(scale[..., None] == 0, 0, code).reshape(x.shape), scale, zero


def unpack(codes: np.ndarray) -> np.ndarray:
    return np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (D,)).astype(np.float64)


def restore(codes, sz, kind: int, group: int) -> np.ndarray:
    """uint8 [..., 64], float64 [..., groups, 4] -> the values they stand for [..., 128]."""
    q = unpack(codes).reshape(codes.shape[:-1] + (D // group, group))
    return (sz[..., 2 * kind + 1, None] + q * sz[..., 2 * kind, None]).reshape(codes.shape[:-1] + (D,))


def tables(batch: int, spans, page_size: int, max_pages: int, rng, spare: int = 2):
    """A page table with a random physical page for every page that touches a span of its request."""
    t = np.full((batch, max_pages), -1, np.int32)
    for b, ranges in enumerate(spans):
        for lo, hi in ranges:
            if hi > lo:
                t[b, lo // page_size:(hi + page_size - 1) // page_size] = 0
    n = int((t == 0).sum())
    t[t == 0] = rng.permutation(n + spare)[:n]
    return t, n + spare


class Cache:
    """seq / hist: tokens and history end of each request; every slot of both pools outside them holds rubbish."""

    def __init__(self, seq, hist=None, n_kv=2, gqa=4, page=16, group=128, sink=64, recent=256, seed=0, extra_pages=0,
                 scale_k=1.0, scale_v=1.0, q_size=1.0, rubbish=True):
        self.rng = rng = np.random.default_rng(seed)
        self.L = ob.Layout(n_kv, gqa, page, group, sink, recent)
        self.seq = np.asarray(seq, np.int64)
        self.hist = np.minimum(self.seq, np.maximum(sink, self.seq - recent)) if hist is None else np.asarray(hist, np.int64)
        self.B = len(seq)
        self.max_pages = max(1, -(-int(self.seq.max()) // page)) + extra_pages
        self.t4, n4 = tables(self.B, [[(sink, int(h))] for h in self.hist], page, self.max_pages, rng)
        self.tb, nb = tables(self.B, [[(0, min(sink, int(t))), (int(h), int(t))] for t, h in zip(self.seq, self.hist)], page,
                             self.max_pages, rng)
        shp = (n4, n_kv, page)
        self.ck = rng.integers(0, 256, shp + (D // 2,), dtype=np.uint8)
        self.cv = rng.integers(0, 256, shp + (D // 2,), dtype=np.uint8)
        s = rng.uniform(0.1, 0.4, shp + (D // group, 2)) * [scale_k, scale_v]
        z = -s * rng.uniform(5, 10, s.shape)
        self.sz = bf16(np.stack([s[..., 0], z[..., 0], s[..., 1], z[..., 1]], -1))
        bshape = (nb, page, n_kv, D)
        self.bk, self.bv = bf16(rng.normal(0, 1.3 * scale_k, bshape)), bf16(rng.normal(0, 1.3 * scale_v, bshape))
        self.q = bf16(rng.normal(0, q_size, (self.B, n_kv * gqa, D)))
        self.sm_scale = 1 / math.sqrt(D)
        if rubbish:                                   # what no position of the batch holds must not be read into a result
            used4, usedb = np.zeros((n4, page), bool), np.zeros((nb, page), bool)
            for b in range(self.B):
                for p in range(int(self.seq[b])):
                    if sink <= p < self.hist[b]:
                        used4[self.t4[b, p // page], p % page] = True
                    else:
                        usedb[self.tb[b, p // page], p % page] = True
            self.sz.transpose(0, 2, 1, 3, 4)[~used4] = np.nan
            self.bk[~usedb], self.bv[~usedb] = np.nan, np.inf

    def upload(self, device="cuda"):
        put = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(device=device, dtype=t)
        self.int4 = ob.Int4Pool(put(self.ck, torch.uint8), put(self.cv, torch.uint8), put(self.sz, torch.bfloat16))
        self.bfp = ob.Bf16Pool(put(self.bk, torch.bfloat16), put(self.bv, torch.bfloat16))
        self.d4, self.db = put(self.t4, torch.int32), put(self.tb, torch.int32)
        self.dT, self.dh = put(self.seq, torch.int32), put(self.hist, torch.int32)
        self.dq = put(self.q, torch.bfloat16)
        return self

    def attention_args(self):
        return (self.L, self.dq, self.bfp, self.db, self.int4, self.d4, self.dT, self.dh, self.sm_scale)

    def rows(self, b, h, kind):
        """Rows of every position of (request, kv head) in float64 [T, 128]."""
        L, T, he, ps = self.L, int(self.seq[b]), int(self.hist[b]), self.L.page_size
        x = np.empty((T, D))
        p = np.arange(T)
        far = (p >= L.sink) & (p < he)
        pf, pn = p[far], p[~far]
        pg = self.t4[b, pf // ps]
        x[far] = restore((self.ck, self.cv)[kind][pg, h, pf % ps], self.sz[pg, h, pf % ps], kind, L.group)
        x[~far] = (self.bk, self.bv)[kind][self.tb[b, pn // ps], pn % ps, h]
        return x

    def logits(self, b, hq):
        return self.rows(b, hq // self.L.gqa, 0) @ self.q[b, hq] * self.sm_scale

    def logit_error(self):
        """How far a logit may be off: q·k as scale·(q·code) + zero·sum(q) has |q|·(15 scale + |zero|) as the sum of its
        terms' sizes, in at most 8 accumulation steps and 4 further fp32 operations of 2^-23 each (BF16 rows: |q|·|k|)."""
        sz, bk = np.abs(np.nan_to_num(self.sz)), np.where(np.isfinite(self.bk), np.abs(self.bk), 0)
        size = max((15 * sz[..., 0] + sz[..., 1]).max(), bk.max())
        return 12 * 2.0 ** -23 * self.sm_scale * np.abs(self.q).sum(-1).max() * size

    def attention(self):
        """Output [B, Hq, 128] and log-sum-exp [B, Hq] in float64."""
        out, lse = np.zeros(self.q.shape), np.full(self.q.shape[:2], -np.inf)
        for b in range(self.B):
            for hq in range(self.L.n_q_heads):
                if self.seq[b] == 0:
                    continue
                z = self.logits(b, hq)
                m = z.max()
                p = np.exp(z - m)
                lse[b, hq] = m + np.log(p.sum())
                out[b, hq] = p @ self.rows(b, hq // self.L.gqa, 1) / p.sum()
        return out, lse

    def output_error(self):
        """How far an output may be off.  A probability times its value scale is rounded to fp16, half a step of 2^-11
        relative, and meets codes up to 15: 2^-11·15 scale, weighted by probabilities that sum to 1 (the running maximum's
        slack keeps fp16 subnormals 2^-24 below that).  A logit error e changes a probability by 2 e, which meets the
        largest value.  Twenty fp32 operations of 2^-24 on values of that size cover sums and the final division."""
        sz = np.abs(np.nan_to_num(self.sz))
        span = (15 * sz[..., 2]).max()
        size = max(span + sz[..., 3].max(), np.where(np.isfinite(self.bv), np.abs(self.bv), 0).max())
        return 2.0 ** -11 * span + (2 * self.logit_error() + 20 * 2.0 ** -24) * size
