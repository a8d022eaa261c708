"""Calls of the paged cache's attention for the tests: a cache is filled, attended and compared with the oracle in 64
bits.

Tolerance, with u = 2^-24. A score is off by e = scale (d + 8) u sum|q k| + 4 u |s|, and a weight p = exp(s - max) by 2 e
+ 2^-21 of itself (exponential, running rescale); twice that of sum p v / sum p. The product of a weight and its row's
scale is rounded to 11 bits (bf16 outputs) or 22 (fp16's), or to 2^-29 of the row's largest such product, whichever is
coarser: the first gives 2^-11 or 2^-22 of sum p |v|, the second n 2^-29 max_t p_t A_t / sum p for n places, A_t the
largest magnitude of a value row (1.1: an e2m1 block's rounding). The few-rows kernel gives that where the values' scales
are alike; where they are not, `floor` is 2^-20 of sum_t p_t A_t / sum p. Half an ulp of the output's type on top. lse: e + u |lse| + (n / 4 + 64) u
for sums of n weights in parts.
"""
import numpy as np
import torch

import random_access_kv_gb300 as fq
from oracle import qcache as oq

U = 2.0 ** -24
TYPES = {"fp16": (torch.float16, 11), "bf16": (torch.bfloat16, 8)}
_CTX = {}


def context(fmt, d, heads, page):
    key = (fmt, d, heads, page)
    if key not in _CTX:
        _CTX[key] = fq.qc_create(*key)
    return _CTX[key]


def host(t):
    return t.double().cpu().numpy()


def half_ulp(x, bits):
    """Half the spacing of a type of `bits` significant bits at |x| (fp16's least spacing 2^-24 included)."""
    a = np.maximum(np.abs(x), 2.0 ** -14 if bits == 11 else 2.0 ** -126)
    return 2.0 ** (np.floor(np.log2(a)) - bits) * 1.0001


def rows(shape, seed, dtype=torch.float32):
    r = np.random.default_rng([seed, *shape])
    x = r.standard_normal(shape) * np.exp(r.uniform(-1, 1, (*shape[:-1], 1))) * np.exp(r.uniform(-1, 1, shape[-1]))
    return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()


def tree_words(sees):
    n_seq, t, _ = sees.shape
    bits = np.zeros((n_seq, t, -(-t // 32) * 32), dtype=np.uint64)
    bits[..., :t] = sees
    w = (bits.reshape(n_seq, t, -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(w.astype(np.uint32).view(np.int32)).cuda()


def chain(n_seq, t):
    return np.tril(np.ones((t, t), bool))[None].repeat(n_seq, 0)


class Case:
    """A cache of n_seq sequences in pages dealt at random (every byte 0xFF before the write), and one call over it. K, V:
    float32 tensors [places, heads, d] per sequence; nodes None: t each; bound: max_len (at least the lengths)."""

    def __init__(self, fmt, d, heads, page, K, V, lens, nodes, t, bound=0, seed=0):
        self.ctx, self.d, self.page, self.lens, self.t = context(fmt, d, heads, page), d, page, list(lens), t
        self.nodes = [t] * len(lens) if nodes is None else list(nodes)
        self.max_len = max([bound, *lens])
        n_seq, each = len(lens), -(-(self.max_len + t) // page)
        r = np.random.default_rng(seed)
        n_pages = n_seq * each + 2
        self.table = r.permutation(n_pages)[:n_seq * each].reshape(n_seq, each).astype(np.int32)
        self.pages = torch.full((n_pages, fq.qc_page_bytes(self.ctx)), 0xFF, dtype=torch.uint8, device="cuda")
        self.K, self.V = [], []
        for b in range(n_seq):
            n = self.lens[b] + self.nodes[b]
            at = np.arange(n)
            slots = torch.from_numpy(self.table[b][at // page].astype(np.int64) * page + at % page).cuda()
            k, v = K[b][:n].contiguous(), V[b][:n].contiguous()
            if n:
                fq.qc_write(self.ctx, k, v, slots, self.pages)
                held = torch.empty_like(k), torch.empty_like(v)
                fq.qc_read(self.ctx, self.pages, slots, *held)
                k, v = held
            self.K.append(host(k))
            self.V.append(host(v))
        assert fq.qc_status(self.ctx) == 0

    def call(self, q, sees=None, scale=None, counts=True, stream=None, table=None, lens=None):
        """out, lse as tensors; sees None: a chain, without a tree."""
        n_seq, t, hq, d = q.shape
        out = torch.full((n_seq, t, hq, d), 9.0, dtype=q.dtype, device="cuda")
        lse = torch.full((n_seq, t, hq), 9.0, device="cuda")
        ws = fq.alloc_attend_workspace(self.ctx, n_seq, t, hq, self.max_len)
        ws.fill_(0xFF)
        i32 = dict(dtype=torch.int32, device="cuda")
        args = (self.ctx, self.pages, q, torch.from_numpy(self.table if table is None else table).cuda(),
                torch.tensor(self.lens if lens is None else lens, **i32), torch.tensor(self.nodes, **i32) if counts else None,
                None if sees is None else tree_words(sees), 1 / np.sqrt(d) if scale is None else scale, self.max_len, out, lse, ws)
        torch.cuda.synchronize()
        fq.qc_attend(*args, stream)
        torch.cuda.synchronize()
        return out, lse

    def check(self, q, out, lse, sees=None, scale=None, heads=None, skip=(), floor=None):
        """Compares with the oracle; returns the largest error over its tolerance. heads: the query heads to look at;
        skip: (sequence, node) pairs that are not."""
        n_seq, t, hq, d = q.shape
        bits = 11 if q.dtype is torch.float16 else 8
        rounding = 2.0 ** -22 if bits == 11 else 2.0 ** -11
        scale = 1 / np.sqrt(d) if scale is None else scale
        sees = chain(n_seq, t) if sees is None else sees
        qh, got, glse, worst = host(q), host(out), host(lse), 0.0
        group = hq // self.K[0].shape[1]
        for b in range(n_seq):
            for i in range(t):
                if (b, i) in skip:
                    continue
                seen = np.concatenate([np.arange(self.lens[b]), self.lens[b] + np.flatnonzero(sees[b, i, :self.nodes[b]])]).astype(int)
                for h in range(hq) if heads is None else heads:
                    if i >= self.nodes[b] or not len(seen):
                        assert (got[b, i, h] == 0).all() and np.isneginf(glse[b, i, h]), (b, i, h)
                        continue
                    k, v, x = self.K[b][seen, h // group], self.V[b][seen, h // group], qh[b, i, h]
                    s = scale * (k @ x)
                    e = abs(scale) * (d + 8) * U * (np.abs(k) @ np.abs(x)).max() + 4 * U * np.abs(s).max()
                    p = np.exp(s - s.max())
                    total = p.sum()
                    want = p @ v / total
                    tol = (rounding + 4 * e + 2.0 ** -20) * (p @ np.abs(v) / total) + half_ulp(want, bits)
                    pA = 1.1 * p * np.abs(v).max(-1) / total
                    tol = tol + len(seen) * (2.0 ** -29 * pA.max() if floor is None else floor * pA.sum())
                    err = np.abs(got[b, i, h] - want)
                    assert (err <= tol).all(), ("out", b, i, h, (err / tol).max())
                    worst = max(worst, (err / tol).max())
                    wl = s.max() + np.log(total)
                    assert abs(glse[b, i, h] - wl) <= e + U * abs(wl) + (len(seen) / 4 + 64) * U, ("lse", b, i, h, glse[b, i, h], wl)
        return worst

    def run(self, q, sees=None, scale=None, **kw):
        out, lse = self.call(q, sees, scale, **kw)
        assert fq.qc_status(self.ctx) == 0
        again, lse2 = self.call(q, sees, scale, **kw)
        assert torch.equal(out, again) and torch.equal(lse, lse2), "the same call gives the same bits"
        return self.check(q, out, lse, sees, scale)


def random_case(fmt, d, heads, page, lens, nodes, t, bound=0, seed=0):
    counts = [t] * len(lens) if nodes is None else nodes
    K = [rows((a + b, heads, d), 10 * seed + i) for i, (a, b) in enumerate(zip(lens, counts))]
    V = [rows((a + b, heads, d), 5000 + 10 * seed + i) for i, (a, b) in enumerate(zip(lens, counts))]
    return Case(fmt, d, heads, page, K, V, lens, nodes, t, bound, seed)
