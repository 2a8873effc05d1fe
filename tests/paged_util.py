"""Inputs of the paged-cache tests: random pools, page tables in random order,
ragged streams."""
from __future__ import annotations

import numpy as np
import torch

from hybrid_linear_attention_arl2_b200 import arl2

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
ABI = {"f32": arl2.ARL2_F32, "bf16": arl2.ARL2_BF16}


def host(t):
    return t.detach().double().cpu().numpy()


class Paged:
    """A pool and the streams [(new tokens, cached keys)] in it.  `spare` pages
    belong to nobody; whatever no stream owns holds NaN, and so do the rows of a
    stream's last page that lie past its keys."""

    def __init__(self, dtype, H, hk, d, page, seqs, seed, spare=3, dst=()):
        g = torch.Generator().manual_seed(seed)
        self.g, self.dtype, self.H, self.hk, self.d, self.page, self.seqs = g, dtype, H, hk, d, page, list(seqs)
        n = len(seqs)
        need = [-(-kv // page) for _, kv in seqs]
        more = [-(-kv // page) for kv in dst]
        total = sum(need) + sum(more) + spare
        order = torch.randperm(total, generator=g).to(torch.int32)
        table = torch.full((n, max(need + [1])), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(need):
            table[b, :c] = order[at:at + c]
            at += c
        self.dst = torch.full((n, max(more + [1])), -1, dtype=torch.int32)
        for b, c in enumerate(more):
            self.dst[b, :c] = order[at:at + c]
            at += c
        self.tables = table
        self.kp, self.vp = (torch.full((total, hk, page, d), float("nan"), dtype=TORCH[dtype]) for _ in range(2))
        for b, (_, kv) in enumerate(seqs):
            for j in range(kv):
                for pool in (self.kp, self.vp):
                    pool[table[b, j // page], :, j % page] = self.randn(hk, d)
        self.T = sum(q for q, _ in seqs)
        self.q_start = torch.tensor(np.cumsum([0] + [q for q, _ in seqs]), dtype=torch.int32)
        self.kv_len = torch.tensor([k for _, k in seqs], dtype=torch.int32)
        self.width = max([k for _, k in seqs] + [1])

    def randn(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(TORCH[self.dtype])

    def to_gpu(self, rows=None, max_q=None, max_kv=None):
        self.kp, self.vp = self.kp.cuda(), self.vp.cuda()
        self.batch = arl2.PagedBatch(self.q_start.cuda(), self.kv_len.cuda(), self.tables.cuda(),
                                     tokens=self.T if rows is None else rows,
                                     max_q=max([q for q, _ in self.seqs]) if max_q is None else max_q,
                                     max_kv=self.width if max_kv is None else max_kv)
        self.layer = arl2.PagedKVLayer(self.H, self.hk, self.d, ABI[self.dtype], self.kp, self.vp)
        return self

    def clean(self, pool):
        """The pool in float64 (rows that nobody may read are NaN)."""
        return host(pool)


def attend_bounds(dtype, d, q, k, kv, mag, o):
    """Elementwise bounds (o, lse) of the kernels' errors, by arithmetic.

    With M the largest sum |q_i k_i| scale of a row, a logit is off by at most
    d steps of float32 of M from its products' sum (a step 2^-24; 2^-22 where the
    tensor core adds without rounding), and by 2^-24 of itself from its scaling
    and its subtraction (it is at most M); an exponential is then off by that
    much relative, and by 2^-21 for its own evaluation; the sums add 2^-24 a key.  A row's output is off by
    that relative to sum p |v|, twice (numerator and denominator); bf16 rounds
    the weights and the output, half a step (2^-8) each.
    """
    M = float(np.sqrt((q ** 2).sum(-1).max() * (k ** 2).sum(-1).max())) * d ** -0.5
    add = 2.0 ** (-24 if dtype == "f32" else -22)
    rel = d * add * M + 4 * 2.0 ** -24 * M + 2.0 ** -21 + kv * add + 16 * 2.0 ** -24
    lse = rel + 2.0 ** -22 * (M + np.log(max(kv, 2)))
    if dtype == "f32":
        return 2 * rel * mag + 2.0 ** -24 * np.abs(o) + 1e-30, lse
    return (2 * rel + 2.0 ** -8) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o) + 1e-30, lse
