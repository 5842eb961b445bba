"""Attention over exact rows and eviction from them in 64 bits, written from the definitions, and
the bounds that float32 and bf16 results are held to."""
from __future__ import annotations

import math

import numpy as np
import torch

D = 128


def visible(n, ql, m, window, sinks):
    """``[m][n]``: which rows the tokens of a sequence with ``n`` rows see (False past ``ql``)."""
    i = np.arange(m)[:, None]
    j = np.arange(n)[None, :]
    p = n - ql + i
    return (i < ql) & (j <= p) & ((j < sinks) | (j > p - window))


class Attended:
    """Outputs of queries ``[r][128]`` over rows ``[n][128]`` under ``see`` ``[r][n]``, and what the
    bounds need."""

    def __init__(self, q, k, v, see):
        q, k, v = (x.double().cpu() for x in (q, k, v))
        see = torch.as_tensor(see)
        used = see.any(0)                               # rows nobody sees may hold anything
        k, v, see = k[used], v[used], see[:, used]
        if k.shape[0] == 0:
            k, v = torch.zeros((1, D)).double(), torch.zeros((1, D)).double()
            see = torch.zeros((q.shape[0], 1), dtype=torch.bool)
        s = (q @ k.T) / math.sqrt(D)
        s = torch.where(see, s, torch.full_like(s, -math.inf))
        top = s.amax(-1, keepdim=True)
        w = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = w.sum(-1, keepdim=True)
        self.used = used
        self.w = w / torch.where(total == 0, torch.ones_like(total), total)
        self.o = self.w @ v
        self.spread = self.w @ v.abs()                  # sum of w |v|
        # products of a score: the largest sum |q_i k_i| / sqrt(128) over visible rows
        a = torch.where(see, (q.abs() @ k.abs().T) / math.sqrt(D), torch.zeros_like(s))
        self.terms = a.amax(-1, keepdim=True)
        self.n = int(see.sum(-1).max())


def weight_bound(ref: Attended):
    """Relative error of a weight w = e^s / sum e^s computed with float32 sums.

    A score sums 128 products of terms that are exact to 2^-24, in float32, with up to four partial
    sums: its error is at most (128 + 8) 2^-24 of the sum of its products' sizes. A tensor core
    may truncate where it adds, which doubles that. e^x itself is good to 2^-21 (two units of an
    approximate 2^x, the scaling by log2 e and the difference to the reference), scores of size x
    round by x 2^-23. The total adds the same error once more, and its own sum of n terms."""
    ds = ref.terms * (2 * 136 + 4) * 2.0 ** -24
    return 2 * (ds + 2.0 ** -20) + (ref.n / 16 + 256) * 2.0 ** -24


def out_bound(ref: Attended, dtype, p_dtype=torch.float32):
    """Error bound of outputs held in ``dtype``: each weight's error times |v|, a rounding of the
    weights to ``p_dtype`` before their products (bf16: half a step, 2^-8), the outputs' own
    rounding, and float32 sums of n products."""
    p = torch.finfo(p_dtype).eps / 2 if p_dtype == torch.bfloat16 else 0.0
    b = ref.spread * (weight_bound(ref) + p + (ref.n / 16 + 256) * 2.0 ** -24)
    return b + (ref.o.abs() + b) * (torch.finfo(dtype).eps / 2) + 1e-30


def evicted(mass, pos, n, budget, recent, sinks):
    """``(slots, keep)`` of one (sequence, kv-head): slot j < keep ends up with row ``slots[j]``."""
    mass, pos = np.asarray(mass)[:n].astype(np.float64), np.asarray(pos)[:n].astype(np.int64)
    keep = min(n, budget)
    if n <= budget:
        return np.arange(n), keep
    fixed = (pos < sinks) | (pos > pos.max() - recent)
    weight = np.where(fixed, np.inf, np.where(np.isnan(mass), np.finfo(np.float64).max, mass))
    kept = np.sort(np.lexsort((np.arange(n), -weight))[:budget])
    slots = np.arange(keep)
    slots[np.setdiff1d(np.arange(keep), kept)] = kept[kept >= keep]
    return slots, keep
