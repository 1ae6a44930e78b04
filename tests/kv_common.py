"""Batches, caches and tolerances shared by the tests of the attention-side operators."""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv as K

F32, BF16 = 2.0 ** -24, 2.0 ** -8  # half a step, relative to the value


def bf16(rng, *shape, scale=1.0):
    """bf16 normal values: the device tensor and the same values in float64."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()
    return t.cuda(), t.double().numpy()


class Setup:
    """A cache of scattered pages for sequences of given lengths, and batches over it."""

    def __init__(self, S, rng, lengths, heads, d, fmt, page, spare=2, extra_cols=0):
        self.S, self.rng, self.heads, self.d, self.fmt, self.page = S, rng, heads, d, fmt, page
        need = [-(-n // page) for n in lengths]
        self.num_pages = sum(need) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lengths), max(1, max(need)) + extra_cols), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lengths = list(lengths)
        self.k_scale = self.v_scale = None
        if fmt == "nvfp4":
            self.k_scale = (rng.uniform(0.6, 1.4, heads) * 4.0 / 2688).astype(np.float32)
            self.v_scale = (rng.uniform(0.6, 1.4, heads) * 4.0 / 2688).astype(np.float32)
        dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        self.cache = S.alloc_kv_cache(self.num_pages, page, heads, d, fmt, dev(self.k_scale), dev(self.v_scale))

    def batch(self, new, lengths=None, tokens=None, table=None, max_q=None):
        cu = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        return self.S.KVBatch(i32(cu), i32(self.lengths if lengths is None else lengths),
                              i32(self.table if table is None else table),
                              max(1, max(new)) if max_q is None else max_q, int(cu[-1]) if tokens is None else tokens)

    def fill(self, k_mul=1.0, v_mul=1.0):
        """Append random keys and values at every position of every sequence."""
        qkv, _ = bf16(self.rng, sum(self.lengths), 3 * self.heads * self.d)
        qkv = qkv.view(-1, 3, self.heads, self.d)
        qkv[:, 1] *= k_mul
        qkv[:, 2] *= v_mul
        self.S.sharq_kv_append(qkv.view(len(qkv), -1), self.cache, self.batch(self.lengths), self.heads)
        return self

    def raw(self, b, positions):
        return K.read_raw(self.cache.pages.cpu().numpy(), self.page, self.heads, self.d, self.fmt, self.table[b], positions)

    def kv(self, b, n):
        """Float64 keys and values of the first n positions of sequence b, from the cache's bytes."""
        kc, ks, vc, vs = self.raw(b, np.arange(n))
        return K.values(kc, ks, self.fmt, self.k_scale), K.values(vc, vs, self.fmt, self.v_scale)


def check_attention(y, lse, ref, where=""):
    """y bf16 and lse against the oracle's (y, lse, mass, flat, dots). Scores: products of exact
    operands summed in float32, off by at most d * 2^-24 of the magnitudes' sum (2^-16 of `dots`
    covers d up to 256). Probabilities are rounded to float16 against a running maximum of at most
    the final one: 2^-11 relative (of `mass`) down to 2^-14, 2^-25 absolute (of `flat`) below. y is
    rounded to bf16."""
    ry, rl, mass, flat, dots = ref
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty), where
    assert not y[empty].any(), where
    assert np.isfinite(y).all(), where
    ds = dots * 2.0 ** -16 + 2.0 ** -20
    tol = np.abs(ry) * BF16 + mass * (2.0 ** -11 + 2 * ds[..., None]) + flat * 2.0 ** -25 + 1e-30
    over = np.abs(y - ry) / tol
    assert over.max(initial=0.0) <= 1.0, (where, over.max(), np.unravel_index(over.argmax(), over.shape))
    dl = np.abs(lse[~empty] - rl[~empty])
    assert (dl <= ds[~empty] + np.abs(rl[~empty]) * 2.0 ** -22 + 2.0 ** -18).all(), (where, dl.max())
