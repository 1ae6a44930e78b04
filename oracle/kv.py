"""The attention side of a block, restated in 64 bits: the paged FP4 cache, attention, gated norms.

TEST INFRASTRUCTURE, like the rest of the oracle. Values are decoded from the cache's bytes by the
layout of include/sharq.h; attention and the norms are float64 on exactly decoded operands. The
quantizer takes the float32 steps that the header fixes.
"""
from __future__ import annotations

import numpy as np

from .formats import E2M1_MAGNITUDES, e2m1_encode, e4m3_decode, e4m3_encode

BLOCK = {"nvfp4": 16, "mxfp4": 32}
_SIGNED = np.concatenate([E2M1_MAGNITUDES, -E2M1_MAGNITUDES])


def group_bytes(d: int, fmt: str) -> int:
    return 16 * d + 32 * (d // BLOCK[fmt])


def places(d: int, fmt: str):
    """Byte offsets inside a group of each row's K codes, V codes, K scales, V scales."""
    nb = d // BLOCK[fmt]
    kc, vc, ks, vs = (np.zeros((16, n), int) for n in (d // 2, d // 2, nb, nb))
    for r in range(16):
        h, t, j = r // 8, r // 2 % 4, r % 2
        for byte in range(d // 2):
            kc[r, byte] = r * (d // 2) + byte
            g, inside = divmod(byte, d // 16)
            at = (64 * h + 2 * (4 * g + t) + j) * 8 if d == 128 else (4 * (4 * g + t) + 2 * h + j) * 4
            vc[r, byte] = 8 * d + at + inside
        for b in range(nb):
            ks[r, b] = 16 * d + r * nb + b
            vs[r, b] = 16 * d + 16 * nb + (4 * b + t) * 4 + 2 * h + j
    return kc, vc, ks, vs


def quantize(x: np.ndarray, fmt: str, scale: np.ndarray | None):
    """float32 [..., heads, d] -> (codes, one per element; block scale bytes), in float32 steps."""
    f = np.float32
    b = BLOCK[fmt]
    y = x.astype(f).reshape(*x.shape[:-1], -1, b)
    amax = np.abs(y).max(-1)
    if fmt == "nvfp4":
        s = np.ones(x.shape[-2], f) if scale is None else scale.astype(f)
        s = s[:, None]
        byte = e4m3_encode((amax * (f(1) / (f(6) * s))).astype(f))
        d = (e4m3_decode(byte).astype(f) * s).astype(f)
        inv = np.where(d == 0, f(0), f(1) / np.where(d == 0, f(1), d)).astype(f)
    else:
        e = np.where(amax == 0, -23, np.clip(np.frexp(amax)[1] - 3, -23, 13))
        byte = (e + 127).astype(np.uint8)
        inv = np.ldexp(f(1), -e).astype(f)
    return e2m1_encode((y * inv[..., None]).astype(f)).reshape(x.shape), byte


def values(codes: np.ndarray, byte: np.ndarray, fmt: str, scale: np.ndarray | None) -> np.ndarray:
    """float64 values of codes [..., heads, d] with block scale bytes [..., heads, blocks]."""
    s = e4m3_decode(byte) if fmt == "nvfp4" else np.ldexp(1.0, byte.astype(int) - 127)
    if fmt == "nvfp4" and scale is not None:
        s = s * scale.astype(np.float64)[:, None]
    v = _SIGNED[codes].reshape(*byte.shape, BLOCK[fmt]) * s[..., None]
    return v.reshape(codes.shape)


def read_raw(pages: np.ndarray, page_size: int, heads: int, d: int, fmt: str, table_row, positions):
    """Codes [n, heads, d] and scale bytes [n, heads, blocks] of K and V at `positions`."""
    view = pages.reshape(-1, heads, page_size // 16, group_bytes(d, fmt))
    kc, vc, ks, vs = places(d, fmt)
    pos = np.asarray(positions)
    rows = view[np.asarray(table_row)[pos // page_size], :, pos % page_size // 16]  # [n, heads, bytes]
    r = pos % 16
    out = []
    for cp, sp in ((kc, ks), (vc, vs)):
        packed = np.take_along_axis(rows, cp[r][:, None].repeat(heads, 1), 2)
        codes = np.stack((packed & 15, packed >> 4), -1).reshape(len(pos), heads, d)
        out += [codes, np.take_along_axis(rows, sp[r][:, None].repeat(heads, 1), 2)]
    return out


def rstd(x: np.ndarray, eps: float) -> np.ndarray:
    """float64 1/sqrt(mean square + eps) of the last axis."""
    x = x.astype(np.float64)
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def rotate(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, interleaved: bool) -> np.ndarray:
    """float64 [tokens, heads, d] turned by position * inv_freq."""
    y = x.astype(np.float64).copy()
    half = len(inv_freq)
    a = positions.astype(np.float64)[:, None, None] * inv_freq.astype(np.float64)
    c, s = np.cos(a), np.sin(a)
    i = np.arange(half)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, v = y[..., p].copy(), y[..., q].copy()
    y[..., p], y[..., q] = u * c - v * s, v * c + u * s
    return y


def attention(q, k, v, first: int, causal: bool, window: int, scale: float, place=None):
    """One sequence: q [m, hq, d], k and v [n, h, d] float64; query i stands at first + i. Returns
    (y, lse, mass, flat, dots): mass the p-weighted sum of |v|, flat the unweighted one over the sum
    of exponentials, dots the largest sum |q||k| * scale that a query sees. `place`: truth values of the positions that have a place in the cache."""
    m, hq, d = q.shape
    n, h = k.shape[:2]
    y, mass, flat = np.zeros((m, hq, d)), np.zeros((m, hq, d)), np.zeros((m, hq, d))
    lse, dots = np.full((m, hq), -np.inf), np.zeros((m, hq))
    pos, key = first + np.arange(m)[:, None], np.arange(n)[None]
    seen = np.ones((m, n), bool) if place is None else np.broadcast_to(place, (m, n)).copy()
    if causal:
        seen &= key <= pos
        if window:
            seen &= key > pos - window
    some = seen.any(1)
    if n == 0 or not some.any():
        return y, lse, mass, flat, dots
    for i in range(hq):
        kk, vv = k[:, i * h // hq], v[:, i * h // hq]
        s = np.where(seen, q[:, i] @ kk.T * scale, -np.inf)
        top = np.where(some, s.max(1, initial=-np.inf), 0.0)
        e = np.exp(s - top[:, None])
        total = e.sum(1)
        ok = total > 0
        y[ok, i] = (e @ vv)[ok] / total[ok, None]
        mass[ok, i] = (e @ np.abs(vv))[ok] / total[ok, None]
        flat[ok, i] = (seen.astype(float) @ np.abs(vv))[ok] / total[ok, None]
        lse[ok, i] = top[ok] + np.log(total[ok])
        dots[:, i] = np.where(seen, np.abs(q[:, i]) @ np.abs(kk).T * abs(scale), 0.0).max(1)
    return y, lse, mass, flat, dots


def norm_residual(y, residual, post, gate, rows_per_gate, alpha):
    """float64 r' before its rounding, and the sum of the magnitudes of its two terms."""
    z = y.astype(np.float64)
    if post is not None:
        z = z * rstd(z, 1e-6) * post.astype(np.float64)
    if gate is not None:
        t = np.arange(len(z)) // rows_per_gate if rows_per_gate else np.zeros(len(z), int)
        z = z * gate.astype(np.float64)[t]
    r = alpha * residual.astype(np.float64)
    return r + z, np.abs(r) + np.abs(z)
