"""Rotated append, key bounds, block selection and attention over chosen blocks,
in numpy, written from the definitions in ``include/pa.h`` ("Rotated append and
sparse attention").  Test infrastructure, like the rest of this package; it
shares no code with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np


def rotate(x: np.ndarray, positions, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """Rows x [T, H, d] (exact in fp32) at their positions, in fp32, before the
    rounding to the rows' type: element by element, each operation in fp32."""
    x = np.asarray(x, np.float32)
    out = x.copy()
    half = cos_sin.shape[1] // 2
    with np.errstate(all="ignore"):
        for t, p in enumerate(positions):
            if not 0 <= p < len(cos_sin):
                continue
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                c, s = np.float32(cos_sin[p, i]), np.float32(cos_sin[p, half + i])
                out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
                out[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return out


def exponent(a: float, most: float) -> int:
    """The smallest e >= -126 with a <= most 2^e."""
    e = -126
    while a > most * 2.0 ** e:
        e += 1
    return e


def bounds_of(keys: np.ndarray):
    """(codes int8 [2, d], scale) of one block's keys [tokens, d]."""
    a = np.abs(keys).max()
    d = keys.shape[1]
    if not np.isfinite(a):
        return np.zeros((2, d), np.int8), math.inf
    if a == 0:
        return np.zeros((2, d), np.int8), 0.0
    g = 2.0 ** exponent(a, 127)
    return np.stack([np.ceil(keys.max(0) / g), np.floor(keys.min(0) / g)]).astype(np.int8), g


def update_bounds(bounds, scales, k_values, tables, lens, q_lens) -> None:
    """In place, for the blocks of the last q_lens[i] tokens of each sequence;
    k_values [NB, H, bs, d]."""
    NB, H, bs, _ = k_values.shape
    for i, (n, q) in enumerate(zip(lens, q_lens)):
        for j in range((n - q) // bs, -(-n // bs)) if q else ():
            b = tables[i, j]
            if not 0 <= b < NB:
                continue
            for h in range(H):
                bounds[b, h], scales[b, h] = bounds_of(k_values[b, h, : n - j * bs])


def scores(q: np.ndarray, bounds: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp32 scores of blocks (bounds [n, 2, d], scales [n]) for a group of queries [G, d]."""
    a = np.abs(q).max()
    c = np.zeros(q.shape, np.int64)
    if np.isfinite(a) and a > 0:
        c = np.rint(q / 2.0 ** exponent(a, 4095)).astype(np.int64)
    w = np.stack([np.maximum(c, 0).sum(0), np.minimum(c, 0).sum(0)])
    total = (bounds.astype(np.int64) * w).sum((1, 2))
    with np.errstate(invalid="ignore", over="ignore"):
        s = total.astype(np.float32) * scales.astype(np.float32)
    return np.where(np.isinf(scales), np.float32(np.inf), s)


def choose(score: np.ndarray, keep: int, sink: int, recent: int) -> list:
    """Indices of the blocks taken, in order."""
    n = len(score)
    if n <= keep:
        return list(range(n))
    taken = set(range(min(sink, n))) | set(range(max(0, n - recent), n))
    rest = sorted((j for j in range(n) if j not in taken), key=lambda j: (-float(score[j]), j))
    return sorted(taken | set(rest[: keep - len(taken)]))


def select(q, bounds, scales, tables, seqs, seen, bs: int, keep: int, sink: int, recent: int):
    """(tables [R, H, keep], lens [R, H]) of rows q [R, Hq, d]; row r belongs to
    sequence seqs[r] and sees its first seen[r] tokens."""
    R, Hq, d = q.shape
    H = bounds.shape[1]
    out, lens = np.full((R, H, keep), -1, np.int32), np.zeros((R, H), np.int32)
    for r in range(R):
        n = -(-int(seen[r]) // bs)
        ids = tables[seqs[r], :n]
        ok = (ids >= 0) & (ids < len(bounds))
        at = np.where(ok, ids, 0)
        for h in range(H):
            s = np.zeros(0, np.float32)
            if n:
                s = scores(q[r].reshape(H, Hq // H, d)[h], bounds[at, h], scales[at, h])
                s = np.where(ok, s.astype(np.float64), -math.inf)
            got = choose(s, keep, sink, recent)
            out[r, h, : len(got)] = ids[got]
            if got:
                lens[r, h] = len(got) * bs - (n * bs - int(seen[r]) if got[-1] == n - 1 else 0)
    return out, lens


def attend(q, k_values, v_values, tables, lens, scale: float):
    """(out, A) [R, Hq, d] in 64 bits: the attention, and sum_j p_j |v_j| beside it."""
    R, Hq, d = q.shape
    H, bs = k_values.shape[1:3]
    out, mag = np.zeros((R, Hq, d)), np.zeros((R, Hq, d))
    for r in range(R):
        for h in range(Hq):
            g = h // (Hq // H)
            n = int(lens[r, g])
            if n == 0:
                continue
            ids = tables[r, g, : -(-n // bs)]
            K = k_values[ids, g].reshape(-1, d)[:n]
            V = v_values[ids, g].reshape(-1, d)[:n]
            z = K @ q[r, h] * scale
            p = np.exp(z - z.max())
            p /= p.sum()
            out[r, h], mag[r, h] = p @ V, p @ np.abs(V)
    return out, mag
