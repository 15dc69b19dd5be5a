"""FP4 KV cache in numpy and 64 bits: the format, its quantising write and
read-back, and attention over it, written from the definitions in
``include/pa.h`` ("FP4 KV cache").  Test infrastructure, like the rest of this
package; it shares no code with the CUDA library.

Element values are looked up in tables made from the bit layouts; the nearest
value of a table is found by comparing exact distances.
"""
from __future__ import annotations

import numpy as np


def _e2m1(code: int) -> float:
    sign, e, m = code >> 3, (code >> 1) & 3, code & 1
    v = m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
    return -v if sign else v


def _e4m3(code: int) -> float:
    sign, e, m = code >> 7, (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if sign else v


E2M1 = np.array([_e2m1(c) for c in range(16)])
E4M3 = np.array([_e4m3(c) for c in range(256)])


def nearest(values: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Index of the entry of the increasing table ``values`` (from 0 up) nearest
    to each x >= 0, ties to the even index, beyond the last entry to the last."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(values, x, side="left"), 1, len(values) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        a, b = x - values[lo], values[hi] - x
    i = np.where(a < b, lo, hi)
    i = np.where((a == b) & (lo % 2 == 0), lo, i)
    return np.where(x >= values[-1], len(values) - 1, i)


def quantise(x: np.ndarray, g: float):
    """(codes uint8 [..., d / 2], scales uint8 [..., d / 16]) of rows x [..., d]
    (any float type whose values are exact in fp32)."""
    x = np.asarray(x, np.float32)
    blk = x.reshape(*x.shape[:-1], -1, 16)
    g = np.float32(g)
    with np.errstate(all="ignore"):
        top = np.abs(blk).max(-1)
        want = top / (np.float32(6.0) * g)
        nan = np.isnan(blk).any(-1)
        s = nearest(E4M3[:127], np.where(nan, 0, want)).astype(np.uint8)
        s = np.where(nan, 0x7F, s).astype(np.uint8)
        z = E4M3[s].astype(np.float32) * g
        inv = np.float32(1.0) / z
        y = blk * inv[..., None]
        keep = (~nan & (s != 0))[..., None]
        mag = nearest(E2M1[:8], np.abs(np.where(keep, y, 0)))
        code = np.where(keep, mag + 8 * np.signbit(y), 0).astype(np.uint8)
    code = code.reshape(x.shape)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), s


def views(cache: np.ndarray, bs: int, d: int):
    """Views of the codes [NB, Hkv, bs, d / 2] and the scales [NB, Hkv, bs, d / 16] of a cache."""
    NB, H, n = cache.shape
    st = cache.strides
    c = np.lib.stride_tricks.as_strided(cache, (NB, H, bs, d // 2), (st[0], st[1], d // 2, 1))
    s = np.lib.stride_tricks.as_strided(cache[:, :, bs * d // 2:], (NB, H, bs, d // 16),
                                        (st[0], st[1], d // 16, 1))
    return c, s


def reshape_and_cache(key, value, k_cache, v_cache, slots, bs: int, k_scale: float,
                      v_scale: float) -> None:
    """The quantising write, in place; key, value [T, Hkv, d] in fp32 or wider."""
    d = key.shape[2]
    for x, cache, g in ((key, k_cache, k_scale), (value, v_cache, v_scale)):
        c, s = views(cache, bs, d)
        codes, scales = quantise(x, g)
        for t, slot in enumerate(slots):
            if slot >= 0:
                c[slot // bs, :, slot % bs] = codes[t]
                s[slot // bs, :, slot % bs] = scales[t]


def values(cache: np.ndarray, bs: int, d: int, g: float) -> np.ndarray:
    """[NB, Hkv, bs, d]: what every code of a cache stands for, in 64 bits."""
    c, s = views(cache, bs, d)
    e = np.stack([E2M1[c & 15], E2M1[c >> 4]], -1).reshape(*c.shape[:-1], d)
    return e * np.repeat(E4M3[s], 16, axis=-1) * float(np.float32(g))


def context(vals: np.ndarray, table_row, n: int) -> np.ndarray:
    """[Hkv, n, d]: a sequence's first n tokens out of ``values``'s result."""
    bs = vals.shape[2]
    ids = np.asarray(table_row)[: -(-n // bs)]
    x = vals[ids].transpose(1, 0, 2, 3)
    return x.reshape(x.shape[0], -1, x.shape[3])[:, :n]


def attend(q, K, V, scale: float, ends) -> np.ndarray:
    """q [rows, Hq, d] over K, V [Hkv, n, d]; row r sees the keys 0..ends[r] - 1."""
    rows, Hq, d = q.shape
    G = Hq // K.shape[0]
    out = np.zeros((rows, Hq, d))
    ends = np.asarray(ends)
    seen = np.arange(K.shape[1]) < ends[:, None]
    for h in range(Hq):
        z = np.where(seen, (q[:, h] @ K[h // G].T) * scale, -np.inf)
        top = z.max(-1, keepdims=True, initial=-np.inf)
        e = np.exp(z - np.where(np.isinf(top), 0, top))
        l = e.sum(-1, keepdims=True)
        v = V[h // G]
        gone = np.isnan(v)
        out[:, h] = (e / np.where(l == 0, 1, l)) @ np.where(gone, 0, v)
        # a NaN of V reaches the rows that see its key, and no others
        out[:, h][seen.astype(float) @ gone > 0] = np.nan
    return out


def decode(q, k_vals, v_vals, tables, lens, scale: float) -> np.ndarray:
    """q [B, Hq, d] in 64 bits; the caches as ``values`` gives them."""
    out = np.zeros(q.shape)
    for i, n in enumerate(lens):
        if n > 0:
            out[i] = attend(q[i:i + 1], context(k_vals, tables[i], n),
                            context(v_vals, tables[i], n), scale, [n])[0]
    return out


def prefill(q, start, k_vals, v_vals, tables, lens, scale: float) -> np.ndarray:
    """q [total_q, Hq, d]; chunk row t of sequence i sees keys 0..len - q_len + t."""
    out = np.zeros(q.shape)
    for i, n in enumerate(lens):
        a, b = int(start[i]), int(start[i + 1])
        if b > a:
            ends = n - (b - a) + 1 + np.arange(b - a)
            out[a:b] = attend(q[a:b], context(k_vals, tables[i], n),
                              context(v_vals, tables[i], n), scale, ends)
    return out
