"""CPU oracle of the paged 8-bit KV cache with a scale per page and head -- TEST
INFRASTRUCTURE ONLY (same import rule as the rest of ``oracle/``).

Quantisation is decided in binary32 with round-to-nearest-even at each step (the
codes are discrete, so the oracle takes the kernels' precision); attention is in
binary64 on the values that the codes stand for.  Sequences, heads and pages
are walked one by one.  Formats: "int8" (codes int8) and "e4m3" (codes uint8 bits).
"""
from __future__ import annotations

import numpy as np

FLOOR = np.float32(2.0 ** -30)
QMAX = {"int8": np.float32(127), "e4m3": np.float32(448)}
STEP = {f: np.float32(1) / q for f, q in QMAX.items()}  # a scale is the maximum times this


def _e4m3_values() -> np.ndarray:
    """Value of each non-negative e4m3 code 0 .. 126 (127 is NaN): 4 exponent bits
    with bias 7, 3 mantissa bits, exponent 0 subnormal."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


_E4M3 = _e4m3_values()


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    """The numbers that codes stand for, binary64 (an e4m3 NaN code: NaN)."""
    if fmt == "int8":
        return codes.view(np.int8).astype(np.float64)
    u = codes.view(np.uint8)
    mag = np.append(_E4M3, np.nan)[u & 127]
    return np.where(u & 128, -mag, mag)


def encode(y: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest code of binary32 y, ties to even, saturating; as int8 (int8) or uint8 bits (e4m3)."""
    y = np.asarray(y, dtype=np.float32)
    if fmt == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8)
    a = np.minimum(np.abs(y).astype(np.float64), 448.0)
    hi = np.clip(np.searchsorted(_E4M3, a), 1, 126)  # _E4M3[hi - 1] <= a <= _E4M3[hi]
    up, down = _E4M3[hi] - a, a - _E4M3[hi - 1]
    c = np.where(down < up, hi - 1, np.where(up < down, hi, np.where(hi & 1, hi - 1, hi)))
    return (c | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def finite(x: np.ndarray, top: float) -> np.ndarray:
    """NaN to 0, infinities to the type's largest finite value."""
    return np.clip(np.nan_to_num(x.astype(np.float32), nan=0.0), -np.float32(top), np.float32(top))


def append(codes, scales, table, kv_len, q_start, x, fmt, top=65504.0):
    """New rows x [rows][Hkv][D] into codes [pages][Hkv][T][D] and scales [pages][Hkv], in place."""
    pages, Hkv, T, _ = codes.shape
    x = finite(x, top)
    for b in range(table.shape[0]):
        n, length = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        old = length - n
        for blk in range(max(old, 0) // T, -(-length // T) if n else 0):
            page = table[b, blk]
            if not 0 <= page < pages:
                continue
            lo, hi = max(old, blk * T, 0), min(length, (blk + 1) * T)
            for h in range(Hkv):
                new = x[q_start[b] + lo - old:q_start[b] + hi - old, h]
                s = max(np.float32(np.abs(new).max() * STEP[fmt]), FLOOR)
                if old > blk * T:
                    was = scales[page, h]
                    if s > was:
                        part = codes[page, h, :lo - blk * T]
                        part[...] = encode(decode(part, fmt).astype(np.float32) * was / s, fmt)
                    s = max(s, was)
                scales[page, h] = s
                codes[page, h, lo - blk * T:hi - blk * T] = encode(new / s, fmt)


def tokens(codes, scales, row, length, h, fmt):
    """Values [length][D] of a sequence's head, and which tokens are there (not in a hole)."""
    pages, _, T, D = codes.shape
    x, there = np.zeros((length, D)), np.zeros(length, dtype=bool)
    for j in range(length):
        p = row[j // T]
        if 0 <= p < pages:
            x[j] = decode(codes[p, h, j % T], fmt) * np.float64(scales[p, h])
            there[j] = True
    return x, there


def attention(Q, k, v, ks, vs, table, kv_len, q_start, fmt, scale=None):
    """Q [rows][Hq][D] (binary64 values) -> out, lse [rows][Hq], w [B][Hkv][max len], and for
    error bounds sum p |v| [rows][Hq][D] and max_j scale sum |q k| [rows][Hq]."""
    rows, Hq, D = Q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    size, reach = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
    w = np.zeros((table.shape[0], Hkv, max(1, int(max(kv_len, default=0)))))
    for b in range(table.shape[0]):
        n, length = int(q_start[b + 1] - q_start[b]), max(int(kv_len[b]), 0)
        for h in range(Hkv):
            kh, there = tokens(k, ks, table[b], length, h, fmt)
            vh, _ = tokens(v, vs, table[b], length, h, fmt)
            for i in range(n):
                seen = there & (np.arange(length) <= length - n + i)
                if not seen.any():
                    continue
                for g in range(G):
                    r, hq = q_start[b] + i, h * G + g
                    s = scale * (kh @ Q[r, hq])
                    m = s[seen].max()
                    e = np.where(seen, np.exp(np.where(seen, s, 0.0) - m), 0.0)
                    p = e / e.sum()
                    out[r, hq], lse[r, hq] = p @ vh, m + np.log(e.sum())
                    size[r, hq] = p @ np.abs(vh)
                    reach[r, hq] = abs(scale) * (np.abs(kh[seen]) @ np.abs(Q[r, hq])).max()
                    w[b, h, :length] += p
    return out, lse, w, size, reach


def evict(pools, table, dst_table, kv_len, w, budget, first, recent, fmt):
    """pools: [(codes, scales)] of keys and values, changed in place.  Returns kept, new_len, w_out."""
    B, Hkv, _ = w.shape
    pages, _, T, D = pools[0][0].shape
    kept = np.full((B, Hkv, budget), -1, dtype=np.int32)
    w_out = np.zeros((B, Hkv, budget), dtype=np.float32)
    new_len = np.zeros(B, dtype=np.int32)
    before = [(c.copy(), s.copy()) for c, s in pools]
    for b in range(B):
        length = max(int(kv_len[b]), 0)
        count = min(length, budget)
        new_len[b] = count
        for h in range(Hkv):
            def rank(j):
                if j < first or j >= length - recent:
                    return (0, 0.0, j)
                if not 0 <= table[b, j // T] < pages or np.isnan(w[b, h, j]):
                    return (2, 0.0, j)
                return (1, -float(w[b, h, j]), j)
            keep = sorted(sorted(range(length), key=rank)[:count])
            kept[b, h, :count] = keep
            w_out[b, h, :count] = w[b, h, keep]
            for (codes, scales), (old, old_s) in zip(pools, before):
                for blk in range(-(-count // T)):
                    to = dst_table[b, blk]
                    if not 0 <= to < pages:
                        continue
                    part = keep[blk * T:(blk + 1) * T]
                    c = np.zeros((T, D), dtype=codes.dtype)
                    s = np.zeros(T, dtype=np.float32)
                    for t, j in enumerate(part):
                        p = table[b, j // T]
                        if 0 <= p < pages:
                            c[t], s[t] = old[p, h, j % T], old_s[p, h]
                    if part[-1] == blk * T + len(part) - 1:  # nothing moved
                        p = table[b, blk]
                        there = 0 <= p < pages
                        if p != to:  # in place nothing is written
                            codes[to, h], scales[to, h] = c, old_s[p, h] if there else FLOOR
                        continue
                    x = decode(c, fmt).astype(np.float32) * s[:, None]
                    now = max(np.float32(np.abs(x).max() * STEP[fmt]), FLOOR)
                    codes[to, h], scales[to, h] = encode(x / now, fmt), now
    return kept, new_len, w_out
