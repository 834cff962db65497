"""CPU oracle of low-rank adapters beside a shared projection -- TEST INFRASTRUCTURE ONLY (same import rule as the
rest of ``oracle/``): binary64, row by row."""
from __future__ import annotations

import numpy as np


def add(Y, X, A, B, scale, ids, q_start, out):
    """out [rows][N] (binary64, holding what rows of no sequence keep) = Y + scale[a] (X A[a]^T) B[a]^T; also returns
    the error bound of fp16 results, counted from the number formats.

    T = X A^T: K products summed in fp32, each addition off by at most 2^-23 of the sum of magnitudes (truncating
    adders), the scale by 2^-24; then once to fp16 (2^-11), or to its subnormals, 2^-39 of the row's largest.
    R products summed likewise, the sum with Y by 2^-23, the result once to fp16 (2^-11, or 2^-25)."""
    out = out.copy()
    bound = np.zeros_like(out)
    n, R, K = A.shape
    for b in range(len(ids)):
        a = int(ids[b])
        for r in range(q_start[b], q_start[b + 1]):
            if not 0 <= a < n:
                out[r], bound[r] = Y[r], 0.0
                continue
            t = scale[a] * (A[a] @ X[r])
            reach = abs(scale[a]) * (np.abs(A[a]) @ np.abs(X[r]))
            dt = (K + 4) * 2.0 ** -23 * reach + 2.0 ** -11 * np.abs(t) + 2.0 ** -39 * np.abs(t).max(initial=0.0)
            mag = np.abs(B[a])
            out[r] = Y[r] + B[a] @ t
            bound[r] = (mag @ dt + (R + 4) * 2.0 ** -23 * (mag @ (np.abs(t) + dt)) + 2.0 ** -23 * np.abs(Y[r]))
            bound[r] += 2.0 ** -11 * (np.abs(out[r]) + bound[r]) + 2.0 ** -25
    return out, bound
