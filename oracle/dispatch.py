"""Plain 64-bit oracle of the operators that bring tokens to the experts and
back, of their gradients, and of the 8-bit integer products.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Operators whose results
are rounded also return the error that fp32 arithmetic in any order may add, so
that the tests' tolerances follow from the inputs: a sum of n products kept in
fp32 is off by at most (n + 1) * U * sum |a b|, U = 2^-23 (half of it per
operation, doubled for sums inside the tensor cores, which may truncate).
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -23
TINY = 2.0 ** -126  # fp32 results below this lose relative accuracy


def sort(ids: np.ndarray, E: int):
    """ids int [T, k] -> (m_splits int32 [E], rows int32 [T, k]).  Ids not below
    E are empty like negative ones."""
    flat = ids.reshape(-1)
    rows = np.empty(flat.size, np.int32)
    splits = np.zeros(E, np.int32)
    at = 0
    for e in range(E):
        for i in range(flat.size):
            if flat[i] == e:
                rows[i] = at
                at += 1
                splits[e] += 1
    for i in range(flat.size):
        if flat[i] < 0 or flat[i] >= E:
            rows[i] = -1 - at
            at += 1
            splits[E - 1] += 1
    return splits, rows.reshape(ids.shape)


def place(entry: int) -> int:
    """The row that a slot's entry owns."""
    return int(entry) if entry >= 0 else -1 - int(entry)


def gather(x: np.ndarray, rows: np.ndarray):
    T, k = rows.shape
    out = np.zeros((T * k,) + x.shape[1:], x.dtype)
    for t in range(T):
        for j in range(k):
            out[place(rows[t, j])] = x[t] if rows[t, j] >= 0 else 0
    return out


def combine(y, rows, weights):
    """float64 y; weights None for 1.  Returns (out, bound)."""
    T, k = rows.shape
    out, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                v = y[rows[t, j]] * (1.0 if weights is None else weights[t, j])
                out[t] += v
                size[t] += np.abs(v)
    return out, (k + 1) * U * size


def combine_backward(dout, y, rows, weights):
    """Returns (dy, dweights, bound of dweights); dy is one product each."""
    T, k = rows.shape
    dy, dw, bound = np.zeros_like(y), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = rows[t, j]
            if r >= 0:
                dy[r] = weights[t, j] * dout[t]
                dw[t, j] = dout[t] @ y[r]
                bound[t, j] = (y.shape[1] + 1) * U * (np.abs(dout[t]) @ np.abs(y[r]))
    return dy, dw, bound


def route_backward(dweights, ids, weights, logits, E, renormalize):
    """All float64 (logits None with renormalize).  Returns (dlogits, bound)."""
    T, k = ids.shape
    out, bound = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(k) if 0 <= ids[t, j] < E]
        w, d = weights[t, on], dweights[t, on]
        s, ds = (w * d).sum(), (k + 1) * U * np.abs(w * d).sum()
        if not renormalize:
            l = logits[t]
            fine = l > -np.inf  # false for NaN
            p = np.zeros(E)
            if fine.any():
                top = l[fine].max()
                p[fine] = [1.0 if v == top else np.exp(v - top) for v in l[fine]]
                p /= p.sum()
            out[t] = -p * s
            # exp within 2 units, a sum of E terms, a division and a product
            bound[t] = p * ds + (E + 8) * U * np.abs(p * s)
        for i, j in enumerate(on):
            v = w[i] * (d[i] - s) if renormalize else w[i] * d[i]
            e = int(ids[t, j])
            bound[t, e] += U * np.abs(v) + (np.abs(w[i]) * (ds + U * (np.abs(d[i]) + np.abs(s))) if renormalize else 0.0)
            out[t, e] += v
            bound[t, e] += U * np.abs(out[t, e]) + U * np.abs(v)
    return out, bound


def int8_quantize(x: np.ndarray):
    """float32 rows (BF16 values) -> (codes int8, scale float32)."""
    codes, scale = np.zeros(x.shape, np.int8), np.zeros(x.shape[0], np.float32)
    for t, row in enumerate(x):
        if not np.isfinite(row).all():
            scale[t] = np.nan
            continue
        a = np.float32(max(np.abs(row).max(initial=0.0), 2.0 ** -100))
        r = np.float32(127) / a
        scale[t] = a / np.float32(127)
        codes[t] = np.rint(row.astype(np.float64) * np.float64(r))  # exact product, ties to even
    return codes, scale


def int8_gemm(qa, sa, qw, sw, splits):
    """Codes (integers) and float32 scales -> (y float64, bound): the product of
    the definition and what fp32 sums and the two scalings may add.  Sums are
    exact where the codes' products do not reach 2^24 in all."""
    S, N = qa.shape[0], qw.shape[0] // len(splits)
    y, bound = np.zeros((S, N)), np.zeros((S, N))
    at = 0
    for g, m in enumerate(splits):
        a, w = qa[at:at + m].astype(np.float64), qw[g * N:(g + 1) * N].astype(np.float64)
        sc = sa[at:at + m].astype(np.float64)[:, None] * sw[g * N:(g + 1) * N].astype(np.float64)
        size = np.abs(a) @ np.abs(w).T
        y[at:at + m] = (a @ w.T) * sc
        bound[at:at + m] = np.where(size < 2.0 ** 24, 0.0, (qa.shape[1] + 1) * U * size) * np.abs(sc) + 2.0 ** -23 * np.abs(y[at:at + m])
        at += m
    return y, bound
