"""Plain 64-bit oracle of the serving operators: top-k routing, the expert
layer of a few tokens and the low-rank adapters.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Each operator also
returns the error that fp32 arithmetic in any order may add to its result, so
that the tests' tolerances follow from the inputs:

* a sum of n products kept in fp32 is off by at most (n + 1) * U * sum |a b|,
  U = 2^-23 (half of it per operation, doubled for sums inside the tensor cores,
  which may truncate);
* rounding an intermediate to MXFP8 is a step: where the 64-bit value lies
  within its own error of a rounding boundary (or the block's largest value of
  a power of two), the fp32 path may land one step away, and the step itself
  times the following weight row is added.
"""

from __future__ import annotations

import numpy as np

from .mx import BLOCK, dequantize_mx, quantize_mx_rowwise

U = 2.0 ** -23


def route(logits: np.ndarray, k: int, renormalize: bool):
    """logits float64 [T, E] -> (ids int32 [T, k], weights float64 [T, k])."""
    T = logits.shape[0]
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        row = [(-float(v), e) for e, v in enumerate(logits[t]) if v > -np.inf]
        if not row:
            continue
        row.sort()
        top = -row[0][0]
        p = [1.0 if -v == top else np.exp(-v - top) for v, _ in row]
        total = sum(p[:k]) if renormalize else sum(p)
        for j, (_, e) in enumerate(row[:k]):
            ids[t, j] = e
            weights[t, j] = p[j] / total
    return ids, weights


def mxfp8_f64(h: np.ndarray, err: np.ndarray):
    """float64 rows -> (MXFP8 values, how far a value within `err` of h may
    round from them)."""
    b = h.reshape(*h.shape[:-1], -1, BLOCK)
    eb = err.reshape(b.shape)
    amax = np.abs(b).max(-1, keepdims=True)
    at = np.argmax(np.abs(b), -1, keepdims=True)
    aerr = np.take_along_axis(eb, at, -1) + eb.max(-1, keepdims=True)

    def exponent(a):
        return np.where(a > 0, np.clip(np.frexp(np.where(a > 0, a, 1.0))[1] - 9, -127, 127), -127)

    e = exponent(amax)
    lo, hi = exponent(np.maximum(amax - aerr, 0)), exponent(amax + aerr)

    def rounded(v, e):
        s = np.abs(v) * 2.0 ** -e.astype(np.float64)
        p = np.maximum(np.frexp(np.where(s > 0, s, 1.0))[1] - 1, -6)
        step = 2.0 ** (p - 3.0)
        q = np.minimum(np.rint(s / step) * step, 448.0)  # rint: ties to even
        return np.sign(v) * q * 2.0 ** e.astype(np.float64)

    q = rounded(b, e)
    off = np.zeros_like(b)
    for ee in (lo, e, hi):
        for v in (b - eb, b + eb):
            off = np.maximum(off, np.abs(rounded(v, ee) - q))
    return q.reshape(h.shape), off.reshape(h.shape)


def moe_experts(x_bits, ids, weights, w13, w2, E):
    """x_bits: BF16 bits [T, H]; w13 [E * 2I, H], w2 [E * H, I]: dequantized
    float64 weights.  Returns (out float64 [T, H], error bound [T, H])."""
    T, H = x_bits.shape
    I = w2.shape[1]
    codes, sc = quantize_mx_rowwise(x_bits, "e4m3")
    xq = dequantize_mx(codes, sc, "e4m3")
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            W = w13[e * 2 * I:(e + 1) * 2 * I]
            gu = W @ xq[t]
            du = (H + 1) * U * (np.abs(W) @ np.abs(xq[t]))
            g, u, dg, dv = gu[:I], gu[I:], du[:I], du[I:]
            with np.errstate(over="ignore"):
                sig = 1.0 / (1.0 + np.exp(-g))
            h = g * sig * u
            # |d silu| <= 1.1; the exponential, division and products add a few units
            dh = 1.1 * dg * (np.abs(u) + dv) + np.abs(g * sig) * dv + 16 * U * np.abs(h)
            hq, off = mxfp8_f64(h[None], dh[None])
            W = w2[e * H:(e + 1) * H]
            w = float(weights[t, j])
            out[t] += w * (W @ hq[0])
            bound[t] += abs(w) * (np.abs(W) @ off[0] + (I + 8) * U * (np.abs(W) @ (np.abs(hq[0]) + off[0])))
    return out, bound


def lora_add(y, x, A, B, ids, scale):
    """All float64 (A [n, R, K], B [n, N, R]); ids int [T].  Returns (out, bound)."""
    out, bound = y.copy(), np.zeros_like(y)
    R, K = A.shape[1:]
    for t, a in enumerate(ids):
        if a < 0:
            continue
        u = A[a] @ x[t]
        du = (K + 1) * U * (np.abs(A[a]) @ np.abs(x[t]))
        s = float(scale[a])
        out[t] += s * (B[a] @ u)
        bound[t] = abs(s) * (np.abs(B[a]) @ (du + (R + 4) * U * np.abs(u))) + U * np.abs(out[t])
    return out, bound
