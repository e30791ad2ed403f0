"""Pins of the serving oracle: hand-worked rows, the MXFP8 rounding against
the BF16 oracle, and the adapters against a written-out sum."""

import numpy as np

import oracle
import synth
from oracle import serve


def test_route_by_hand():
    inf = np.inf
    ids, w = serve.route(np.array([[0.0, 1.0, 1.0, -inf], [-inf] * 4, [np.nan, inf, 2.0, inf], [5.0, -inf, -inf, -inf]]),
                         2, True)
    assert ids.tolist() == [[1, 2], [-1, -1], [1, 3], [0, -1]]
    assert w.tolist() == [[0.5, 0.5], [0.0, 0.0], [0.5, 0.5], [1.0, 0.0]]
    ids, w = serve.route(np.log(np.array([[1.0, 2.0, 5.0]])), 2, False)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[5 / 8, 2 / 8]], rtol=1e-15)


def test_mxfp8_matches_the_bf16_oracle():
    bits = synth.normal_bf16(np.random.default_rng(5), (9, 256), std=3.0, outlier_frac=0.02)
    codes, sc = oracle.quantize_mx_rowwise(bits, "e4m3")
    want = oracle.dequantize_mx(codes, sc, "e4m3")
    q, off = serve.mxfp8_f64(synth.bf16_bits_to_f32(bits).astype(np.float64), np.zeros((9, 256)))
    assert np.array_equal(q, want) and not off.any()


def test_mxfp8_step_is_seen_at_a_boundary():
    h = np.zeros((1, 32))
    h[0, 0], h[0, 1] = 256.0, 17.0  # 17 lies half way between 16 and 18
    q, off = serve.mxfp8_f64(h, np.where(h > 0, 1e-6, 0.0))
    assert q[0, 1] == 16.0 and off[0, 1] == 2.0


def test_lora_by_hand():
    y, x = np.zeros((2, 2)), np.array([[1.0, 2.0], [3.0, 4.0]])
    A = np.array([[[1.0, 1.0]]])
    B = np.array([[[2.0], [3.0]]])
    out, _ = serve.lora_add(y, x, A, B, [0, -1], [0.5])
    assert out.tolist() == [[3.0, 4.5], [0.0, 0.0]]
