"""Integer products whose sums pass 2^24, in every form, against 64-bit sums."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def mxg():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_bf16_mxfp4_gb300 as mxg
    return mxg


@pytest.mark.parametrize("kind", ["one sign", "cancelling", "in turn"])
@pytest.mark.parametrize("S,N,K,tile", [(4, 136, 7168, 8), (16, 136, 7168, 16), (20, 136, 7168, 32), (300, 520, 7168, 64),
                                        (2000, 520, 7168, 128), (600, 8200, 7168, 256), (3, 136, 20000, 32), (14, 40, 16384, 8)])
def test_sums_past_the_exact_range(mxg, S, N, K, tile, kind):
    """Codes of 64 to 127: all of one sign, the second half against the first, or signs in turn.  A sum of 16 products
    and what is there keeps 24 bits or more of the largest of them, so each loses less than 2^-23 of the largest partial
    sum, whichever way a form cuts the contraction; at most 80 partial sums are added up at the end, and the scales are 1."""
    assert mxg._lib.load().mxg_diag_int8_tile_tokens(1, S, N, K) == tile
    rng = np.random.default_rng(S + K)
    qa, qw = rng.integers(64, 128, (S, K)).astype(np.int8), rng.integers(64, 128, (N, K)).astype(np.int8)
    if kind == "cancelling":
        qw[:, K // 2:] *= -1
    elif kind == "in turn":
        qw[:, 1::2] *= -1
    a = torch.from_numpy(qa).double()
    w = torch.from_numpy(qw).double()
    want = a @ w.t()                                               # integers below 2^53
    most = torch.maximum(a @ w.clamp(min=0).t(), a @ -w.clamp(max=0).t())  # no partial sum is larger
    assert most.min() > 2 ** 24
    ones = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    for codes in (torch.float16, torch.int8):
        got = mxg.int8_gemm_dense(mxg.Int8Operand(torch.from_numpy(qa).to(DEV).to(codes), ones(S)),
                                  mxg.Int8Operand(torch.from_numpy(qw).to(DEV), ones(N)), out_dtype=torch.float32, check=True)
        off = (got.cpu().double() - want).abs()
        assert (off <= (K / 16 + 80) * 2.0 ** -23 * most).all(), float((off / most).max())
    if kind == "one sign":
        assert (off / want).max() < 2.0 ** -12  # far inside a BF16 result's half step
