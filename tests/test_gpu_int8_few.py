"""The few-rows form of the integer products where an expert has more rows than
a tile: staged again within a CTA's run, short last tiles, runs that end in the
middle of a tile.  Small codes, whose sums are exact: every bit is compared."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mxg():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_bf16_mxfp4_gb300 as mxg
    return mxg


CASES = [  # splits, N, K, rows of a tile (0: of the tensor-core forms, 32 and more)
    ([57, 0, 0, 3, 0, 0, 4, 0], 264, 272, 16), ([0] * 31 + [100], 1096, 1040, 16), ([128] + [0] * 31, 520, 272, 16),
    ([33, 0, 1], 2056, 2064, 16), ([0, 0, 36], 8, 16, 16), ([9, 7, 8, 24, 0, 0, 0, 16], 1032, 2064, 16),
    ([1, 17, 0, 30], 1096, 656, 16), ([25, 3], 72, 7168, 16), ([17, 0, 2, 0, 0, 1, 0, 4], 136, 14336, 8),
    ([0, 31, 0, 17, 0, 0, 0, 0], 1032, 9008, 8), ([12], 264, 14336, 8), ([16], 1048, 16384, 8), ([9], 40, 17280, 8),
    ([12], 4096, 14336, 0), ([33, 0, 1], 136, 14336, 8), ([33, 0, 1], 136, 17296, 0), ([5], 136, 17296, 0)]


@pytest.mark.parametrize("splits,N,K,tile", CASES)
def test_experts_of_several_tiles(mxg, splits, N, K, tile):
    S, G = sum(splits), len(splits)
    form = mxg._lib.load().mxg_diag_int8_tile_tokens(G, S, N, K)
    assert form == tile or tile == 0 and form >= 32
    rng = np.random.default_rng(S + N + K)
    qa = rng.integers(-20, 21, (S, K)).astype(np.int8)
    qw = rng.integers(-20, 21, (G * N, K)).astype(np.int8)  # |sums| <= 400 * 17296 < 2^24
    sa = (rng.random(S) + 0.5).astype(np.float32)
    sw = (rng.random(G * N) + 0.5).astype(np.float32)
    want, at = np.zeros((S, N), np.float32), 0
    for g, m in enumerate(splits):
        acc = (qa[at:at + m].astype(np.float64) @ qw[g * N:(g + 1) * N].astype(np.float64).T).astype(np.float32)
        want[at:at + m] = (acc * sw[g * N:(g + 1) * N]) * sa[at:at + m, None]
        at += m
    want = torch.from_numpy(want)
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    w, m = mxg.Int8Operand(t(qw), t(sw)), t(np.array(splits, np.int32))
    for codes in (t(qa), t(qa).to(torch.float16)):
        a = mxg.Int8Operand(codes, t(sa))
        for dtype in (F32, BF):
            out = torch.full((S + 2, N + 8), 9.0, dtype=dtype, device=DEV)
            mxg.int8_grouped_gemm_fwd(a, w, m, N, out=out[1:-1, :N], check=True)
            assert torch.equal(out[1:-1, :N].cpu(), want.to(dtype))
            out[1:-1, :N] = 9.0
            assert (out == 9.0).all()
        if G == 1:
            assert torch.equal(mxg.int8_gemm_dense(a, w, out_dtype=F32, check=True).cpu(), want)
