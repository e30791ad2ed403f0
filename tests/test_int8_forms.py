"""Which form the integer products take: the one that was measured to be the
faster, by a tenth or more for most, on both sides of what the few-rows form is taken for."""

import pytest


@pytest.fixture(scope="module")
def tile():
    from fp8_bf16_mxfp4_gb300 import build, _lib
    build.build()
    return _lib.load().mxg_diag_int8_tile_tokens


FEW = [  # experts, rows, N, K
    (1, 1, 8192, 16384), (1, 8, 4096, 14336), (1, 16, 1024, 16384), (1, 16, 14336, 4096), (1, 16, 4096, 7168), (2, 4, 4096, 14336),
    (2, 24, 2048, 7168), (3, 36, 2048, 2048), (4, 48, 2048, 7168), (8, 48, 4096, 14336), (8, 48, 4096, 7168),
    (32, 128, 4096, 7168), (32, 192, 4096, 14336), (64, 192, 1024, 1024), (22, 96, 96, 2336), (19, 145, 48, 304), (6, 72, 200, 4304),
    (13, 85, 120, 2688)]
NEXT = [
    (1, 1, 8192, 22016), (1, 8, 512, 24576), (1, 12, 4096, 14336), (1, 9, 4096, 11264), (1, 16, 8192, 8192), (1, 16, 28672, 8192),
    (2, 28, 28672, 8192), (2, 14, 4096, 14336), (3, 30, 11008, 2048), (3, 36, 11008, 2048), (3, 36, 4096, 4096), (4, 8, 2048, 22016),
    (8, 56, 4096, 14336), (32, 256, 4096, 14336), (64, 320, 1024, 1024), (128, 768, 768, 2048), (32, 256, 2048, 2048)]


@pytest.mark.parametrize("G,S,N,K", FEW)
def test_few_rows_where_it_is_faster(tile, G, S, N, K):
    assert tile(G, S, N, K) in (8, 16)


@pytest.mark.parametrize("G,S,N,K", NEXT)
def test_tensor_cores_where_they_are(tile, G, S, N, K):
    assert tile(G, S, N, K) >= 32
