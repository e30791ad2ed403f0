"""Sizes of integer products whose work does not fit 32-bit counts: the call, the
workspace query and the tile diagnostic refuse the same ones (no GPU: fake
pointers, every call fails before any CUDA call)."""

import ctypes

import pytest

FAKE = 0x10000
vp, p = ctypes.c_void_p, ctypes.byref


@pytest.fixture(scope="module")
def lib():
    from fp8_bf16_mxfp4_gb300 import build, _lib
    build.build()
    return _lib.load()


def call(lib, G, S, N, K):
    from fp8_bf16_mxfp4_gb300 import _lib
    a, w = (_lib.Int8OperandC(FAKE, FAKE, rows, K, K * c, c, 0) for rows, c in ((S, 2), (G * N, 1)))
    return lib.int8_grouped_gemm_fwd(p(a), p(w), vp(FAKE), G, N, vp(FAKE), N, 1, vp(FAKE), 0, vp(FAKE), None)


@pytest.mark.parametrize("G,S,N,K", [(1, 2 ** 30, 4096, 2 ** 16), (1, 2 ** 31 - 300, 2 ** 16, 4096), (512, 2 ** 30, 2 ** 21, 2 ** 20),
                                     (4, 40000, 2 ** 28, 2 ** 20)])
def test_sizes_that_do_not_fit_are_refused_everywhere(lib, G, S, N, K):
    assert call(lib, G, S, N, K) == 2
    assert lib.int8_gemm_workspace_size(G, S, N, K, 2) == 0
    assert lib.mxg_diag_int8_tile_tokens(G, S, N, K) == 0


@pytest.mark.parametrize("G,S,N,K", [(1, 32, 33554432, 16), (1, 32, 33554688, 16), (1, 1, 134217728, 16), (3, 2 ** 20, 4096, 4096)])
def test_sizes_that_fit(lib, G, S, N, K):
    need = lib.int8_gemm_workspace_size(G, S, N, K, 2)
    assert need >= 256 and lib.mxg_diag_int8_tile_tokens(G, S, N, K) >= 8
    assert call(lib, G, S, N, K) == 9  # refused for its workspace of no bytes alone
