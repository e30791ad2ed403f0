"""lora_add_form: which kernels a call takes, from its sizes (no GPU)."""

import pytest


@pytest.fixture(scope="module")
def lib():
    from fp8_bf16_mxfp4_gb300 import build, _lib
    build.build()
    return _lib.load()


def test_lora_form(lib):
    f = lib.lora_add_form
    assert f(1, 4096, 7168, 16) == 1 and f(8192, 28672, 8192, 32) == 2 and f(0, 8, 8, 8) == 1
    assert f(1, 2 ** 24, 2 ** 24, 128) == 2                    # one token of a huge adapter
    assert f(65535, 8, 8, 8) == 1 and f(65536, 8, 8, 8) == 2   # the per-token grids' limit
    # the adapters' reads, 2 T R (K + N) bytes, of the per-token form: at most 150 MB
    assert 2 * 3125 * 8 * (1000 + 2000) == 150e6
    assert f(3125, 1000, 2000, 8) == 1 and f(3126, 1000, 2000, 8) == 2


def test_lora_form_of_refused_sizes(lib):
    f = lib.lora_add_form
    for bad in ((-1, 64, 64, 8), (65535 * 128 + 1, 64, 64, 8), (4, 60, 64, 8), (4, 0, 64, 8), (4, 64, 60, 8), (4, 64, 0, 8),
                (4, 64, 64, 0), (4, 64, 64, 12), (4, 64, 64, 136), (4, 2 ** 31, 64, 8)):
        assert f(*bad) == 0, bad


@pytest.mark.parametrize("T,n", [(1024, 64), (2000, 30), (8192, 64), (8192, 500), (8193, 64), (16384, 100), (16384, 500),
                                 (65536, 64), (65536, 500), (65536, 512), (65536, 1000), (100000, 700)])
def test_planned_adapters_of_a_tile(lib, T, n):
    """The adapters that a tile meets: tokens on adapters at random, sorted within segments of 8192, cut into tiles of
    128.  The plan has room for one more than the average, and never less than the average."""
    import numpy as np
    ids = np.random.default_rng(T + n).integers(0, n, T)
    met = [len(set(tile)) for s in range(0, T, 8192) for seg in [np.sort(ids[s:s + 8192])]
           for tile in np.split(seg, range(128, len(seg), 128))]
    plan = lib.mxg_diag_lora_tile_adapters(T, n)
    assert np.mean(met) - 0.5 <= plan <= np.mean(met) + 2, (plan, np.mean(met))


def test_planned_adapters_of_no_tile(lib):
    assert lib.mxg_diag_lora_tile_adapters(0, 4) == 0 and lib.mxg_diag_lora_tile_adapters(4, 0) == 0


@pytest.mark.parametrize("R", [8, 64, 128])
@pytest.mark.parametrize("K", [8, 1000, 8192, 65536])
@pytest.mark.parametrize("T", [1, 100, 3000, 8192, 32768, 65535, 65536, 200000])
def test_lora_workspace_is_what_a_form_uses(lib, T, K, R):
    """Partial sums of A x: one per 1024 elements of K where the per-token form may run (for some N), at most 16 in the
    tiles; an order of the tokens beside them."""
    size = lib.lora_add_workspace_size(T, K, R)
    token = -(-K // 1024) if lib.lora_add_form(T, 8, K, R) == 1 else 0
    least, most = max(token, 1), max(token, min(16, max(1, -(-K // 64) // 8)))
    assert least * T * R * 4 + T * 4 <= size <= most * T * R * 4 + T * 4
