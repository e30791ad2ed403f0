"""Host-side refusals of the dispatch operators and the integer products (no
GPU: fake pointers that are never dereferenced, every call fails before any
CUDA call)."""

import ctypes

import pytest

FAKE = 0x10000
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from fp8_bf16_mxfp4_gb300 import build, _lib
    build.build()
    return _lib.load()


def refuse(fn, args, at, value, code):
    bad = list(args)
    bad[at] = value
    assert fn(*bad) == code, (at, value)


ODD = vp(FAKE + 2)     # not aligned to an element
OFF8 = vp(FAKE + 8)    # not aligned to 16 bytes


def test_sort_refusals(lib):
    f = lib.moe_sort
    need = lib.moe_sort_workspace_size(9000, 2, 32)
    assert need > 256
    #       ids       T     k  E   splits    rows      ws        bytes status    stream
    args = [vp(FAKE), 9000, 2, 32, vp(FAKE), vp(FAKE), vp(FAKE), need, vp(FAKE), None]
    for at, value, code in ((0, None, 1), (4, None, 1), (5, None, 1), (8, None, 1), (1, -1, 2), (2, 0, 2), (2, 33, 2),
                            (1, 2 ** 30, 2), (3, 0, 2), (3, 513, 2), (6, None, 9), (7, need - 1, 9), (0, ODD, 3),
                            (4, ODD, 3), (5, ODD, 3), (6, vp(FAKE + 128), 3)):
        refuse(f, args, at, value, code)
    for bad in ((-1, 2, 32), (4, 0, 32), (4, 33, 32), (4, 2, 0), (4, 2, 513), (2 ** 30, 2, 32)):
        assert lib.moe_sort_workspace_size(*bad) == 0
    assert lib.moe_sort_workspace_size(0, 1, 1) > 0


def test_gather_refusals(lib):
    f = lib.moe_gather
    #       x         ld  rows      T  k  H   dt out       ld  status    stream
    args = [vp(FAKE), 64, vp(FAKE), 4, 2, 64, 1, vp(FAKE), 64, vp(FAKE), None]
    for at, value, code in ((0, None, 1), (2, None, 1), (7, None, 1), (9, None, 1), (1, 56, 2), (1, 68, 3), (8, 56, 2),
                            (8, 68, 3), (5, 60, 2), (5, 0, 2), (6, 0, 5), (6, 3, 5), (3, -1, 2), (4, 0, 2), (4, 33, 2),
                            (0, OFF8, 3), (7, OFF8, 3), (2, ODD, 3)):
        refuse(f, args, at, value, code)
    assert f(None, 64, None, 0, 2, 64, 2, None, 64, vp(FAKE), None) == 0
    refuse(f, [vp(FAKE), 64, vp(FAKE), 4, 2, 60, 2, vp(FAKE), 64, vp(FAKE), None], 5, 62, 2)


def test_combine_refusals(lib):
    f = lib.moe_combine
    #       y         ld  rows of y, rows, weights   T  k  H   dt out       ld  status    stream
    args = [vp(FAKE), 64, 8, vp(FAKE), vp(FAKE), 4, 2, 64, 1, vp(FAKE), 64, vp(FAKE), None]
    for at, value, code in ((0, None, 1), (3, None, 1), (9, None, 1), (11, None, 1), (1, 56, 2), (1, 68, 3), (10, 56, 2),
                            (10, 68, 3), (7, 60, 2), (7, 0, 2), (8, 0, 5), (2, -1, 2), (5, -1, 2), (6, 0, 2), (6, 33, 2),
                            (0, OFF8, 3), (9, OFF8, 3), (3, ODD, 3), (4, ODD, 3)):
        refuse(f, args, at, value, code)
    assert f(None, 64, 0, None, None, 0, 2, 64, 1, None, 64, vp(FAKE), None) == 0


def test_combine_backward_refusals(lib):
    f = lib.moe_combine_backward
    #       dout      ld  y         ld  rows      weights   T  k  H   dt dy               ld  dweights  status    stream
    args = [vp(FAKE), 64, vp(FAKE), 64, vp(FAKE), vp(FAKE), 4, 2, 64, 1, vp(FAKE + 4096), 64, vp(FAKE), vp(FAKE), None]
    for at in (0, 2, 4, 5, 10, 12, 13):
        refuse(f, args, at, None, 1)
    for at, value, code in ((1, 56, 2), (1, 68, 3), (3, 56, 2), (3, 68, 3), (11, 56, 2), (11, 68, 3), (8, 60, 2), (9, 0, 5),
                            (6, -1, 2), (7, 0, 2), (7, 33, 2), (0, OFF8, 3), (2, OFF8, 3), (10, OFF8, 3), (4, ODD, 3),
                            (5, ODD, 3), (12, ODD, 3)):
        refuse(f, args, at, value, code)
    in_place = list(args)
    in_place[10] = vp(FAKE)
    refuse(f, in_place, 11, 72, 2)  # dy is y, but not its rows
    assert f(None, 64, None, 64, None, None, 0, 2, 64, 1, None, 64, None, vp(FAKE), None) == 0


def test_route_backward_refusals(lib):
    f = lib.moe_route_backward
    #       dweights  ids       weights   logits    ld  T  E   k  renorm dt dlogits ld  status    stream
    args = [vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE), 32, 4, 32, 8, 0, 2, vp(FAKE), 32, vp(FAKE), None]
    for at in (0, 1, 2, 3, 10, 12):
        refuse(f, args, at, None, 1)
    for at, value, code in ((4, 31, 2), (5, -1, 2), (6, 0, 2), (6, 513, 2), (6, 7, 2), (7, 0, 2), (7, 33, 2), (9, 0, 5),
                            (11, 31, 2), (0, ODD, 3), (1, ODD, 3), (2, ODD, 3), (3, ODD, 3), (10, ODD, 3)):
        refuse(f, args, at, value, code)
    assert f(None, None, None, None, 0, 0, 32, 8, 1, 1, None, 32, vp(FAKE), None) == 0


def test_int8_quantize_refusals(lib):
    f = lib.int8_quantize_rowwise
    #       x         ld  rows      T  k  cols codes q       ld  scale     status    stream
    args = [vp(FAKE), 64, vp(FAKE), 4, 2, 64, 1, vp(FAKE), 64, vp(FAKE), vp(FAKE), None]
    for at, value, code in ((0, None, 1), (7, None, 1), (9, None, 1), (10, None, 1), (1, 56, 2), (1, 68, 3), (8, 48, 2),
                            (8, 72, 3), (5, 56, 2), (5, 0, 2), (6, 0, 5), (6, 3, 5), (6, 2, 2), (3, -1, 2), (4, 0, 2),
                            (4, 33, 2), (0, OFF8, 3), (7, OFF8, 3), (9, ODD, 3), (2, ODD, 3)):
        refuse(f, args, at, value, code)
    assert f(None, 64, None, 0, 0, 64, 2, None, 128, None, None, None) == 0


def _op(rows, cols, codes=1, data=FAKE, scale=FAKE, ld=None, reserved=0):
    from fp8_bf16_mxfp4_gb300 import _lib
    return _lib.Int8OperandC(data, scale, rows, cols, ld or cols * codes, codes, reserved)


def test_int8_gemm_refusals(lib):
    f, g = lib.int8_grouped_gemm_fwd, lib.int8_gemm_dense
    p = ctypes.byref
    G, S, N, K = 3, 400, 64, 128
    need = lib.int8_gemm_workspace_size(G, S, N, K, 1)
    assert need >= S * K * 2 and 0 < lib.int8_gemm_workspace_size(G, S, N, K, 2) < need
    a, w = _op(S, K), _op(G * N, K)
    #       A     W     splits    G  N  out       ld dt ws        bytes status    stream
    args = [p(a), p(w), vp(FAKE), G, N, vp(FAKE), N, 1, vp(FAKE), need, vp(FAKE), None]
    for at in (0, 1, 2, 5, 10):
        refuse(f, args, at, None, 1)
    for at, value, code in ((3, 0, 2), (3, 513, 2), (3, 2, 2), (4, 60, 2), (4, 0, 2), (6, 56, 2), (6, 68, 3), (7, 0, 5),
                            (8, None, 9), (9, need - 1, 9), (8, vp(FAKE + 128), 3), (5, OFF8, 3), (2, ODD, 3)):
        refuse(f, args, at, value, code)
    for bad, code in ((_op(S, K, codes=3), 5), (_op(S, K, reserved=1), 5), (_op(S, K - 8), 2), (_op(S, K, ld=K - 16), 2),
                      (_op(S, K, ld=K + 8), 3), (_op(S, K, data=None), 1), (_op(S, K, scale=None), 1),
                      (_op(S, K, data=FAKE + 8), 3), (_op(S, K, scale=FAKE + 2), 3), (_op(S, K + 16), 2),
                      (_op(-1, K), 2), (_op(S, 0, ld=16), 2), (_op(S, K, codes=2, ld=K), 2)):
        refuse(f, args, 0, p(bad), code)
    refuse(f, args, 1, p(_op(G * N, K, codes=2)), 5)
    refuse(f, args, 1, p(_op(G * N - 8, K)), 2)
    dense = [p(a), p(_op(N, K)), vp(FAKE), N, 1, vp(FAKE), need, vp(FAKE), None]
    for at, value, code in ((0, None, 1), (1, None, 1), (2, None, 1), (7, None, 1), (3, 56, 2), (4, 5, 5), (5, None, 9)):
        refuse(g, dense, at, value, code)
    refuse(g, dense, 1, p(_op(N - 4, K)), 2)
    for bad in ((0, S, N, K, 1), (513, S, N, K, 1), (G, -1, N, K, 1), (G, S, 4, K, 1), (G, S, N, 8, 1), (G, S, N, K, 3)):
        assert lib.int8_gemm_workspace_size(*bad) == 0


def test_int8_tiles_go_by_the_rows_of_an_expert(lib):
    f = lib.mxg_diag_int8_tile_tokens
    got = {f(G, S, 4096, 4096) for G, S in ((1, 1), (1, 9), (8, 160), (4, 160), (2, 160), (2, 4096))}
    assert got == {8, 16, 32, 64, 128, 256}
    assert f(0, 1, 64, 64) == 0 and f(1, -1, 64, 64) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    import fp8_bf16_mxfp4_gb300 as mxg
    z = torch.zeros
    rows, bf = z(2, 2, dtype=torch.int32), torch.bfloat16
    op = mxg.Int8Operand(z(4, 16, dtype=torch.int8), z(4))
    for call in (lambda: mxg.moe_sort(rows, 4), lambda: mxg.moe_gather(z(2, 8, dtype=bf), rows),
                 lambda: mxg.moe_combine(z(4, 8), rows), lambda: mxg.moe_combine_backward(z(2, 8), z(4, 8), rows, z(2, 2)),
                 lambda: mxg.moe_route_backward(z(2, 2), rows, z(2, 2), z(2, 8)),
                 lambda: mxg.int8_quantize_rowwise(z(2, 16, dtype=bf)), lambda: mxg.int8_gemm_dense(op, op),
                 lambda: mxg.int8_grouped_gemm_fwd(op, op, z(1, dtype=torch.int32), 4)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="unknown codes"):
        mxg.int8_quantize_rowwise(z(2, 16, dtype=bf), codes="e4m3")
