"""Host-side refusals of the serving entry points (no GPU: fake pointers that
are never dereferenced, every call fails before any CUDA call)."""

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


def test_route_refusals(lib):
    f = lib.moe_route
    #       logits    T  E   ld  dt k  renorm ids      weights   stream
    args = [vp(FAKE), 4, 32, 32, 2, 8, 1, vp(FAKE), vp(FAKE), None]
    for at, value, code in ((0, None, 1), (7, None, 1), (8, None, 1), (1, -1, 2), (2, 0, 2), (2, 513, 2), (3, 31, 2),
                            (4, 3, 5), (5, 0, 2), (5, 33, 2), (0, vp(FAKE + 2), 3), (7, vp(FAKE + 2), 3)):
        refuse(f, args, at, value, code)
    refuse(f, [vp(FAKE), 4, 4, 4, 2, 4, 1, vp(FAKE), vp(FAKE), None], 5, 5, 2)  # top_k > experts
    assert f(None, 0, 32, 32, 1, 8, 1, None, None, None) == 0                   # no tokens


def _op(rows, cols, elem, layout=1, data=FAKE, ld=None):
    from fp8_bf16_mxfp4_gb300 import _lib
    return _lib.MxOperandC(data, FAKE, rows, cols, ld or (cols // 2 if elem == 1 else cols), cols // 32, elem, layout)


def test_experts_refusals(lib):
    f = lib.moe_experts
    E, H, I = 4, 256, 128
    need = lib.moe_experts_workspace_size(8, 2, E, H, I)
    assert need > 0
    p = ctypes.byref
    w13, w2 = _op(E * 2 * I, H, 1), _op(E * H, I, 1)
    #       x         T  ld_x ids      weights   k  E  W13     W2     out       ld dt ws        bytes status
    args = [vp(FAKE), 8, H, vp(FAKE), vp(FAKE), 2, E, p(w13), p(w2), vp(FAKE), H, 1, vp(FAKE), need, vp(FAKE), None]
    for at in (0, 3, 4, 7, 8, 9, 14):
        refuse(f, args, at, None, 1)
    for at, value, code in ((1, -1, 2), (1, 2049, 2), (5, 0, 2), (5, 33, 2), (6, 0, 2), (6, 513, 2), (6, 3, 2),
                            (2, H - 8, 2), (2, H + 4, 3), (10, H - 8, 2), (10, H + 4, 3), (11, 0, 5), (12, None, 9),
                            (13, need - 1, 9), (0, vp(FAKE + 8), 3), (9, vp(FAKE + 8), 3), (12, vp(FAKE + 64), 3),
                            (3, vp(FAKE + 1), 3), (4, vp(FAKE + 2), 3)):
        refuse(f, args, at, value, code)
    for bad, code in ((_op(E * 2 * I, H, 1, layout=0), 5), (_op(E * 2 * I, H, 2), 5), (_op(E * 2 * I - 32, H, 1), 2),
                      (_op(E * 2 * I, H, 1, data=FAKE + 16), 3), (_op(E * 2 * I, H, 1, ld=144), 3),
                      (_op(E * 2 * I, H + 32, 1, ld=160), 2), (_op(E * 2 * I, H, 3), 5)):
        refuse(f, args, 7, p(bad), code)
    refuse(f, args, 8, p(_op(E * H, I + 128, 1)), 2)
    assert lib.moe_experts_workspace_size(2049, 2, E, H, I) == 0
    assert lib.moe_experts_workspace_size(8, 2, E, H + 32, I) == 0
    assert f(None, 0, H, None, None, 2, E, p(w13), p(w2), None, H, 1, None, 0, vp(FAKE), None) == 0


def test_lora_refusals(lib):
    f = lib.lora_add
    need = lib.lora_add_workspace_size(8, 256, 16)
    assert need > 0
    #       y        ld_y x        ld_x A         B         ids       scale     T  N   K    R  n dt out       ld  ws
    args = [vp(FAKE), 64, vp(FAKE), 256, vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE), 8, 64, 256, 16, 3, 1, vp(FAKE), 64,
            vp(FAKE), need, vp(FAKE), None]
    for at in (0, 2, 4, 5, 6, 14, 18):
        refuse(f, args, at, None, 1)
    for at, value, code in ((1, 56, 2), (1, 68, 3), (3, 248, 2), (3, 260, 3), (8, -1, 2), (9, 60, 2), (9, 0, 2),
                            (10, 252, 2), (11, 0, 2), (11, 12, 2), (11, 136, 2), (12, 0, 2), (13, 0, 5), (15, 56, 2),
                            (15, 68, 3), (16, None, 9), (17, need - 1, 9), (16, vp(FAKE + 128), 3), (0, vp(FAKE + 8), 3),
                            (2, vp(FAKE + 2), 3), (4, vp(FAKE + 8), 3), (5, vp(FAKE + 8), 3), (14, vp(FAKE + 8), 3),
                            (6, vp(FAKE + 2), 3), (7, vp(FAKE + 2), 3)):
        refuse(f, args, at, value, code)
    assert lib.lora_add_workspace_size(8, 252, 16) == 0 and lib.lora_add_workspace_size(8, 256, 12) == 0
    assert f(None, 64, None, 256, None, None, None, None, 0, 64, 256, 16, 3, 1, None, 64, None, 0, vp(FAKE), None) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    import fp8_bf16_mxfp4_gb300 as mxg
    z = torch.zeros
    with pytest.raises(ValueError):
        mxg.moe_route(z(4, 8), 2)
    op = mxg.MXOperand(z(256, 64, dtype=torch.uint8), z(2048, dtype=torch.uint8), "e2m1", 128, "packed")
    with pytest.raises(ValueError):
        mxg.moe_experts(z(1, 128, dtype=torch.bfloat16), z(1, 1, dtype=torch.int32), z(1, 1), op, op)
    with pytest.raises(ValueError):
        mxg.lora_add(z(1, 8), z(1, 8, dtype=torch.bfloat16), z(1, 8, 8), z(1, 8, 8), z(1, dtype=torch.int32))
