"""GPU parity of the serving operators against the 64-bit oracle
(oracle/serve.py), whose error bounds set the tolerances: outputs rounded to
BF16 (FP32) may differ by one rounding, 2^-8 (2^-23) of the value, plus the
bound of the fp32 sums in front of it."""

import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import serve

pytestmark = pytest.mark.gpu

from gpu_util import bf16_to_dev, i32_to_dev, u8_to_dev  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _mxg():
    import fp8_bf16_mxfp4_gb300 as mxg
    return mxg


def f64(t):
    return t.detach().cpu().double().numpy()


# --------------------------------------------------------------------------- routing

# fp32 exp (2 units), a sum of at most 512 terms in any order and one division
ROUTE_RTOL = (512 + 8) * 2.0 ** -24


def check_route(logits, k, renorm, **kw):
    ids, w = _mxg().moe_route(logits, k, renormalize=renorm, **kw)
    want_ids, want_w = serve.route(f64(logits), k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    np.testing.assert_allclose(f64(w), want_w, rtol=ROUTE_RTOL, atol=2.0 ** -126)
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 32, 8), (3, 2, 2), (7, 8, 2), (33, 31, 31), (64, 33, 6), (5, 64, 32),
                                   (130, 65, 8), (9, 128, 8), (17, 161, 6), (50, 256, 8), (11, 257, 3), (8, 512, 32),
                                   (3000, 32, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, dtype, renorm):
    g = torch.Generator().manual_seed(T * 1000 + E)
    check_route((2 * torch.randn(T, E, generator=g)).to(dtype).to(DEV), k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_special_values(renorm):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    rows = [[-inf] * 6, [nan] * 6, [nan, 1, nan, 1, nan, 1], [inf, 0, inf, 0, -inf, 1], [0.0, -0.0, 0.0, -0.0, 0, 0],
            [-inf, -inf, 3, -inf, -inf, -inf], [low] * 6, [low, -inf, low, 0, low, -inf], [-inf, nan, inf, 2, 1, 0],
            [88, 87, -200, 0, 88, 3], [1e-40, -1e-40, 0, 2e-40, 0, 0], [-5, -5, -5, -4, -4, -4]]
    check_route(torch.tensor(rows, device=DEV), 4, renorm)


def test_route_strided_offset_and_given_outputs():
    g = torch.Generator().manual_seed(3)
    big = torch.randn(20, 77, generator=g).to(torch.bfloat16).to(DEV)
    view = big[3:, 5:42]  # odd start, rows longer than the view
    ids = torch.full((17, 5), 99, dtype=torch.int32, device=DEV)
    w = torch.full((17, 5), 9.0, device=DEV)
    got, gw = check_route(view, 5, True, ids=ids, weights=w)
    assert got.data_ptr() == ids.data_ptr() and gw.data_ptr() == w.data_ptr()
    e = _mxg().moe_route(big[:0], 3)
    assert e[0].shape == (0, 3) and e[1].shape == (0, 3)


# --------------------------------------------------------------------------- experts


def expert_weights(rng, rows, cols, fmt, groups):
    """Oracle-quantized weights -> (packed operand on the device, float64 values)."""
    data, scale = oracle.quantize_mx_rowwise(synth.normal_bf16(rng, (rows, cols), std=cols ** -0.5), fmt)
    codes = oracle.unpack_e2m1(data) if fmt == "e2m1" else data
    packed = oracle.pack_scales_mma(scale, [rows // groups] * groups)
    op = _mxg().MXOperand(u8_to_dev(data), u8_to_dev(packed), fmt, cols, "packed")
    return op, oracle.dequantize_mx(codes, scale, fmt)


def choose(rng, T, E, k, how):
    if how == "one":      # every token to expert E-1 (more than one 64-token tile when T > 64)
        ids = np.full((T, k), -1)
        ids[:, k - 1] = E - 1
    elif how == "none":
        ids = np.full((T, k), -1)
    else:
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
        if how == "holes":
            ids[rng.random((T, k)) < 0.5] = -1
            ids[T // 2] = -1
            ids[0] = 0        # a token whose slots name one expert k times
    return ids.astype(np.int32)


def check_experts(T, E, k, H, I, fmt, how="all", out_dtype=torch.bfloat16, std=1.0, seed=0, **kw):
    rng = np.random.default_rng(seed + 17 * T + H + I)
    w13, f13 = expert_weights(rng, E * 2 * I, H, fmt, E)
    w2, f2 = expert_weights(rng, E * H, I, fmt, E)
    bits = synth.normal_bf16(rng, (T, H), std=std, outlier_frac=0.01)
    ids = choose(rng, T, E, k, how)
    wts = rng.random((T, k)).astype(np.float32) - 0.2
    want, bound = serve.moe_experts(bits, ids, wts, f13, f2, E)
    args = (bf16_to_dev(bits), i32_to_dev(ids), torch.from_numpy(wts).to(DEV), w13, w2)
    got = _mxg().moe_experts(*args, out_dtype=out_dtype, check=True, **kw)
    tol = bound + np.abs(want) * (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -23) + 2.0 ** -126
    bad = np.abs(f64(got) - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}"
    return args, got, want


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,E,k,H,I,how", [
    (1, 1, 1, 128, 128, "all"), (1, 4, 2, 256, 128, "all"), (2, 3, 3, 384, 256, "all"), (5, 8, 2, 640, 384, "holes"),
    (15, 4, 2, 256, 256, "all"), (16, 2, 1, 512, 128, "one"), (17, 2, 2, 128, 640, "one"), (33, 6, 3, 384, 128, "holes"),
    (63, 3, 2, 256, 128, "one"), (64, 3, 1, 128, 256, "one"), (65, 2, 2, 384, 128, "one"), (130, 5, 2, 256, 128, "one"),
    (200, 3, 3, 128, 128, "all"), (9, 4, 2, 256, 128, "none"), (40, 16, 8, 256, 128, "all")])
def test_experts(T, E, k, H, I, how, fmt):
    check_experts(T, E, k, H, I, fmt, how)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_experts_fp32_output_and_wide_values(fmt):
    check_experts(6, 4, 2, 384, 256, fmt, out_dtype=torch.float32)
    check_experts(6, 4, 2, 256, 128, fmt, std=2.0 ** 20)
    check_experts(6, 4, 2, 256, 128, fmt, std=2.0 ** -60)


def test_experts_long_contractions():
    check_experts(3, 2, 2, 2048, 1152, "e2m1", seed=5)
    check_experts(20, 2, 1, 1152, 2048, "e4m3", seed=6)


def test_experts_most_slots():
    check_experts(512, 9, 8, 128, 128, "e2m1", seed=7)  # 4096 slots, several 64-token tiles of every expert


def test_experts_strides_streams_and_repeats():
    mxg = _mxg()
    args, got, _ = check_experts(21, 5, 2, 384, 256, "e2m1", seed=9)
    x = args[0]
    wide = torch.zeros(21, 512, dtype=torch.bfloat16, device=DEV)
    wide[:, 64:448] = x
    out = torch.full((21, 400), 7.0, dtype=torch.bfloat16, device=DEV)
    r = mxg.moe_experts(wide[:, 64:448], *args[1:], out=out[:, 8:392], check=True)
    assert torch.equal(r, got) and bool((out[:, :8] == 7).all()) and bool((out[:, 392:] == 7).all())
    assert torch.equal(mxg.moe_experts(*args), got)            # no order of arrival in the result
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = mxg.moe_experts(*args)
    side.synchronize()
    assert torch.equal(other, got)
    ws = torch.full((mxg.moe_experts_workspace_size(21, 2, 5, 384, 256),), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        assert torch.equal(mxg.moe_experts(*args, workspace=ws), got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = mxg.moe_experts(*args)
    args[0].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, mxg.moe_experts(*args, check=True)) and not torch.equal(cap, got)


def test_experts_bad_id_is_reported_and_nothing_written():
    mxg = _mxg()
    args, _, _ = check_experts(4, 3, 2, 256, 128, "e4m3", seed=11)
    ids = args[1].clone()
    ids[2, 1] = 3
    out = torch.full((4, 256), 5.0, dtype=torch.bfloat16, device=DEV)
    mxg.moe_experts(args[0], ids, *args[2:], out=out)
    with pytest.raises(mxg.MXGError) as e:
        mxg.check_status()
    assert e.value.code == 11 and bool((out == 5).all())
    assert torch.isfinite(mxg.moe_experts(*args, check=True)).all()  # the next call is whole again


def test_experts_no_tokens():
    mxg = _mxg()
    args, _, _ = check_experts(2, 2, 1, 128, 128, "e2m1")
    r = mxg.moe_experts(args[0][:0], args[1][:0], args[2][:0], *args[3:], check=True)
    assert r.shape == (0, 128)


def test_experts_same_quantization_as_the_grouped_gemm():
    """The down projection of a single expert equals the dense GEMM path on
    the same operands up to the rounding of its output."""
    mxg = _mxg()
    rng = np.random.default_rng(2)
    H, I, T = 256, 128, 8
    w13, f13 = expert_weights(rng, 2 * I, H, "e2m1", 1)
    w2, f2 = expert_weights(rng, H, I, "e2m1", 1)
    x = bf16_to_dev(synth.normal_bf16(rng, (T, H)))
    gu = mxg.mx_gemm_dense(mxg.mx_quantize_rowwise(x, "e4m3"), w13, out_dtype=torch.float32).double()
    h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    hq, off = serve.mxfp8_f64(f64(h), np.abs(f64(h)) * 2.0 ** -16)
    want = hq @ f2.T
    tol = off @ np.abs(f2.T) + 2.0 ** -8 * np.abs(want) + (I + 8) * serve.U * (np.abs(hq) @ np.abs(f2.T))
    got = mxg.moe_experts(x, torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.ones(T, 1, device=DEV), w13, w2,
                          check=True)
    assert (np.abs(f64(got) - want) <= tol).all()


# --------------------------------------------------------------------------- adapters


def check_lora(T, K, N, R, n, dtype=torch.bfloat16, runs=1, scale=True, seed=0, pad=0, inplace=False):
    g = torch.Generator().manual_seed(seed + T + 7 * K + N)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = rnd(T, K + pad).to(torch.bfloat16).to(DEV)[:, :K]
    y = rnd(T, N + pad).to(dtype).to(DEV)[:, pad:]
    A = (rnd(n, R, K) * K ** -0.5).to(torch.bfloat16).to(DEV)
    B = (rnd(n, N, R) * R ** -0.5).to(torch.bfloat16).to(DEV)
    ids = torch.randint(-(n // 4 + 1), n, (-(-T // runs),), generator=g).clamp(min=-1).repeat_interleave(runs)[:T]
    sc = torch.rand(n, generator=g) + 0.5 if scale else None
    want, bound = serve.lora_add(f64(y), f64(x), f64(A), f64(B), ids.tolist(), sc.tolist() if scale else [1.0] * n)
    y0 = y.clone()
    kw = dict(out=y) if inplace else {}
    got = _mxg().lora_add(y, x, A, B, ids.to(torch.int32).to(DEV), sc.to(DEV) if scale else None, check=True, **kw)
    tol = bound + np.abs(want) * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23) + 2.0 ** -126
    bad = np.abs(f64(got) - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}"
    off = (ids < 0).nonzero().flatten().tolist()
    assert torch.equal(got[off], y0[off])
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,N,R,n,runs", [
    (1, 8, 8, 8, 1, 1), (1, 1024, 512, 16, 3, 1), (2, 136, 40, 24, 2, 1), (15, 512, 256, 8, 40, 1),
    (16, 264, 520, 16, 16, 1), (17, 1000, 1544, 32, 5, 1), (31, 96, 72, 40, 31, 1), (33, 4096, 128, 64, 4, 3),
    (64, 640, 1032, 16, 64, 1), (100, 2056, 264, 128, 7, 9), (257, 328, 88, 56, 3, 1), (600, 512, 1000, 8, 5, 37),
    (1030, 256, 384, 16, 12, 100), (1500, 200, 304, 32, 2, 1)])
def test_lora(T, K, N, R, n, runs, dtype):
    check_lora(T, K, N, R, n, dtype, runs)


# more adapter reads than the per-token form takes on: 128-token tiles
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,N,R,n,runs", [
    (129, 2056, 2064, 128, 70, 1), (130, 4104, 4120, 64, 3, 1), (257, 8200, 520, 16, 40, 1), (300, 2048, 2048, 32, 1, 1),
    (600, 1160, 2056, 72, 9, 5), (1000, 1000, 1544, 24, 5, 37), (2000, 520, 600, 40, 2, 500), (4000, 520, 600, 8, 9, 100),
    (700, 72, 3080, 56, 12, 128), (1200, 3080, 72, 96, 4, 1)])
def test_lora_tiles(T, K, N, R, n, runs, dtype):
    assert T * R * (K + N) * 2 > 64e6
    check_lora(T, K, N, R, n, dtype, runs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lora_tiles_strides_in_place_and_no_scale(dtype):
    check_lora(400, 1032, 1544, 40, 5, dtype, pad=24, runs=3)
    check_lora(400, 1032, 1544, 40, 5, dtype, pad=8, runs=3, inplace=True)
    check_lora(400, 1032, 1544, 40, 5, dtype, runs=90, inplace=True, scale=False)


def test_lora_tiles_select_rows():
    """Infinities and NaN of an adapter, or of a token, stay with its tokens."""
    mxg = _mxg()
    g = torch.Generator().manual_seed(6)
    T, K, N, R, n = 300, 1800, 2000, 32, 5
    to = lambda t: t.to(torch.bfloat16).to(DEV)  # noqa: E731
    x, y = to(torch.randn(T, K, generator=g)), to(torch.randn(T, N, generator=g))
    A, B = to(torch.randn(n, R, K, generator=g) * 0.03), to(torch.randn(n, N, R, generator=g))
    ids = torch.randint(-1, n, (T,), generator=g).to(torch.int32)
    ids[ids == 4] = 1  # adapter 4 is not used
    want = mxg.lora_add(y, x, A, B, ids.to(DEV), check=True)
    assert torch.equal(want[(ids < 0).to(DEV)], y[(ids < 0).to(DEV)])
    A[4], B[4] = float("nan"), float("nan")
    assert torch.equal(mxg.lora_add(y, x, A, B, ids.to(DEV), check=True), want)
    A[2], B[2] = float("inf"), float("nan")
    x[ids == -1] = float("nan")
    hit = int((ids == 3).nonzero()[0])
    x[hit] = float("nan")
    got = mxg.lora_add(y, x, A, B, ids.to(DEV), check=True)
    keep = (ids != 2).to(DEV)
    keep[hit] = False
    assert torch.equal(got[keep], want[keep]) and bool(got[~keep].isnan().all())
    bad = ids.clone()
    bad[150] = n
    mxg.lora_add(y, x, A, B, bad.to(DEV))
    with pytest.raises(mxg.MXGError) as e:
        mxg.check_status()
    assert e.value.code == 11


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lora_strides_in_place_and_no_scale(dtype):
    check_lora(37, 520, 264, 16, 5, dtype, pad=24)
    check_lora(37, 520, 264, 16, 5, dtype, pad=8, inplace=True)
    check_lora(600, 520, 264, 16, 5, dtype, runs=50, inplace=True, scale=False)


def test_lora_cases_without_adapters():
    mxg = _mxg()
    y = torch.randn(40, 64, device=DEV).to(torch.bfloat16)
    x = torch.full((40, 128), float("nan"), dtype=torch.bfloat16, device=DEV)  # not read into rows without an adapter
    A = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    B = torch.zeros(2, 64, 8, dtype=torch.bfloat16, device=DEV)
    ids = torch.full((40,), -1, dtype=torch.int32, device=DEV)
    assert torch.equal(mxg.lora_add(y, x, A, B, ids, check=True), y)
    ids[3] = 1  # that row is NaN, and no other
    r = mxg.lora_add(y, x, A, B, ids, check=True)
    assert bool(r[3].isnan().all())
    keep = [i for i in range(40) if i != 3]
    assert torch.equal(r[keep], y[keep])
    assert mxg.lora_add(y[:0], x[:0], A, B, ids[:0], check=True).shape == (0, 64)


def test_lora_an_unused_adapter_is_not_read_into_others():
    mxg = _mxg()
    g = torch.Generator().manual_seed(4)
    x, y = torch.randn(20, 256, generator=g), torch.randn(20, 72, generator=g)
    A, B = torch.randn(4, 16, 256, generator=g) * 0.1, torch.randn(4, 72, 16, generator=g)
    ids = torch.tensor([0, 1, 2, 1] * 5, dtype=torch.int32)
    to = lambda t: t.to(torch.bfloat16).to(DEV)  # noqa: E731
    a, b = to(A), to(B)
    want = mxg.lora_add(to(y), to(x), a, b, ids.to(DEV), check=True)
    a[3], b[3] = float("nan"), float("inf")
    assert torch.equal(mxg.lora_add(to(y), to(x), a, b, ids.to(DEV), check=True), want)
    a[2], b[2] = float("inf"), float("nan")  # tokens of adapter 2 alone change
    got = mxg.lora_add(to(y), to(x), a, b, ids.to(DEV), check=True)
    keep = (ids != 2).nonzero().flatten().tolist()
    assert torch.equal(got[keep], want[keep]) and bool(got[2::4].isnan().all())


def test_workspaces_kept_by_streams_do_not_meet():
    """Calls of several sizes and operators interleaved on three streams give
    what they give alone."""
    mxg = _mxg()
    cases = []
    for n, (T, H, I) in enumerate(((3, 256, 128), (40, 384, 256), (70, 256, 256))):
        args, got, _ = check_experts(T, 4, 2, H, I, "e2m1" if n % 2 else "e4m3", seed=40 + n)
        g = torch.Generator().manual_seed(n)
        to = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
        lora = (to(T, 520), to(T, H), to(3, 16, H), to(3, 520, 16), torch.arange(T, dtype=torch.int32, device=DEV) % 3)
        cases.append((args, got, lora, mxg.lora_add(*lora, check=True)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for r in range(6):
        for i, s in enumerate(streams):
            args, got, lora, want = cases[(i + r) % 3]
            with torch.cuda.stream(s):
                outs.append((mxg.moe_experts(*args), got))
                outs.append((mxg.lora_add(*lora), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)


def test_calls_of_threads_on_one_stream_do_not_meet():
    """Two threads that enqueue on the same stream do not share a workspace."""
    import threading
    mxg = _mxg()
    bf = torch.bfloat16
    g = torch.Generator().manual_seed(12)
    to = lambda *s: torch.randn(*s, generator=g).to(bf).to(DEV)  # noqa: E731
    sets = [(to(T, 520), to(T, 512), to(3, 16, 512), to(3, 520, 16), torch.arange(T, dtype=torch.int32, device=DEV) % 3)
            for T in (40, 40)]
    wants = [mxg.lora_add(*s, check=True) for s in sets]
    wrong = [0, 0]

    def work(i):
        for _ in range(200):
            wrong[i] += not torch.equal(mxg.lora_add(*sets[i]), wants[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert wrong == [0, 0]
    mxg.check_status()


def test_lora_bad_id_is_reported():
    mxg = _mxg()
    y = torch.zeros(20, 64, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(20, 128, dtype=torch.bfloat16, device=DEV)
    A = torch.ones(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    B = torch.ones(2, 64, 8, dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(20, dtype=torch.int32, device=DEV)
    ids[7] = 2
    r = mxg.lora_add(y, x, A, B, ids)
    with pytest.raises(mxg.MXGError) as e:
        mxg.check_status()
    keep = [i for i in range(20) if i != 7]
    assert e.value.code == 11 and bool((r[keep] == 1024).all())


def test_lora_side_stream_and_graph():
    mxg = _mxg()
    g = torch.Generator().manual_seed(8)
    to = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    y, x, A, B = to(30, 264), to(30, 512), to(6, 16, 512), to(6, 264, 16)
    ids = torch.randint(-1, 6, (30,), generator=g).to(torch.int32).to(DEV)
    want = mxg.lora_add(y, x, A, B, ids, check=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mxg.lora_add(y, x, A, B, ids)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = mxg.lora_add(y, x, A, B, ids)
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, mxg.lora_add(y, x, A, B, ids, check=True)) and not torch.equal(cap, want)


# batches that tiles of sorted tokens take: few tiles with many adapters, K splits, one pass and several
@pytest.mark.parametrize("T,K,N,R,n,runs", [
    (129, 3144, 3200, 128, 300, 1), (250, 2056, 2064, 104, 130, 1), (511, 4104, 2056, 32, 40, 1), (640, 72, 3080, 56, 12, 128),
    (1500, 3080, 72, 96, 4, 1), (2000, 1032, 1544, 40, 2, 500), (4001, 520, 608, 24, 90, 1),
    (8192, 512, 520, 64, 64, 1),    # one segment, every adapter in every 128 tokens of the batch
    (8193, 1032, 264, 128, 3, 1),   # a segment of one token
    (16391, 72, 1032, 64, 200, 5),  # three segments, K inside one 64-element step
    (700, 4104, 8, 128, 9, 1),      # columns inside one block
    (9000, 264, 248, 128, 1, 9000),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lora_mixed_batches(T, K, N, R, n, runs, dtype):
    check_lora(T, K, N, R, n, dtype, runs)


def test_lora_adapters_past_the_sorted_count():
    mxg = _mxg()
    T, K, N, R = 2048, 512, 8, 128
    g = torch.Generator().manual_seed(3)
    to = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    few = (to(5, R, K), to(5, N, R))
    y, x = to(T, N), to(T, K)
    ids = torch.randint(-1, 5, (T,), generator=g).to(torch.int32).to(DEV)
    want = mxg.lora_add(y, x, *few, ids, check=True)
    for n in (8190, 8191, 8192, 8200):  # the same adapters at the end of a long list
        A = torch.zeros(n, R, K, dtype=torch.bfloat16, device=DEV)
        B = torch.zeros(n, N, R, dtype=torch.bfloat16, device=DEV)
        A[-5:], B[-5:] = few
        many = torch.where(ids < 0, ids, ids + n - 5)
        assert torch.equal(mxg.lora_add(y, x, A, B, many, check=True), want)


def test_lora_results_do_not_depend_on_the_place_in_the_batch():
    mxg = _mxg()
    T, K, N, R, n = 1500, 1024, 1544, 96, 40
    g = torch.Generator().manual_seed(4)
    to = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    y, x, A, B = to(T, N), to(T, K), to(n, R, K), to(n, N, R)
    ids = torch.randint(-1, n, (T,), generator=g).to(torch.int32).to(DEV)
    want = mxg.lora_add(y, x, A, B, ids, check=True)
    for _ in range(3):
        perm = torch.randperm(T, generator=g).to(DEV)
        assert torch.equal(mxg.lora_add(y[perm], x[perm], A, B, ids[perm], check=True), want[perm])


# --------------------------------------------------------------------------- bounds and refusals

BAND = 4096


def banded(nbytes):
    """nbytes of 256-byte aligned device memory between sentinel bands."""
    n = (nbytes + 255) // 256 * 256
    buf = torch.full((BAND + n + BAND,), 0xA5, dtype=torch.uint8, device=DEV)
    return buf, buf[BAND: BAND + nbytes]


def bands_hold(buf, nbytes):
    return bool((buf[:BAND] == 0xA5).all()) and bool((buf[BAND + nbytes:] == 0xA5).all())


@pytest.mark.parametrize("T,E,k,H,I,fmt,how", [(1, 2, 2, 256, 128, "e2m1", "all"), (1, 1, 1, 1152, 1152, "e4m3", "all"),
                                               (130, 3, 2, 384, 256, "e2m1", "one"), (33, 12, 3, 640, 384, "e4m3", "holes")])
def test_experts_write_only_their_output_and_workspace(T, E, k, H, I, fmt, how):
    mxg = _mxg()
    args, got, _ = check_experts(T, E, k, H, I, fmt, how)
    need = mxg.moe_experts_workspace_size(T, k, E, H, I)
    wbuf, ws = banded(need)
    obuf, ob = banded(T * H * 2)
    out = ob.view(torch.bfloat16).view(T, H)
    assert torch.equal(mxg.moe_experts(*args, out=out, workspace=ws, check=True), got)
    assert bands_hold(wbuf, need) and bands_hold(obuf, T * H * 2)


@pytest.mark.parametrize("T,K,N,R,n", [(1, 264, 72, 8, 2), (19, 1032, 520, 24, 5), (300, 2048, 2056, 32, 4), (129, 4104, 4120, 72, 9)])
def test_lora_writes_only_its_output_and_workspace(T, K, N, R, n):
    mxg = _mxg()
    g = torch.Generator().manual_seed(T)
    to = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    args = (to(T, N), to(T, K), to(n, R, K), to(n, N, R), (torch.arange(T, device=DEV) % n).to(torch.int32))
    want = mxg.lora_add(*args, check=True)
    need = mxg.lora_add_workspace_size(T, K, R)
    wbuf, ws = banded(need)
    ld = N + 8  # padding between rows
    obuf, ob = banded((T * ld - 8) * 2)
    out = ob.view(torch.bfloat16).as_strided((T, N), (ld, 1))
    assert torch.equal(mxg.lora_add(*args, out=out, workspace=ws, check=True), want)
    assert bands_hold(wbuf, need) and bands_hold(obuf, (T * ld - 8) * 2)
    gaps = ob.view(torch.int16).as_strided((T - 1, 8), (ld, 1), BAND // 2 + N) if T > 1 else None
    assert gaps is None or bool((gaps == 0xA5A5 - 0x10000).all())


def test_route_writes_only_its_outputs():
    mxg = _mxg()
    x = torch.randn(37, 33, device=DEV)
    ids, w = mxg.moe_route(x, 5)
    ibuf, ib = banded(37 * 5 * 4)
    wbuf, wb = banded(37 * 5 * 4)
    mxg.moe_route(x, 5, ids=ib.view(torch.int32).view(37, 5), weights=wb.view(torch.float32).view(37, 5))
    assert torch.equal(ib.view(torch.int32).view(37, 5), ids) and torch.equal(wb.view(torch.float32).view(37, 5), w)
    assert bands_hold(ibuf, 37 * 20) and bands_hold(wbuf, 37 * 20)


def test_binding_refusals():
    mxg = _mxg()
    bf = torch.bfloat16
    z = lambda *s, d=bf: torch.zeros(*s, dtype=d, device=DEV)  # noqa: E731
    i32 = lambda *s: z(*s, d=torch.int32)  # noqa: E731
    f32 = lambda *s: z(*s, d=torch.float32)  # noqa: E731
    for bad in (lambda: mxg.moe_route(f32(4, 16)[:, ::2], 2), lambda: mxg.moe_route(f32(1, 16)[:, ::2], 2),
                lambda: mxg.moe_route(z(4, 8, d=torch.float16), 2), lambda: mxg.moe_route(f32(8), 2),
                lambda: mxg.moe_route(f32(4, 8), 2, ids=i32(4, 3)), lambda: mxg.moe_route(f32(4, 8), 2, weights=z(4, 2))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(mxg.MXGError):
        mxg.moe_route(f32(4, 8), 9)
    w13 = mxg.mx_quantize_rowwise_packed(z(2 * 256, 256), "e2m1", groups=2)
    w2 = mxg.mx_quantize_rowwise_packed(z(2 * 256, 128), "e2m1", groups=2)
    ok = dict(x=z(3, 256), ids=i32(3, 2), weights=f32(3, 2), W13=w13, W2=w2)
    mxg.moe_experts(**ok, check=True)
    plain = mxg.mx_quantize_rowwise(z(2 * 256, 256), "e2m1")
    # the quantizer allocates for every split (2560 bytes); 512 x 128 weights need 512 * 128 / 32 = 2048 of them
    assert w2.scale.numel() == 2560
    mxg.moe_experts(**{**ok, "W2": mxg.MXOperand(w2.data, w2.scale[:-512], "e2m1", 128, "packed")}, check=True)
    short = mxg.MXOperand(w2.data, w2.scale[:-513], "e2m1", 128, "packed")
    for k, v in (("x", z(3, 512)[:, ::2]), ("x", z(1, 512)[:, ::2]), ("x", f32(3, 256)), ("x", z(4, 256)), ("ids", i32(2, 3).t()),
                 ("ids", z(3, 2, d=torch.int64)), ("weights", f32(3, 1)), ("W13", plain), ("W13", w2), ("W2", short),
                 ("out", z(3, 128)), ("out", z(3, 256, d=torch.float16)), ("out", z(3, 512)[:, ::2])):
        with pytest.raises(ValueError):
            mxg.moe_experts(**{**ok, k: v})
    with pytest.raises(mxg.MXGError):
        mxg.moe_experts(**ok, workspace=z(256, d=torch.uint8))
    ok = dict(y=z(3, 64), x=z(3, 128), A=z(2, 8, 128), B=z(2, 64, 8), ids=i32(3), scale=f32(2))
    mxg.lora_add(**ok, check=True)
    for k, v in (("y", z(3, 128)[:, ::2]), ("y", z(3, 64, d=torch.float16)), ("x", z(3, 120)), ("x", f32(3, 128)), ("A", z(2, 128, 8).transpose(1, 2)),
                 ("B", z(2, 64, 16)[:, :, ::2]), ("B", z(3, 64, 8)), ("ids", z(3, d=torch.int64)), ("ids", i32(6)[::2]),
                 ("scale", f32(3)), ("scale", z(2)), ("out", z(3, 64, d=torch.float32))):
        with pytest.raises(ValueError):
            mxg.lora_add(**{**ok, k: v})
    for k, v in (("A", z(2, 12, 128)), ("A", z(2, 136, 128))):  # ranks not a multiple of 8, or past 128
        with pytest.raises(mxg.MXGError):
            mxg.lora_add(**{**ok, "A": v, "B": z(2, 64, v.shape[1])})


def test_example_runs_the_operators_together(capsys):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_moe_block.py")
    spec = importlib.util.spec_from_file_location("serve_moe_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    us = example.main(["--tokens", "5", "--hidden", "512", "--inter", "256", "--experts", "6", "--top-k", "2", "--steps", "3"])
    assert us > 0 and "experts used" in capsys.readouterr().out


# --------------------------------------------------------------------------- offsets past 32 bits


def test_lora_offsets_past_32_bits():
    """More than 2^31 elements of y and 2^32 bytes of x and out, padded rows; sampled rows against the oracle."""
    T, K, N, R, n = 70003, 72, 32776, 64, 3
    ld_x = 33000  # 4.6 GB of rows of which a few columns are used
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.empty(T, ld_x, dtype=torch.bfloat16, device=DEV)[:, :K]
    x.copy_(torch.randn(T, K, generator=g, device=DEV))
    y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    A = (torch.randn(n, R, K, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
    B = (torch.randn(n, N, R, generator=g, device=DEV) * R ** -0.5).to(torch.bfloat16)
    ids = torch.randint(-1, n, (T,), generator=g, device=DEV).to(torch.int32)
    got = _mxg().lora_add(y, x, A, B, ids, check=True)
    rows = [0, 1, 65535, 65536, 69999, 70000, 70001, 70002]
    want, bound = serve.lora_add(f64(y[rows]), f64(x[rows]), f64(A), f64(B), ids[rows].tolist(), [1.0] * n)
    tol = bound + np.abs(want) * 2.0 ** -8 + 2.0 ** -126
    assert (np.abs(f64(got[rows]) - want) <= tol).all()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_experts_offsets_past_32_bits(fmt):
    """The last experts of weights with more than 2^32 (E2M1: 2^31) bytes of
    codes give what the same experts give in a list of their own: the work is
    split by the experts used."""
    mxg = _mxg()
    E, H, I, T, few = 70, 4096, 8192, 5, 3
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    per = 2 if fmt == "e2m1" else 1

    def operand(rows, cols):
        data = torch.zeros(rows, cols // per, dtype=torch.uint8, device=DEV)
        scale = torch.full((cols // 128, rows // 128, 512), 127, dtype=torch.uint8, device=DEV)
        last = rows // E * few
        data[-last:].random_(0, 256, generator=g)
        if fmt == "e4m3":
            data[-last:] &= 0xB7  # no NaN, magnitudes below 2
        scale[:, -(last // 128):].random_(116, 122, generator=g)
        return (mxg.MXOperand(data, scale.view(-1), fmt, cols, "packed"),
                mxg.MXOperand(data[-last:], scale[:, -(last // 128):].contiguous().view(-1), fmt, cols, "packed"))

    w13, w13_few = operand(E * 2 * I, H)
    w2, w2_few = operand(E * H, I)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.tensor([[0, 1], [2, 0], [1, 2], [-1, 2], [1, -1]], dtype=torch.int32, device=DEV)
    w = torch.rand(T, 2, generator=g, device=DEV)
    want = mxg.moe_experts(x, ids, w, w13_few, w2_few, check=True)
    got = mxg.moe_experts(x, torch.where(ids < 0, ids, ids + E - few), w, w13, w2, check=True)
    assert bool(want.isfinite().all()) and float(want.float().abs().max()) > 0
    assert torch.equal(got, want)
