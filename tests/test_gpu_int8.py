"""GPU parity of the 8-bit integer quantizer and products: codes and scales
exactly; products exactly where fp32 sums of the codes are (below 2^24), the
scalings in their order, and otherwise within the oracle's bound."""

import numpy as np
import pytest
import torch

from oracle import dispatch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _mxg():
    import fp8_bf16_mxfp4_gb300 as mxg
    return mxg


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def bf16_values(rng, *shape, spread=0):
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(BF)
    if spread:
        x = (x.float() * torch.exp2(torch.from_numpy(rng.integers(-spread, spread, (shape[0], 1))).float())).to(BF)
    return x


# --------------------------------------------------------------------------- quantizer


@pytest.mark.parametrize("codes", ["int8", "f16"])
@pytest.mark.parametrize("T,K", [(1, 16), (3, 48), (7, 256), (33, 1040), (64, 4096), (5, 7168), (2, 20016), (700, 64)])
def test_quantize(T, K, codes):
    rng = np.random.default_rng(T + K)
    x = bf16_values(rng, T, K, spread=60)
    x[T // 2] = 0
    op = _mxg().int8_quantize_rowwise(x.to(DEV), codes=codes, check=True)
    q, s = dispatch.int8_quantize(x.float().numpy())
    assert op.data.dtype == (torch.int8 if codes == "int8" else torch.float16)
    assert np.array_equal(op.data.cpu().float().numpy(), q)
    assert np.array_equal(op.scale.cpu().numpy().view(np.uint32), s.view(np.uint32))


def test_quantize_every_magnitude():
    """Every finite BF16 value against the largest of its row, over the whole range of rows."""
    bits = np.arange(0x7F80, dtype=np.uint16)
    v = torch.from_numpy(bits.view(np.int16)).view(BF)
    rows = []
    for top in (0x0001, 0x0080, 0x0D7F, 0x0D80, 0x3F80, 0x3FFF, 0x4B01, 0x7F7F):
        keep = torch.where(v.float() <= float(v[top]), v, torch.zeros_like(v))
        rows.append(torch.cat([keep, -keep]))
    x = torch.stack(rows)
    op = _mxg().int8_quantize_rowwise(x.to(DEV))
    q, s = dispatch.int8_quantize(x.float().numpy())
    assert np.array_equal(op.data.cpu().numpy(), q) and np.array_equal(op.scale.cpu().numpy(), s)


@pytest.mark.parametrize("codes", ["int8", "f16"])
def test_quantize_rows_that_are_not_finite(codes):
    x = torch.ones(5, 32, dtype=BF)
    x[1, 7], x[2, 31], x[3, 0] = float("inf"), float("nan"), -float("inf")
    op = _mxg().int8_quantize_rowwise(x.to(DEV), codes=codes)
    assert op.scale.isnan().tolist() == [False, True, True, True, False]
    assert (op.data[1:4] == 0).all() and (op.data[[0, 4]] == 127).all()


@pytest.mark.parametrize("codes", ["int8", "f16"])
@pytest.mark.parametrize("T,k,K", [(1, 1, 16), (9, 3, 272), (40, 8, 1024), (3, 32, 9008)])
def test_quantize_in_expert_order(T, k, K, codes):
    mxg = _mxg()
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, 6, (T, k)).astype(np.int32)
    _, rows = mxg.moe_sort(dev(ids), 6)
    x = bf16_values(rng, T, K, spread=8).to(DEV)
    got = mxg.int8_quantize_rowwise(x, rows=rows, codes=codes, check=True)
    want = mxg.int8_quantize_rowwise(mxg.moe_gather(x, rows), codes=codes)
    assert torch.equal(got.data, want.data) and torch.equal(got.scale, want.scale)


def test_quantize_strides_and_bounds_of_writes():
    mxg = _mxg()
    x = torch.randn(6, 120, device=DEV).to(BF)[:, 24:72]
    for codes, dtype in (("int8", torch.int8), ("f16", torch.float16)):
        q = torch.full((8, 96), 3, dtype=dtype, device=DEV)
        s = torch.full((8,), 9.0, device=DEV)
        op = mxg.int8_quantize_rowwise(x, codes=codes, q=q[1:7, 16:64], scale=s[1:7])
        want = mxg.int8_quantize_rowwise(x.contiguous(), codes=codes)
        assert torch.equal(op.data, want.data) and torch.equal(op.scale, want.scale)
        q[1:7, 16:64] = 3
        assert (q == 3).all() and s[0] == 9 and s[7] == 9


# --------------------------------------------------------------------------- product


def operands(rng, splits, N, K, most=127):
    S, G = sum(splits), len(splits)
    qa = rng.integers(-most, most + 1, (S, K)).astype(np.int8)
    qw = rng.integers(-most - 1, most + 1, (G * N, K)).astype(np.int8)
    sa = (rng.random(S) + 0.5).astype(np.float32)
    sw = (rng.random(G * N) + 0.5).astype(np.float32) * np.float32(0.01)
    return qa, sa, qw, sw


def product(qa, sa, qw, sw, splits, N, out_dtype=BF, codes="f16", dense=False, **kw):
    mxg = _mxg()
    a = mxg.Int8Operand(dev(qa, torch.float16 if codes == "f16" else None), dev(sa))
    w = mxg.Int8Operand(dev(qw), dev(sw))
    if dense:
        return mxg.int8_gemm_dense(a, w, out_dtype=out_dtype, check=True, **kw)
    return mxg.int8_grouped_gemm_fwd(a, w, dev(np.array(splits, np.int32)), N, out_dtype=out_dtype, check=True, **kw)


def verify(got, qa, sa, qw, sw, splits, N):
    want, bound = dispatch.int8_gemm(qa, sa, qw, sw, splits)
    if got.dtype == BF:
        bound = bound + np.abs(want) * 2.0 ** -8
    bad = ~(np.abs(got.cpu().double().numpy() - want) <= bound + 2.0 ** -126)
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}"


def in_order(qa, sa, qw, sw, splits, N):
    """fp32(fp32(sum * sw) * sa): what the epilogue computes where the sums are exact."""
    y = np.zeros((len(qa), N), np.float32)
    at = 0
    for g, m in enumerate(splits):
        acc = (qa[at:at + m].astype(np.int64) @ qw[g * N:(g + 1) * N].astype(np.int64).T).astype(np.float32)
        y[at:at + m] = (acc * sw[g * N:(g + 1) * N]) * sa[at:at + m, None]
        at += m
    return y


CASES = [  # splits, N, K
    ([1], 8, 16), ([1], 128, 128), ([3], 136, 144), ([16], 128, 2064), ([0, 1, 0], 40, 48), ([5, 0, 11, 2], 264, 272),
    ([17], 72, 400), ([30, 1, 33], 128, 128), ([64], 520, 1040), ([40, 45], 136, 640), ([65, 3, 100], 256, 256),
    ([128], 128, 512), ([130, 100], 392, 272), ([1, 1, 1, 1, 1, 1, 1, 1], 1096, 1040), ([0, 0, 0], 64, 64),
    ([300], 200, 144), ([256, 256], 256, 256), ([257, 700, 0, 513], 264, 400), ([1000], 136, 1040), ([513], 520, 2000)]


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("splits,N,K", CASES)
def test_product(splits, N, K, out_dtype):
    rng = np.random.default_rng(sum(splits) + N + K)
    ops = operands(rng, splits, N, K)
    got = product(*ops, splits, N, out_dtype)
    verify(got, *ops, splits, N)
    if K <= 1024:  # |sum| <= K 127 128 < 2^24: exact
        want = torch.from_numpy(in_order(*ops, splits, N)).to(out_dtype)
        assert torch.equal(got.cpu(), want)
    assert torch.equal(got, product(*ops, splits, N, out_dtype, codes="int8"))


CUT = [  # splits, N, K, tile: few units, whose contraction is cut
    ([17], 40, 2064, 32), ([33], 264, 8208, 32), ([20, 0, 41], 776, 2064, 32), ([500], 40, 4112, 32), ([1, 280, 19], 264, 4112, 32),
    ([65], 2056, 2064, 64), ([129], 776, 8208, 64), ([90, 200, 3], 776, 4112, 64), ([64, 0, 64, 65, 1], 520, 8208, 64),
    ([1000], 264, 4112, 64), ([129], 2056, 4112, 128), ([300], 2056, 8208, 128), ([150, 350, 0], 776, 4112, 128),
    ([900], 776, 8208, 128), ([1, 127, 600, 172], 520, 8208, 128)]


def test_every_form_is_among_the_cases():
    from fp8_bf16_mxfp4_gb300 import _lib
    f = _lib.load().mxg_diag_int8_tile_tokens
    assert {f(len(s), sum(s), N, K) for s, N, K in CASES if sum(s)} >= {8, 16, 256}
    assert [f(len(s), sum(s), N, K) for s, N, K, _ in CUT] == [tile for *_, tile in CUT]


@pytest.mark.parametrize("splits,N,K,tile", CUT)
def test_cut_forms(splits, N, K, tile):
    """Small codes, whose sums are exact whatever the order: every part of every unit is in the result, once."""
    rng = np.random.default_rng(N + K)
    ops = operands(rng, splits, N, K, most=20)
    want = torch.from_numpy(in_order(*ops, splits, N))
    for codes in ("f16", "int8"):
        assert torch.equal(product(*ops, splits, N, F32, codes=codes).cpu(), want)
    got = product(*ops, splits, N, BF)
    assert torch.equal(got.cpu(), want.to(BF)) and torch.equal(got, product(*ops, splits, N, BF))


@pytest.mark.parametrize("S", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 600])
def test_dense_row_counts(S):
    rng = np.random.default_rng(S)
    ops = operands(rng, [S], 264, 528, most=100)
    got = product(*ops, [S], 264, F32, dense=True)
    assert torch.equal(got.cpu(), torch.from_numpy(in_order(*ops, [S], 264)))
    assert torch.equal(got, product(*ops, [S], 264, F32))


@pytest.mark.parametrize("S,N,K", [(1, 4096, 7168), (3, 1032, 16384), (20, 640, 20000), (50, 384, 9216), (100, 264, 8192), (3, 264, 40000)])
def test_units_cut_over_ctas(S, N, K):
    """Few tiles and a long contraction: every unit is cut and joined; exact sums show every part."""
    rng = np.random.default_rng(S)
    ops = operands(rng, [S], N, K, most=20)
    want = torch.from_numpy(in_order(*ops, [S], N))
    for _ in range(3):
        assert torch.equal(product(*ops, [S], N, F32).cpu(), want)


def test_sums_past_the_exact_range():
    """All codes at their largest: 4112 * 127 * 127 is past 2^24 and the sums round."""
    qa, qw = np.full((20, 4112), 127, np.int8), np.full((136, 4112), 127, np.int8)
    qw[::2] = -128
    sa, sw = np.full(20, 0.5, np.float32), np.full(136, 2.0, np.float32)
    for S in (20,):
        verify(product(qa, sa, qw, sw, [S], 136, F32), qa, sa, qw, sw, [S], 136)
    qa, sa = np.full((700, 4112), -128, np.int8), np.full(700, 0.5, np.float32)
    verify(product(qa, sa, qw, sw, [700], 136, F32), qa, sa, qw, sw, [700], 136)


def test_many_experts():
    rng = np.random.default_rng(5)
    splits = rng.integers(0, 4, 512).tolist()
    ops = operands(rng, splits, 40, 64)
    got = product(*ops, splits, 40, F32)
    assert torch.equal(got.cpu(), torch.from_numpy(in_order(*ops, splits, 40)))


@pytest.mark.parametrize("splits", [[9, 0, 30], [300, 500]])
def test_strides_and_bounds_of_writes(splits):
    mxg = _mxg()
    rng = np.random.default_rng(0)
    N, K, S = 136, 272, sum(splits)
    qa, sa, qw, sw = operands(rng, splits, N, K)
    want = product(qa, sa, qw, sw, splits, N)
    wide_a = torch.full((S, K + 48), 100, dtype=torch.float16, device=DEV)
    wide_w = torch.full((len(splits) * N, K + 32), 100, dtype=torch.int8, device=DEV)
    wide_a[:, 16:16 + K], wide_w[:, 16:16 + K] = dev(qa, torch.float16), dev(qw)
    a, w = mxg.Int8Operand(wide_a[:, 16:16 + K], dev(sa)), mxg.Int8Operand(wide_w[:, 16:16 + K], dev(sw))
    for dtype in (BF, F32):
        big = torch.full((S + 2, N + 24), 9.0, dtype=dtype, device=DEV)
        need = mxg.int8_gemm_workspace_size(len(splits), S, N, K, "f16")
        ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
        got = mxg.int8_grouped_gemm_fwd(a, w, dev(np.array(splits, np.int32)), N, out=big[1:-1, 8:8 + N],
                                        workspace=ws[:need], check=True)
        assert torch.equal(got.to(BF), want) and (ws[need:] == 0x5A).all()
        big[1:-1, 8:8 + N] = 9.0
        assert (big == 9.0).all()


@pytest.mark.parametrize("splits", [[4, -1, 5], [4, 4, 1], [4, 4, 4], [2 ** 31 - 1, 2 ** 31 - 1, 10]])
@pytest.mark.parametrize("S", [8, 1600])
def test_bad_splits_write_nothing(splits, S):
    mxg = _mxg()
    a = mxg.Int8Operand(torch.ones(S, 64, dtype=torch.float16, device=DEV), torch.ones(S, device=DEV))
    w = mxg.Int8Operand(torch.ones(3 * 64, 64, dtype=torch.int8, device=DEV), torch.ones(3 * 64, device=DEV))
    out = torch.full((S, 64), 9.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    mxg.int8_grouped_gemm_fwd(a, w, dev(np.array(splits, np.int32)), 64, out=out, status=st)
    with pytest.raises(mxg.MXGError) as e:
        mxg.check_status(st)
    assert e.value.code == 4 and (out == 9.0).all()


def test_rows_and_channels_that_are_not_finite():
    """A scale of NaN or infinity stays in its row or channel; so does, in tiles of 32 rows and more, an FP16 code that
    is no integer's."""
    mxg = _mxg()
    rng = np.random.default_rng(3)
    for S in (8, 20, 600):
        qa, sa, qw, sw = operands(rng, [S], 136, 256)
        clean = product(qa, sa, qw, sw, [S], 136, F32)
        sa[3], sw[7] = np.nan, np.inf
        got = product(qa, sa, qw, sw, [S], 136, F32)
        keep = torch.ones_like(clean, dtype=torch.bool)
        keep[3], keep[:, 7] = False, False
        assert torch.equal(got[keep], clean[keep]) and got[3].isnan().all() and not got[:, 7].isfinite().any()
        if S == 8:  # codes that are no integers are not for this form
            continue
        a = dev(qa, torch.float16)
        a[5, 100] = float("inf")
        sa[3], sw[7] = 1, 1
        got = mxg.int8_gemm_dense(mxg.Int8Operand(a, dev(sa)), mxg.Int8Operand(dev(qw), dev(sw)), out_dtype=F32)
        keep[5] = False
        assert torch.equal(got[keep], clean[keep]) and not got[5].isfinite().any()


def test_no_rows():
    mxg = _mxg()
    w = mxg.Int8Operand(torch.ones(2 * 64, 64, dtype=torch.int8, device=DEV), torch.ones(2 * 64, device=DEV))
    for dtype in (torch.int8, torch.float16):
        a = mxg.Int8Operand(torch.empty(0, 64, dtype=dtype, device=DEV), torch.empty(0, device=DEV))
        z = torch.zeros(2, dtype=torch.int32, device=DEV)
        assert mxg.int8_grouped_gemm_fwd(a, w, z, 64, check=True).shape == (0, 64)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        mxg.int8_grouped_gemm_fwd(a, w, z + 1, 64, status=st)
        with pytest.raises(mxg.MXGError):
            mxg.check_status(st)


def test_weights_past_32_bits():
    """The last expert's codes lie past 2^32 bytes, its output past 2^31 elements."""
    mxg = _mxg()
    G, N, K = 3, 20480, 73728
    w = torch.randint(-3, 4, (G * N, K), dtype=torch.int8, device=DEV)
    sw = torch.rand(G * N, device=DEV)
    S = 5
    a = torch.randint(-3, 4, (S, K), device=DEV).to(torch.float16)
    out = torch.zeros((S, 1 << 29), device=DEV)[:, :N]
    got = mxg.int8_grouped_gemm_fwd(mxg.Int8Operand(a, torch.ones(S, device=DEV)), mxg.Int8Operand(w, sw),
                                    dev(np.array([1, 0, 4], np.int32)), N, out=out, check=True)
    acc = torch.cat([a[:1].float() @ w[:N].float().t(), a[1:].float() @ w[2 * N:].float().t()])  # integers below 2^24
    assert torch.equal(got, acc * torch.cat([sw[:N].expand(1, N), sw[2 * N:].expand(4, N)]))


def test_quantized_layer_over_experts():
    """Route, sort, quantize in expert order, two products and the way back, against 64 bits from the same codes."""
    mxg = _mxg()
    T, H, I, E, k = 45, 256, 160, 6, 2
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)  # noqa: E731
    x, w1, w2 = r(T, H), r(E * I, H), r(E * H, I)
    ids, wts = mxg.moe_route(r(T, E).float(), k)
    splits, rows = mxg.moe_sort(ids, E)
    q1, q2 = mxg.int8_quantize_rowwise(w1), mxg.int8_quantize_rowwise(w2)
    a = mxg.int8_quantize_rowwise(x, rows=rows, codes="f16")
    h = torch.relu(mxg.int8_grouped_gemm_fwd(a, q1, splits, I))
    b = mxg.int8_quantize_rowwise(h, codes="f16")
    y = mxg.int8_grouped_gemm_fwd(b, q2, splits, H, check=True)
    out = mxg.moe_combine(y, rows, wts, check=True)
    n = lambda t: t.cpu().numpy()  # noqa: E731
    verify(mxg.int8_grouped_gemm_fwd(a, q1, splits, I), n(a.data), n(a.scale), n(q1.data), n(q1.scale), splits.tolist(), I)
    verify(y, n(b.data), n(b.scale), n(q2.data), n(q2.scale), splits.tolist(), H)
    want, bound = dispatch.combine(y.cpu().double().numpy(), n(rows), n(wts).astype(np.float64))
    assert (np.abs(out.cpu().double().numpy() - want) <= bound + np.abs(want) * 2.0 ** -8).all()


@pytest.mark.parametrize("S", [40, 700])
def test_captured_graphs_replay_with_new_inputs(S):
    mxg = _mxg()
    rng = np.random.default_rng(S)
    sets = []
    for _ in range(4):
        qa, sa, qw, sw = operands(rng, [S // 2, S // 2], 264, 1040, most=30)
        sets.append((dev(qa), dev(sa), dev(qw), dev(sw)))
    splits = dev(np.array([S // 2, S // 2], np.int32))

    def call(s):
        return mxg.int8_grouped_gemm_fwd(mxg.Int8Operand(s[0], s[1]), mxg.Int8Operand(s[2], s[3]), splits, 264)

    call(sets[0])
    graphs = []
    for s in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(s)
        graphs.append((g, out))
    want = [call(s).clone() for s in sets[2:]]
    for s, n in zip(sets[:2], sets[2:]):
        for t, u in zip(s, n):
            t.copy_(u)
    for _ in range(3):
        graphs[0][0].replay()
        call(sets[2])
        graphs[1][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for (_, o), w in zip(graphs, want))
    mxg.check_status(device=DEV)


@pytest.mark.parametrize("S", [30, 700])
def test_two_streams_at_once(S):
    mxg = _mxg()
    rng = np.random.default_rng(1)
    data = [operands(rng, [S], 520, 2000, most=20) for _ in range(2)]
    ops = [(mxg.Int8Operand(dev(d[0]), dev(d[1])), mxg.Int8Operand(dev(d[2]), dev(d[3]))) for d in data]
    want = [mxg.int8_gemm_dense(a, w) for a, w in ops]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(mxg.int8_gemm_dense(*ops[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in (0, 1) for g in got[i])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T", [4, 90, 800])  # 2 experts: 4, 90 and 800 rows each
def test_operands_of_the_operations_just_before(T, captured):
    """Calls whose inputs come from a copy, a fill, another stream, or from the call before, right before each of them:
    nothing is read before it is there.  (Kernels of these calls start while the kernel before them ends.)"""
    mxg = _mxg()
    rng = np.random.default_rng(T)
    E, K, N = 2, 1040, 520
    side = torch.cuda.Stream()
    slow = torch.randn(2048, 2048, device=DEV)
    new = []  # an iteration's inputs
    for i in range(4):
        new.append((torch.randn(T, K, device=DEV).bfloat16(), dev(rng.integers(0, E, (T, 2)).astype(np.int32)),
                    torch.randn(E * N, K, device=DEV).bfloat16()))
    x, ids, w = (torch.zeros_like(t) for t in new[0])
    splits = torch.empty(E, dtype=torch.int32, device=DEV)
    rows = torch.empty(T, 2, dtype=torch.int32, device=DEV)
    q, sc = torch.empty(2 * T, K, dtype=torch.float16, device=DEV), torch.empty(2 * T, device=DEV)
    wq, ws = torch.empty(E * N, K, dtype=torch.int8, device=DEV), torch.empty(E * N, device=DEV)
    xs, out = torch.empty(2 * T, K, dtype=torch.bfloat16, device=DEV), torch.empty(2 * T, N, dtype=torch.bfloat16, device=DEV)
    staged = [torch.empty_like(t) for t in (splits, rows)]

    def chain(src):
        here = torch.cuda.current_stream()
        ids.copy_(src[1])
        mxg.moe_sort(ids, E, m_splits=staged[0], rows=staged[1])
        rows.copy_(staged[1])                                  # a copy, then the gather of its rows
        side.wait_stream(here)
        with torch.cuda.stream(side):                          # x from another stream, late
            y = slow
            for _ in range(4):
                y = y @ slow
            x.copy_(src[0])
        mxg.moe_sort(ids, E, m_splits=splits)                  # a kernel that the next one may overtake
        here.wait_stream(side)
        mxg.moe_gather(x, rows, out=xs)
        w.copy_(src[2])
        mxg.int8_quantize_rowwise(x, rows=rows, codes="f16", q=q, scale=sc)
        mxg.int8_quantize_rowwise(w, q=wq, scale=ws)           # weights from the kernel before the product
        mxg.int8_grouped_gemm_fwd(mxg.Int8Operand(q, sc), mxg.Int8Operand(wq, ws), splits, N, out=out)
        first = out.clone()
        out.zero_()
        mxg.moe_sort(ids, E, m_splits=splits)                  # splits from the kernel before
        mxg.int8_grouped_gemm_fwd(mxg.Int8Operand(q, sc), mxg.Int8Operand(wq, ws), splits, N, out=out)
        return first

    want = []
    for s in new:  # every operation by itself
        def alone(f, *a, **k):
            r = f(*a, **k)
            torch.cuda.synchronize()
            return r
        sp, ro = alone(mxg.moe_sort, s[1], E)
        g = alone(mxg.moe_gather, s[0], ro)
        a = alone(mxg.int8_quantize_rowwise, s[0], rows=ro, codes="f16")
        b = alone(mxg.int8_quantize_rowwise, s[2])
        want.append((g, alone(mxg.int8_grouped_gemm_fwd, a, b, sp, N)))
    chain(new[0])
    torch.cuda.synchronize()
    if captured:
        inputs = [torch.empty_like(t) for t in new[0]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            first = chain(inputs)
    for i in (1, 2, 3, 0, 2):
        for t in (splits, *staged, rows, xs, q, out):  # what a call that came too early would find
            t.zero_()
        if captured:
            for d, s in zip(inputs, new[i]):
                d.copy_(s)
            graph.replay()
        else:
            first = chain(new[i])
        torch.cuda.synchronize()
        assert torch.equal(xs, want[i][0]), i
        assert torch.equal(first, want[i][1]) and torch.equal(out, want[i][1]), i


@pytest.mark.parametrize("S,N,K", [(20, 4104, 8208), (3000, 2056, 8208)])
def test_waits_that_run_out(S, N, K):
    """With a limit of 1 ns a call finishes or gives up cleanly; either way the next one is right."""
    mxg = _mxg()
    rng = np.random.default_rng(1)
    lib = mxg._lib.load()
    ops = operands(rng, [S], N, K, most=20)
    want = product(*ops, [S], N)
    before = lib.mxg_get_wait_timeout_ns()
    mxg.set_wait_timeout_ns(1)
    try:
        product(*ops, [S], N)
    except mxg.MXGError as e:
        assert e.code == 8
    finally:
        mxg.set_wait_timeout_ns(before)
    assert torch.equal(product(*ops, [S], N), want)


@pytest.mark.parametrize("bad", ["grad", "codes", "scale", "strided", "weights", "splits", "out", "workspace"])
def test_arguments_that_do_not_fit_are_refused(bad):
    mxg = _mxg()
    z = lambda *s, d=F32: torch.zeros(*s, dtype=d, device=DEV)  # noqa: E731
    op = lambda d, s: mxg.Int8Operand(d, s)  # noqa: E731
    a, w, m = op(z(4, 32, d=torch.int8), z(4)), op(z(16, 32, d=torch.int8), z(16)), z(2, d=torch.int32) + 2
    mxg.int8_grouped_gemm_fwd(a, w, m, 8, check=True)
    kw = {}
    if bad == "grad":
        a = op(a.data, a.scale.clone().requires_grad_())
    elif bad == "codes":
        a = op(z(4, 32, d=torch.uint8), z(4))
    elif bad == "scale":
        a = op(a.data, z(8)[::2])
    elif bad == "strided":
        a = op(z(4, 64, d=torch.int8)[:, ::2], z(4))
    elif bad == "weights":
        w = op(w.data.to(torch.float16), w.scale)
    elif bad == "splits":
        m = m.long()
    elif bad == "out":
        kw["out"] = z(4, 8, d=torch.float16)
    else:
        kw["workspace"] = z(16, d=torch.uint8)
    with pytest.raises((ValueError, mxg.MXGError)):
        mxg.int8_grouped_gemm_fwd(a, w, m, 8, **kw)
