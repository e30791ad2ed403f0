"""GPU parity of the operators that bring tokens to the experts and back, and of
their gradients, against the 64-bit oracle (oracle/dispatch.py): integers and
copies exactly, sums within the oracle's bound of fp32 arithmetic plus one
rounding of the result (half a step: 2^-8 of a BF16 value, 2^-24 of an FP32 one)."""

import numpy as np
import pytest
import torch

from oracle import dispatch, serve

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _mxg():
    import fp8_bf16_mxfp4_gb300 as mxg
    return mxg


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def close(got, want, bound, dtype, what=""):
    tol = bound + np.abs(want) * HALF[dtype] + dispatch.TINY
    bad = ~(np.abs(f64(got) - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}"


def choose(rng, T, k, E, how):
    if how == "one":
        return np.full((T, k), E - 1)
    if how == "first":
        return np.zeros((T, k), int)
    if how == "none":
        return np.full((T, k), -1)
    ids = rng.integers(0, E, (T, k))
    if how == "holes":
        ids[rng.random((T, k)) < 0.3] = -1 - rng.integers(0, 5)
        ids[T // 2] = -2 ** 31
    return ids


# --------------------------------------------------------------------------- sort


@pytest.mark.parametrize("T,k,E,how", [
    (1, 1, 1, "all"), (1, 8, 32, "all"), (3, 2, 1, "holes"), (8, 8, 32, "all"), (33, 3, 31, "holes"), (31, 1, 32, "one"),
    (64, 32, 512, "all"), (128, 32, 7, "holes"), (128, 32, 511, "all"), (1, 32, 512, "none"), (100, 2, 3, "first"),
    # more than one chunk of slots: around 1024 slots, 32 chunks and 128 keys, odd tails, chunks of one expert, none
    (1024, 1, 7, "holes"), (1025, 1, 7, "holes"), (683, 3, 126, "holes"), (2048, 8, 127, "all"), (2048, 8, 128, "all"),
    (16384, 1, 16, "holes"), (16385, 1, 16, "holes"), (16385, 1, 127, "all"), (131073, 1, 3, "holes"), (4097, 1, 5, "all"), (1366, 3, 512, "holes"), (2500, 2, 33, "one"), (3000, 3, 64, "none"), (5001, 7, 161, "holes"),
    (20000, 8, 32, "all"), (75000, 8, 512, "holes")])
def test_sort(T, k, E, how):
    rng = np.random.default_rng(T + k + E)
    ids = choose(rng, T, k, E, how)
    splits, rows = _mxg().moe_sort(i32(ids), E, check=True)
    if T * k <= 50000:
        want_s, want_r = dispatch.sort(ids, E)
    else:  # the same by a stable argsort
        key = np.where(ids.reshape(-1) < 0, E, ids.reshape(-1))
        want_r = np.empty(T * k, np.int64)
        want_r[np.argsort(key, kind="stable")] = np.arange(T * k)
        want_r = np.where(key == E, -1 - want_r, want_r).reshape(T, k)
        want_s = np.bincount(key, minlength=E + 1)
        want_s[E - 1] += want_s[E]
        want_s = want_s[:E]
    assert np.array_equal(splits.cpu().numpy(), want_s)
    assert np.array_equal(rows.cpu().numpy(), want_r)


def test_sort_of_no_tokens():
    splits, rows = _mxg().moe_sort(torch.empty(0, 4, dtype=torch.int32, device=DEV), 6, check=True)
    assert splits.tolist() == [0] * 6 and rows.shape == (0, 4)


@pytest.mark.parametrize("T", [40, 4000])
def test_sort_reports_ids_past_the_experts(T):
    mxg = _mxg()
    rng = np.random.default_rng(2)
    ids = rng.integers(-1, 9, (T, 3))
    ids[T // 2, 1] = 12
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    splits, rows = mxg.moe_sort(i32(ids), 9, status=st)
    with pytest.raises(mxg.MXGError) as e:
        mxg.check_status(st)
    assert e.value.code == 11
    want_s, want_r = dispatch.sort(ids, 9)  # its slot is empty
    assert np.array_equal(splits.cpu().numpy(), want_s) and np.array_equal(rows.cpu().numpy(), want_r)


def test_sort_into_given_outputs():
    mxg = _mxg()
    ids = i32(choose(np.random.default_rng(0), 5000, 2, 12, "holes"))
    need = mxg.moe_sort_workspace_size(5000, 2, 12)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    splits = torch.full((12,), -7, dtype=torch.int32, device=DEV)
    rows = torch.full((5000, 2), -7, dtype=torch.int32, device=DEV)
    s, r = mxg.moe_sort(ids, 12, m_splits=splits, rows=rows, workspace=ws[:need], check=True)
    assert s is splits and r is rows and (ws[need:] == 0x5A).all()
    s2, r2 = mxg.moe_sort(ids, 12, check=True)
    assert torch.equal(s, s2) and torch.equal(r, r2)


# --------------------------------------------------------------------------- gather and combine

SIZES = [(700, 1, 5, 24, "holes"), (90, 2, 4, 1032, "holes"), (1300, 4, 9, 264, "holes"), (40, 3, 4, 520, "all"),
         (650, 2, 3, 2048, "holes"), (1, 1, 1, 8, "all"), (1, 8, 32, 64, "all"), (2, 3, 4, 256, "none"), (7, 2, 3, 40, "holes"), (33, 6, 5, 1160, "holes"),
         (16, 32, 64, 104, "holes"), (129, 9, 16, 2056, "all"), (300, 1, 7, 16, "holes"), (5, 8, 9, 7168, "holes"),
         (3, 17, 8, 20000, "all")]


def made(T, k, E, H, how, dtype, seed=0):
    rng = np.random.default_rng(seed + T * 31 + H)
    ids = choose(rng, T, k, E, how)
    _, rows = dispatch.sort(ids, E)
    g = torch.Generator().manual_seed(seed + T)
    rand = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)  # noqa: E731
    w = torch.from_numpy((rng.random((T, k)) - 0.3).astype(np.float32)).to(DEV)
    return rows, rand, w


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,E,H,how", SIZES)
def test_gather(T, k, E, H, how, dtype):
    rows, rand, _ = made(T, k, E, H, how, dtype)
    x = rand(T, H)
    got = _mxg().moe_gather(x, i32(rows), check=True)
    assert got.dtype == dtype and np.array_equal(f64(got), dispatch.gather(f64(x), rows))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,H,how", SIZES)
def test_combine(T, k, E, H, how, weighted, dtype):
    rows, rand, w = made(T, k, E, H, how, dtype)
    y = rand(T * k, H)
    got = _mxg().moe_combine(y, i32(rows), w if weighted else None, check=True)
    want, bound = dispatch.combine(f64(y), rows, f64(w) if weighted else None)
    assert got.dtype == dtype
    close(got, want, bound, dtype)
    assert torch.equal(got, _mxg().moe_combine(y, i32(rows), w if weighted else None))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,k,E,H,how", SIZES)
def test_combine_backward(T, k, E, H, how, in_place, dtype):
    rows, rand, w = made(T, k, E, H, how, dtype)
    y, dout = rand(T * k, H), rand(T, H)
    want_dy, want_dw, bound = dispatch.combine_backward(f64(dout), f64(y), rows, f64(w))
    dy, dw = _mxg().moe_combine_backward(dout, y, i32(rows), w, dy=y if in_place else None, check=True)
    # a BF16 product is rounded to FP32 first
    close(dy, want_dy, np.abs(want_dy) * 2.0 ** -23, dtype, "dy")
    close(dw, want_dw, bound, F32, "dweights")


def test_gather_and_combine_round_trip():
    """Copies there and back with weights that sum to 1 in powers of two give x."""
    mxg = _mxg()
    x = torch.randn(50, 96, device=DEV).to(BF)
    ids = i32(choose(np.random.default_rng(4), 50, 4, 6, "all"))
    _, rows = mxg.moe_sort(ids, 6)
    w = torch.full((50, 4), 0.25, device=DEV)
    assert torch.equal(mxg.moe_combine(mxg.moe_gather(x, rows), rows, w, check=True), x)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_bounds_of_writes(dtype):
    """Rows of wider tensors, at odd 16-byte offsets; nothing beside them changes."""
    mxg = _mxg()
    rows_h, rand, w = made(21, 3, 5, 72, "holes", dtype)
    rows, P = i32(rows_h), 63
    frame = lambda n: torch.full((n + 2, 104), 9.0, dtype=dtype, device=DEV)  # noqa: E731
    x, y, dout = rand(21, 88)[:, 8:80], rand(P, 96)[:, 16:88], rand(21, 80)[:, :72]
    for call, n, args in ((mxg.moe_gather, P, (x, rows)), (mxg.moe_combine, 21, (y, rows, w))):
        big = frame(n)
        got = call(*args, out=big[1:-1, 16:88], check=True)
        assert torch.equal(got, call(*(a.contiguous() for a in args)))
        big[1:-1, 16:88] = 9.0
        assert (big == 9.0).all()
    big = frame(P)
    dw = torch.full((23, 3), 9.0, device=DEV)
    got, gw = mxg.moe_combine_backward(dout, y, rows, w, dy=big[1:-1, 16:88], dweights=dw[1:-1], check=True)
    want, ww = mxg.moe_combine_backward(dout.contiguous(), y.contiguous(), rows, w)
    assert torch.equal(got, want) and torch.equal(gw, ww)
    big[1:-1, 16:88] = 9.0
    assert (big == 9.0).all() and (dw[0] == 9.0).all() and (dw[-1] == 9.0).all()


def test_what_lies_in_empty_slots_does_not_matter():
    mxg = _mxg()
    nan, inf = float("nan"), float("inf")
    rows_h, rand, w = made(12, 4, 3, 64, "holes", F32)
    rows = i32(rows_h)
    y, dout = rand(48, 64), rand(12, 64)
    tail = torch.tensor([dispatch.place(e) for e in rows_h.flat if e < 0], device=DEV)
    base = mxg.moe_combine(y, rows, w), *mxg.moe_combine_backward(dout, y, rows, w)
    y2, w2 = y.clone(), w.clone()
    y2[tail] = nan
    w2[rows < 0] = inf
    assert torch.equal(mxg.moe_combine(y2, rows, w2, check=True), base[0])
    dy, dw = mxg.moe_combine_backward(dout, y2, rows, w2, check=True)
    assert torch.equal(dy, base[1]) and torch.equal(dw, base[2])
    assert (dy[tail] == 0).all() and (dw[rows < 0] == 0).all()


def test_infinities_and_nan_stay_in_their_rows():
    mxg = _mxg()
    nan, inf = float("nan"), float("inf")
    rows = i32([[0, 2], [1, 3]])
    y = torch.ones(4, 8, device=DEV)
    y[0, 0], y[1, 1], y[3, 2] = inf, nan, -inf
    w = torch.tensor([[0.5, 0.0], [1.0, 2.0]], device=DEV)
    out = mxg.moe_combine(y, rows, w, check=True).cpu()
    assert out[0, 0] == inf and out[0, 1:].tolist() == [0.5] * 7
    assert out[1, 1].isnan() and out[1, 2] == -inf and out[1, 0] == 3.0
    w[0, 0] = 0.0  # 0 times an infinity
    assert mxg.moe_combine(y, rows, w).cpu()[0, 0].isnan()


@pytest.mark.parametrize("bad", [8, 2 ** 31 - 1, -9, -2 ** 31])
def test_rows_past_the_matrix_are_reported(bad):
    """rows that are not from moe_sort: the slot is left out and nothing is read or written past the matrix."""
    mxg = _mxg()
    rows = i32([[0, 1], [2, bad], [4, 5], [6, 7]])
    x, w = torch.randn(4, 32, device=DEV), torch.rand(4, 2, device=DEV)
    y = torch.randn(8, 32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)

    def reported():
        with pytest.raises(mxg.MXGError) as e:
            mxg.check_status(st)
        return e.value.code == 11

    out = torch.full((10, 32), 9.0, device=DEV)
    mxg.moe_gather(x, rows, out=out[1:9], status=st)
    assert reported() and (out[[0, 4, 9]] == 9.0).all() and torch.equal(out[1:3], x[[0, 0]])
    if bad >= 0:  # an empty slot's row is not read
        c = mxg.moe_combine(y, rows, w, status=st)
        assert reported() and torch.equal(c[1], mxg.moe_combine(y, i32([[0, 1], [2, -9], [4, 5], [6, 7]]), w)[1])
    dy = torch.full((10, 32), 9.0, device=DEV)
    _, dw = mxg.moe_combine_backward(x, y, rows, w, dy=dy[1:9], status=st)
    assert reported() and (dy[[0, 4, 9]] == 9.0).all() and dw[1, 1] == 0
    q = torch.full((8, 32), 7, dtype=torch.int8, device=DEV)
    mxg.int8_quantize_rowwise(x.to(BF), rows=rows, q=q, status=st)
    assert reported() and (q[3] == 7).all()


def test_no_tokens():
    mxg = _mxg()
    rows = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    e = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    assert mxg.moe_gather(e(0, 8), rows, check=True).shape == (0, 8)
    assert mxg.moe_combine(e(0, 8), rows, e(0, 3), check=True).shape == (0, 8)
    dy, dw = mxg.moe_combine_backward(e(0, 8), e(0, 8), rows, e(0, 3), check=True)
    assert dy.shape == (0, 8) and dw.shape == (0, 3)


def test_combine_of_a_matrix_with_more_rows():
    """rows may name rows of any matrix that has them (a buffer of a larger capacity)."""
    mxg = _mxg()
    rows = np.array([[9, 0], [3, 7]])
    y = torch.randn(12, 16, device=DEV)
    close(mxg.moe_combine(y, i32(rows), check=True), *dispatch.combine(f64(y), rows, None), F32)


# --------------------------------------------------------------------------- gradient of the routing


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 32, 8), (3, 2, 2), (33, 31, 31), (64, 33, 6), (5, 64, 32), (130, 65, 8),
                                   (17, 161, 6), (50, 256, 8), (8, 512, 32), (3000, 32, 4)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward(T, E, k, dtype, renorm):
    mxg = _mxg()
    g = torch.Generator().manual_seed(T + E)
    logits = (2 * torch.randn(T, E, generator=g)).to(dtype).to(DEV)
    logits[torch.rand(T, E, generator=g).to(DEV) < 0.2] = -float("inf")
    if T > 2:
        logits[T // 2] = -float("inf")
        logits[0, 0] = float("nan")
    d = torch.randn(T, k, generator=g).to(DEV)
    ids, w = mxg.moe_route(logits, k, renormalize=renorm)
    got = mxg.moe_route_backward(d, ids, w, logits, renormalize=renorm, check=True)
    assert got.dtype == dtype
    want, bound = dispatch.route_backward(f64(d), ids.cpu().numpy(), f64(w), f64(logits), E, renorm)
    close(got, want, bound, dtype)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(renorm):
    """The gradient of a loss of moe_route's weights, by steps of the logits (FP32 weights: the difference of two
    losses of size 3 is off by 2^-20 or so over a step of 2^-6, the third derivative adds 2^-12)."""
    mxg = _mxg()
    logits = torch.tensor([[0.5, -1, 2, 1, 0, -0.25], [1, 1.5, -2, 0, 0.25, 3]], device=DEV)
    d = torch.tensor([[1.0, -2, 0.5], [0.25, 3, -1]], device=DEV)
    ids, w = mxg.moe_route(logits, 3, renormalize=renorm)
    got = mxg.moe_route_backward(d, ids, w, logits, renormalize=renorm)
    h = 2.0 ** -6
    for e in np.ndindex(2, 6):
        step = torch.zeros_like(logits)
        step[e] = h
        loss = [float((mxg.moe_route(logits + s * step, 3, renormalize=renorm)[1].double() * d).sum()) for s in (1, -1)]
        assert abs((loss[0] - loss[1]) / (2 * h) - float(got[e])) < 2.0 ** -9


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E", [128, 256, 264, 512])
def test_route_backward_of_rows_at_any_offset(E, dtype):
    """Rows that 16-byte pieces fit, and the same values in rows that they do not."""
    mxg = _mxg()
    g = torch.Generator().manual_seed(E)
    logits = (2 * torch.randn(19, E, generator=g)).to(dtype).to(DEV)
    ids, w = mxg.moe_route(logits, 8, renormalize=False)
    d = torch.randn(19, 8, generator=g).to(DEV)
    want = mxg.moe_route_backward(d, ids, w, logits, renormalize=False, check=True)
    oracle, bound = dispatch.route_backward(f64(d), ids.cpu().numpy(), f64(w), f64(logits), E, False)
    close(want, oracle, bound, dtype)
    for at, room in ((1, 3), (16, 32), (4, 12)):
        big, out = torch.zeros(19, E + room, dtype=dtype, device=DEV), torch.full((19, E + room), 9.0, dtype=dtype, device=DEV)
        big[:, at:at + E] = logits
        for dst in (None, out[:, at:at + E]):
            got = mxg.moe_route_backward(d, ids, w, big[:, at:at + E], renormalize=False, dlogits=dst, check=True)
            close(got, oracle, bound, dtype)
        out[:, at:at + E] = 9.0
        assert (out == 9.0).all()


@pytest.mark.parametrize("E,k", [(7, 5), (40, 32), (100, 3), (256, 32), (500, 17)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_of_experts_named_several_times(E, k, renorm):
    mxg = _mxg()
    g = torch.Generator().manual_seed(E + k)
    logits = (2 * torch.randn(41, E, generator=g)).to(DEV)
    ids = torch.randint(-1, E, (41, k), generator=g, dtype=torch.int32).to(DEV)
    ids[3] = E - 1
    w, d = torch.rand(41, k, generator=g).to(DEV), torch.randn(41, k, generator=g).to(DEV)
    got = mxg.moe_route_backward(d, ids, w, logits, renormalize=renorm, check=True)
    want, bound = dispatch.route_backward(f64(d), ids.cpu().numpy(), f64(w), f64(logits), E, renorm)
    close(got, want, bound, F32)
    for _ in range(3):  # adds in the order of the slots
        assert torch.equal(got, mxg.moe_route_backward(d, ids, w, logits, renormalize=renorm))


def test_route_backward_special_cases():
    mxg = _mxg()
    nan, inf = float("nan"), float("inf")
    ids = i32([[2, 2, 0], [-1, -1, -1], [1, -1, 5]])  # one expert twice; no slots; an empty slot among others
    w = torch.tensor([[0.5, 0.25, 0.25], [nan, inf, 1], [1.0, nan, 0.5]], device=DEV)
    d = torch.tensor([[1.0, 2, 3], [nan, inf, nan], [2.0, inf, -1]], device=DEV)
    logits = torch.zeros(3, 6, device=DEV)
    logits[1] = -inf
    logits[2, 3:] = torch.tensor([inf, -inf, inf], device=DEV)  # p: a half each
    for renorm in (True, False):
        got = mxg.moe_route_backward(d, ids, w, logits, renormalize=renorm, check=True)
        want, bound = dispatch.route_backward(f64(d), ids.cpu().numpy(), f64(w), f64(logits), 6, renorm)
        close(got, want, bound, F32)
        assert (got[1] == 0).all()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids[0, 0] = 6
    out = torch.full((5, 8), 9.0, device=DEV)
    got = mxg.moe_route_backward(d, ids, w, logits, dlogits=out[1:4, 1:7], status=st)
    with pytest.raises(mxg.MXGError):
        mxg.check_status(st)
    close(got, *dispatch.route_backward(f64(d), ids.cpu().numpy(), f64(w), f64(logits), 6, True), F32)
    out[1:4, 1:7] = 9.0
    assert (out == 9.0).all()


# --------------------------------------------------------------------------- as they are used


def layer(mxg, x, router, k, w13, w2, E, I, dout):
    """A mixture-of-experts layer in BF16 products of torch, with the library's dispatch: output and gradients."""
    logits = x @ router.t()
    ids, w = mxg.moe_route(logits, k)
    splits, rows = mxg.moe_sort(ids, E)
    xs = mxg.moe_gather(x, rows)
    ends = torch.cumsum(splits, 0).tolist()
    spans = [(e, ends[e - 1] if e else 0, ends[e]) for e in range(E)]
    y = torch.empty(x.shape[0] * k, x.shape[1], dtype=x.dtype, device=DEV)
    for e, a, b in spans:
        y[a:b] = torch.tanh(xs[a:b] @ w13[e].t()) @ w2[e].t()
    out = mxg.moe_combine(y, rows, w)
    dy, dw = mxg.moe_combine_backward(dout, y, rows, w)
    dxs = torch.empty_like(xs)
    for e, a, b in spans:
        h = torch.tanh(xs[a:b] @ w13[e].t())
        dxs[a:b] = (dy[a:b] @ w2[e] * (1 - h * h)) @ w13[e]
    dx = mxg.moe_combine(dxs, rows) + mxg.moe_route_backward(dw, ids, w, logits) @ router
    return out, dx


def test_a_layer_forward_and_backward():
    """The operators together against autograd through plain indexing, in FP32."""
    mxg = _mxg()
    T, H, I, E, k = 60, 48, 40, 5, 2
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    x, router, w13, w2, dout = r(T, H), r(E, H) * 0.2, r(E, I, H) * 0.15, r(E, H, I) * 0.15, r(T, H)
    out, dx = layer(mxg, x, router, k, w13, w2, E, I, dout)
    xd = x.double().requires_grad_()
    v, i = torch.topk(xd @ router.double().t(), k)
    p = torch.softmax(v, -1)
    full = torch.einsum("teh,td->tedh", torch.ones(T, E, 1, device=DEV).double(), xd).squeeze(-1)
    per = torch.stack([torch.tanh(full[:, e] @ w13[e].double().t()) @ w2[e].double().t() for e in range(E)], 1)
    want = (torch.gather(per, 1, i.unsqueeze(-1).expand(-1, -1, H)) * p.unsqueeze(-1)).sum(1)
    want.backward(dout.double())
    # FP32 through three products of up to 48 terms and a few more operations: 2^-24 * ~200 of the largest values
    assert (out - want).abs().max() <= 2.0 ** -16 * want.abs().max()
    assert (dx - xd.grad).abs().max() <= 2.0 ** -16 * xd.grad.abs().max()


def test_rows_of_an_mx_layer():
    """The splits are those the quantizers and grouped GEMMs check: with empty slots, their rows are zeros."""
    mxg = _mxg()
    T, k, E, K, N = 70, 3, 4, 256, 128
    ids = i32(choose(np.random.default_rng(1), T, k, E, "holes"))
    x = torch.randn(T, K, device=DEV).to(BF)
    splits, rows = mxg.moe_sort(ids, E)
    xs = mxg.moe_gather(x, rows)
    a = mxg.mx_quantize_rowwise_packed(xs, "e4m3", m_splits=splits, check=True)
    w = mxg.mx_quantize_rowwise_packed(torch.randn(E * N, K, device=DEV).to(BF), "e4m3", groups=E)
    y = mxg.grouped_gemm_fwd(a, w, splits, N, check=True)
    tail = torch.tensor([dispatch.place(e) for e in rows.cpu().numpy().flat if e < 0], device=DEV)
    assert len(tail) and (y[tail] == 0).all()
    out = mxg.moe_combine(y, rows, torch.rand(T, k, device=DEV), check=True)
    assert out.isfinite().all() and (out[T // 2] == 0).all()


def step(mxg, s):
    splits, rows = mxg.moe_sort(s["ids"], 12)
    xs = mxg.moe_gather(s["x"], rows)
    out = mxg.moe_combine(xs, rows, s["w"])
    dy, dw = mxg.moe_combine_backward(s["x"], xs, rows, s["w"])
    return splits, rows, xs, out, dy, dw, mxg.moe_route_backward(dw, s["ids"], s["w"], s["logits"], renormalize=False)


def inputs(seed, T=3000, k=2):
    g = torch.Generator().manual_seed(seed)
    return dict(ids=i32(choose(np.random.default_rng(seed), T, k, 12, "holes")), w=torch.rand(T, k, generator=g).to(DEV),
                x=torch.randn(T, 128, generator=g).to(BF).to(DEV), logits=torch.randn(T, 12, generator=g).to(DEV))


def test_captured_graphs_replay_with_new_inputs():
    """Two graphs of the same calls and an eager call between: none sees another's workspace."""
    mxg = _mxg()
    a, b = inputs(1), inputs(2)
    step(mxg, a)
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(mxg, s)
        graphs.append((g, out))
    c, d = inputs(3), inputs(4)
    want = [step(mxg, c), step(mxg, d)]
    for s, n in ((a, c), (b, d)):
        for name in s:
            s[name].copy_(n[name])
    graphs[0][0].replay()
    step(mxg, c)
    graphs[1][0].replay()
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for (_, got), w in zip(graphs, want):
        assert all(torch.equal(x, y) for x, y in zip(got, w))
    mxg.check_status(device=DEV)


def test_two_streams_at_once():
    mxg = _mxg()
    data = [inputs(5), inputs(6)]
    want = [step(mxg, s) for s in data]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = step(mxg, data[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31 elements of their matrix (BF16: 2^32 bytes)."""
    mxg = _mxg()
    H = 1 << 20
    P = 2 * 1040
    ids = i32(np.arange(P).reshape(1040, 2)[::-1] % 3)
    splits, rows = mxg.moe_sort(ids, 3)
    x = torch.randn(1040, H, device=DEV, dtype=BF)
    xs = mxg.moe_gather(x, rows, check=True)
    last = int(rows.max())
    assert last == P - 1
    t, j = divmod(int((rows.reshape(-1) == last).nonzero()), 2)
    assert torch.equal(xs[last], x[t]) and torch.equal(xs[0], x[int((rows.reshape(-1) == 0).nonzero()) // 2])
    w = torch.full((1040, 2), 0.5, device=DEV)
    assert torch.equal(mxg.moe_combine(xs, rows, w, check=True), x)
    dy, dw = mxg.moe_combine_backward(x, xs, rows, w, dy=xs, check=True)
    assert torch.equal(dy[last], x[t] * 0.5)


# --------------------------------------------------------------------------- autograd and given memory


def calls():
    """name -> (function, arguments, those that can require grad, those that are written)"""
    mxg = _mxg()
    rows = i32([[0, 2], [1, 3]])
    z = lambda *s, d=F32: torch.zeros(*s, dtype=d, device=DEV)  # noqa: E731
    return {
        "moe_sort": (mxg.moe_sort, dict(ids=z(2, 2, d=torch.int32), experts=2, m_splits=z(2, d=torch.int32),
                                        rows=z(2, 2, d=torch.int32)), (), ("m_splits", "rows")),
        "moe_gather": (mxg.moe_gather, dict(x=z(2, 8), rows=rows, out=z(4, 8)), ("x", "out"), ("out",)),
        "moe_combine": (mxg.moe_combine, dict(y=z(4, 8), rows=rows, weights=z(2, 2), out=z(2, 8)), ("y", "weights", "out"),
                        ("out",)),
        "moe_combine_backward": (mxg.moe_combine_backward,
                                 dict(dout=z(2, 8), y=z(4, 8), rows=rows, weights=z(2, 2), dy=z(4, 8), dweights=z(2, 2)),
                                 ("dout", "y", "weights", "dy", "dweights"), ("dy", "dweights")),
        "moe_route_backward": (mxg.moe_route_backward,
                               dict(dweights=z(2, 2), ids=rows, weights=z(2, 2), logits=z(2, 5), dlogits=z(2, 5)),
                               ("dweights", "weights", "logits", "dlogits"), ("dlogits",)),
        "int8_quantize_rowwise": (mxg.int8_quantize_rowwise,
                                  dict(x=z(2, 16, d=BF), rows=rows, q=z(4, 16, d=torch.int8), scale=z(4)), ("x", "scale"),
                                  ("q", "scale")),
    }


NAMES = ["moe_sort", "moe_gather", "moe_combine", "moe_combine_backward", "moe_route_backward", "int8_quantize_rowwise"]


@pytest.mark.parametrize("name", NAMES)
def test_autograd(name):
    fn, args, diff, written = calls()[name]
    fn(**args, check=True)
    for k in diff:
        asks = {**args, k: args[k].detach().clone().requires_grad_()}
        with pytest.raises(ValueError, match="forward only"):
            fn(**asks)
        with torch.no_grad():
            fn(**asks)
    versions = {k: t._version for k, t in args.items() if isinstance(t, torch.Tensor)}
    fn(**args)
    assert all(args[k]._version == v + (k in written) for k, v in versions.items())


@pytest.mark.parametrize("name", NAMES)
def test_arguments_that_do_not_fit_are_refused(name):
    fn, args, _, _ = calls()[name]
    for k, t in args.items():
        if not isinstance(t, torch.Tensor):
            continue
        wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=DEV)
        for bad in (t.double() if t.is_floating_point() else t.long(), t.cpu(), t.unsqueeze(0), wide, wide[..., ::2],
                    t.new_zeros(())):
            with pytest.raises((ValueError, _mxg().MXGError)):
                fn(**{**args, k: bad})


def test_workspace_and_status():
    mxg = _mxg()
    u8 = torch.uint8
    ids = torch.zeros(3000, 2, dtype=torch.int32, device=DEV)
    a = mxg.Int8Operand(torch.zeros(700, 64, dtype=torch.int8, device=DEV), torch.ones(700, device=DEV))
    b = mxg.Int8Operand(torch.zeros(64, 64, dtype=torch.int8, device=DEV), torch.ones(64, device=DEV))
    for fn, args, need in ((mxg.moe_sort, (ids, 7), mxg.moe_sort_workspace_size(3000, 2, 7)),
                           (mxg.int8_gemm_dense, (a, b), mxg.int8_gemm_workspace_size(1, 700, 64, 64, "int8"))):
        whole = torch.zeros(2 * need + 256, dtype=u8, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        fn(*args, workspace=whole[256:256 + need], status=st, check=True)
        for bad in (torch.zeros(1, dtype=u8, device=DEV).expand(need), whole[: 2 * need: 2], whole[: need // 4 * 4].view(F32),
                    whole[: need - 1], whole[8: need + 8], whole.cpu()):
            with pytest.raises((ValueError, mxg.MXGError)):
                fn(*args, workspace=bad)
        for bad in (torch.zeros(1, dtype=u8, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)):
            with pytest.raises(ValueError):
                fn(*args, status=bad)


def test_two_threads_on_one_stream():
    """Each thread's calls have a workspace of their own."""
    import threading
    mxg = _mxg()
    data = [inputs(7), inputs(8)]
    want = [step(mxg, s) for s in data]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        for _ in range(40):
            got = step(mxg, data[i])
            torch.cuda.synchronize()
            if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
