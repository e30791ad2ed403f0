"""Infinities, NaN, overflow and the precision of intermediates in the serving
operators, at sizes that take each of their forms."""

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16_MAX = (2.0 - 2.0 ** -7) * 2.0 ** 127


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _mxg():
    import fp8_bf16_mxfp4_gb300 as mxg
    return mxg


def f64(t):
    return t.detach().cpu().double().numpy()


# --------------------------------------------------------------------------- adapters

# tokens, K, N, rank, adapters: the first takes the per-token form (its adapters' reads, T * R * (K + N) values of
# 2 bytes, stay below 150 MB), the second 128-token tiles
FORMS = {"per_token": (60, 264, 1544, 16, 4), "tiles": (600, 1800, 2416, 32, 4), "tiles_wide_rank": (400, 264, 1544, 128, 4)}
assert all((T * R * (K + N) * 2 > 150e6) == name.startswith("tiles") for name, (T, K, N, R, n) in FORMS.items())


def adapters(form, dtype, seed=0):
    T, K, N, R, n = FORMS[form]
    g = torch.Generator().manual_seed(seed + T)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    x, y = rnd(T, K), rnd(T, N).to(dtype)
    A, B = (rnd(n, R, K) * K ** -0.5).to(torch.bfloat16), (rnd(n, N, R) * R ** -0.5).to(torch.bfloat16)
    ids = torch.randint(-1, n, (T,), generator=g).to(torch.int32)
    return y, x, A, B, ids


def check(y, x, A, B, ids, scale=None):
    """lora_add against the definition in 64 bits: where that is infinite or NaN, so is the result."""
    dtype = y.dtype
    sc = [1.0] * A.shape[0] if scale is None else scale.tolist()
    with np.errstate(invalid="ignore", over="ignore"):
        want, bound = serve.lora_add(f64(y), f64(x), f64(A), f64(B), ids.tolist(), sc)
        to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        got = f64(_mxg().lora_add(to(y), to(x), to(A), to(B), to(ids), to(scale), check=True))
        fin = np.isfinite(want)
        tol = bound + np.abs(want) * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23) + 2.0 ** -126
        assert np.array_equal(np.isnan(got), np.isnan(want)), f"{(np.isnan(got) != np.isnan(want)).sum()} differ in NaN"
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf])
        assert (np.abs(got[fin] - want[fin]) <= tol[fin]).all()
    return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", list(FORMS))
def test_lora_infinite_and_overflowing_products(form, dtype):
    """A x that is infinite, or finite but past the largest BF16, against a finite B."""
    y, x, A, B, ids = adapters(form, dtype)
    A[2] = 0
    A[2, :, :2] = 1.0                         # adapter 2: x0 + x1 in every rank
    B[2] = B[2].abs().clamp(min=2.0 ** -6) * 2.0 ** -120  # exact, of one sign, and keeps the sums in range
    at = (torch.arange(len(ids)) % 7 == 1).nonzero().flatten()
    ids[at] = 2
    x[at] = 0
    x[at[0::4], 0] = BF16_MAX                 # past the largest BF16 by 3/4 of its step: finite in FP32
    x[at[0::4], 1] = 1.5 * 2.0 ** 119
    x[at[1::4], 0] = -BF16_MAX
    x[at[1::4], 1] = -1.5 * 2.0 ** 119
    x[at[2::4], 0] = float("inf")
    x[at[3::4], 1] = -float("inf")
    want = check(y, x, A, B, ids)
    assert np.isinf(want[at[2::4]]).all() and np.isfinite(want[at[0::4]]).all()
    rest = torch.ones(len(ids), dtype=torch.bool)
    rest[at] = False
    assert np.isfinite(want[rest]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", list(FORMS))
def test_lora_infinite_columns(form, dtype):
    """Infinities and NaN in B, against A x of either sign, with and without a part below BF16's step, and zero."""
    y, x, A, B, ids = adapters(form, dtype, seed=1)
    N = B.shape[1]
    B[1, 5, 3], B[1, N - 1, 0], B[1, 129, 1], B[1, 300, 2] = float("inf"), -float("inf"), float("inf"), float("nan")
    A[1, 1] = 0
    A[1, 1, 0] = 1.0                          # rank 1: A x = x0, a BF16 value
    one = (ids == 1).nonzero().flatten()
    x[one[0], 0] = 0                          # 0 * inf
    x[one[1]] = float("nan")
    x[one[2], 0] = float("inf")               # infinite in every rank that uses it
    want = check(y, x, A, B, ids)
    assert np.isinf(want[one[3:]][:, [5, N - 1, 129]]).all() and np.isnan(want[one, 300]).all()
    assert np.isnan(want[one[0], 129]) and np.isnan(want[one[1]]).all()
    cols = [c for c in range(N) if c not in (5, N - 1, 129, 300)]
    assert np.isfinite(want[one[3:]][:, cols]).all()
    assert np.isfinite(want[(ids != 1).numpy()]).all()


# --------------------------------------------------------------------------- experts


def operand(w, fmt, groups):
    """float64 weights that the format holds exactly -> packed operand on the device."""
    import oracle
    from gpu_util import u8_to_dev
    t = torch.from_numpy(w).to(torch.bfloat16)
    assert np.array_equal(f64(t), w)
    data, scale = oracle.quantize_mx_rowwise(t.view(torch.int16).numpy().view(np.uint16), fmt)
    codes = oracle.unpack_e2m1(data) if fmt == "e2m1" else data
    assert np.array_equal(oracle.dequantize_mx(codes, scale, fmt), w)
    packed = oracle.pack_scales_mma(scale, [w.shape[0] // groups] * groups)
    return _mxg().MXOperand(u8_to_dev(data), u8_to_dev(packed), fmt, w.shape[1], "packed")


def silu_rounded(g, u):
    """silu(g) * u rounded to MXFP8 from exact g and u, and how far fp32 arithmetic may land from it: a few units of
    the result (16, as in the oracle), and the step of a subnormal exp and silu."""
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    return serve.mxfp8_f64(h, 16 * serve.U * np.abs(h) + np.abs(u) * (np.abs(g) + 1) * 2.0 ** -148)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("up", [0, 100])
def test_experts_gates_far_below_zero(fmt, up):
    """Gates at which exp(-g) is near the end of the FP32 range or past it, where silu(g) is tiny and not zero."""
    H = I = 128
    # each block of 32 channels has one gate: 64 a + 16 b + c / 16 with weights of 4 bits
    parts = [(-64, -24, 8), (-64, -24, 0), (-64, -24, -8), (-64, -24, -32)]
    x = np.zeros((1, H))
    x[0, :3] = 1, 1, 2.0 ** -4
    w13 = np.zeros((2 * I, H))
    w13[:I, :3] = np.repeat(np.array(parts, float), 32, 0)
    w13[I:, 0] = 2.0 ** up * np.where(np.arange(I) % 3 == 1, -1.5, 1.0)
    g, u = x[0] @ w13[:I].T, x[0] @ w13[I:].T
    assert sorted(set(g)) == [-90, -88.5, -88, -87.5]
    want, off = silu_rounded(g[None], u[None])
    got = _mxg().moe_experts(torch.from_numpy(x).to(torch.bfloat16).to(DEV), torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                             torch.ones(1, 1, device=DEV), operand(w13, fmt, 1), operand(np.eye(H, I), fmt, 1),
                             out_dtype=torch.float32, check=True)
    assert (want != 0).all()
    assert (np.abs(f64(got) - want) <= off + serve.U * np.abs(want)).all()


GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def expert_layer(T, E, k, H, I, fmt, seed, scale=1.0 / 16):
    """(x, ids, weights, W13, W2) as numpy values that the formats hold exactly, and as the call's arguments."""
    rng = np.random.default_rng(seed)
    pick = lambda v, *s: rng.choice(v, s) * rng.choice([-1.0, 1.0], s)  # noqa: E731
    x, w13, w2 = pick(GRID, T, H), pick(GRID, E * 2 * I, H) * scale, pick(GRID, E * H, I) * scale
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    wts = rng.random((T, k)).astype(np.float32) + 0.25
    ops = operand(w13, fmt, E), operand(w2, fmt, E)
    return x, ids, wts, w13, w2, ops


def run_experts(x, ids, wts, ops, dtype=torch.float32):
    return _mxg().moe_experts(torch.from_numpy(x).to(torch.bfloat16).to(DEV), torch.from_numpy(ids).to(DEV),
                              torch.from_numpy(wts).to(DEV), *ops, out_dtype=dtype, check=True)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,E,k,H,I", [(5, 2, 2, 256, 128), (70, 3, 2, 384, 256), (200, 2, 1, 128, 256), (13, 3, 2, 4096, 512),
                                       (9, 2, 1, 384, 4096)])
def test_experts_nan_stays_with_its_token(T, E, k, H, I, fmt):
    """NaN in a token (all of it, or one value) or in a routing weight reaches no other row: not through tiles that the
    token shares, nor through what it leaves in the stage buffers, partial sums or the workspace."""
    x, ids, wts, _, _, ops = expert_layer(T, E, k, H, I, fmt, seed=T)
    ids[T - 1] = -1
    want = run_experts(x, ids, wts, ops)
    assert bool(want.isfinite().all()) and not want[T - 1].any()
    bad = sorted({0, T // 3, T // 2, T - 2})
    for t in bad:
        x[t] = np.nan
    x[bad[-1]] = 0.5
    x[bad[-1], H - 1] = np.nan
    x[T - 1] = np.nan  # no slot: still zeros
    others = [t for t in range(T) if t not in bad]
    for _ in range(2):
        got = run_experts(x, ids, wts, ops)
        assert bool(got[bad].isnan().all()) and torch.equal(got[others], want[others])
    wts[1, 0] = np.nan
    got = run_experts(x, ids, wts, ops)
    others = [t for t in others if t != 1]
    assert bool(got[1].isnan().all()) and torch.equal(got[others], want[others])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_experts_infinities_saturate(fmt, dtype):
    """An infinite x, and a product silu(g) * u past the FP32 range, become 448 * 2^120 in MXFP8, as the quantizers
    have it; the other tokens do not change."""
    T, E, k, H, I = 12, 2, 2, 384, 256
    x, ids, wts, w13, w2, ops = expert_layer(T, E, k, H, I, fmt, seed=3, scale=2.0 ** -16)
    want = run_experts(x, ids, wts, ops, dtype)
    hit = {2: (100, 1.0), 7: (383, -1.0)}
    for t, (c, s) in hit.items():
        x[t, c] = s * np.inf
    got = run_experts(x, ids, wts, ops, dtype)
    others = [t for t in range(T) if t not in hit]
    assert torch.equal(got[others], want[others])
    q = _mxg().mx_quantize_rowwise(torch.from_numpy(x).to(torch.bfloat16).to(DEV), "e4m3")
    top = 448 * 2.0 ** 120
    for t, (c, s) in hit.items():
        codes, sc = q.data[t, c // 32 * 32: c // 32 * 32 + 32].cpu().numpy(), int(q.scale[t, c // 32])
        assert sc == 247 and codes[c % 32] == (0x7E if s > 0 else 0xFE) and not (np.delete(codes, c % 32) & 0x7F).any()
        xq = x[t].copy()
        xq[c // 32 * 32: c // 32 * 32 + 32] = 0
        xq[c] = s * top
        row, bound = np.zeros(H), np.zeros(H)
        for j, e in enumerate(ids[t]):
            gu = w13[e * 2 * I:(e + 1) * 2 * I] @ xq
            assert np.abs(gu).max() < 2.0 ** 126
            with np.errstate(over="ignore"):
                h = gu[:I] / (1.0 + np.exp(-gu[:I])) * gu[I:]
            inf = np.abs(h) > np.finfo(np.float32).max
            assert inf.reshape(-1, 32).any(1).all() and (np.abs(h[~inf]) < 2.0 ** 110).all()  # the rest rounds to 0
            hq = np.where(inf, np.sign(h) * top, 0.0)
            W = w2[e * H:(e + 1) * H]
            row += wts[t, j] * (W @ hq)
            bound += wts[t, j] * (I + 8) * serve.U * (np.abs(W) @ np.abs(hq))
        tol = bound + np.abs(row) * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22)
        assert np.isfinite(row).all() and (np.abs(f64(got[t]) - row) <= tol).all()


# --------------------------------------------------------------------------- routing


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(500, 2, 1), (500, 5, 2), (400, 32, 8), (300, 161, 6), (200, 512, 32)])
def test_route_weights_within_their_own_terms(T, E, k, renorm):
    """The weights' error by the terms that are summed: k or E additions, exp (2 units), its argument's rounding
    (a unit of the difference of logits, in numerator and sum) and the division."""
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(T, E, generator=g)
    ids, w = _mxg().moe_route(logits.to(DEV), k, renormalize=renorm)
    want_ids, want = serve.route(f64(logits), k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    spread = float((logits.max(1).values - logits.min(1).values).max())
    rtol = ((k if renorm else E) + 6 + 2 * spread) * 2.0 ** -24
    np.testing.assert_allclose(f64(w), want, rtol=rtol, atol=0)
