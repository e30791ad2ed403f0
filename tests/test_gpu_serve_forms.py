"""The adapter tiles at sizes that take them (each test asks lora_add_form):
strides, in place, without a scale, infinities and NaN beside other tokens, ids
out of range, and the bits that A x keeps."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_serve import BAND, banded, bands_hold, check_lora  # noqa: E402

DEV = "cuda:0"
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _mxg():
    import fp8_bf16_mxfp4_gb300 as mxg
    return mxg


def form(T, N, K, R):
    from fp8_bf16_mxfp4_gb300 import _lib
    return {1: "per_token", 2: "tiles"}[_lib.load().lora_add_form(T, N, K, R)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", [dict(pad=24), dict(pad=8, inplace=True), dict(scale=False, runs=90),
                                dict(inplace=True, scale=False), dict(pad=40, scale=False, runs=1)])
@pytest.mark.parametrize("T,K,N,R,n", [(700, 1032, 2056, 40, 5), (400, 1544, 1000, 80, 3), (260, 520, 2312, 128, 40)])
def test_tiles_strides_in_place_and_no_scale(T, K, N, R, n, kw, dtype):
    assert form(T, N, K, R) == "tiles"
    check_lora(T, K, N, R, n, dtype, **{"runs": 3, **kw})


@pytest.mark.parametrize("dtype", DTYPES)
def test_tiles_in_place_leave_rows_without_an_adapter(dtype):
    """Whole tiles, and rows inside a tile, that have no adapter: in place they are not touched, else copied."""
    T, K, N, R, n = 1100, 1032, 2056, 40, 3
    assert form(T, N, K, R) == "tiles"
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, A, B, y = rnd(T, K), rnd(n, R, K), rnd(n, N, R), rnd(T, N).to(dtype)
    for ids in (torch.full((T,), -1), torch.where(torch.arange(T) < 200, torch.arange(T) % n, -7)):
        ids = ids.to(torch.int32).to(DEV)
        off = ids < 0
        xs = x.clone()
        xs[off] = float("nan")
        want = _mxg().lora_add(y, xs, A, B, ids, check=True)
        assert bool(want.isfinite().all())
        assert torch.equal(want[off], y[off])
        z = y.clone()
        assert _mxg().lora_add(z, xs, A, B, ids, out=z, check=True).data_ptr() == z.data_ptr()
        assert torch.equal(z, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_tiles_select_rows(dtype):
    """Infinities and NaN of an adapter, or of a token, stay with its tokens; so does an id out of range."""
    mxg = _mxg()
    T, K, N, R, n = 600, 1800, 2416, 32, 5
    assert form(T, N, K, R) == "tiles"
    g = torch.Generator().manual_seed(6)
    to = lambda t: t.to(torch.bfloat16).to(DEV)  # noqa: E731
    x, y = to(torch.randn(T, K, generator=g)), to(torch.randn(T, N, generator=g)).to(dtype)
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
    for sc in (None, torch.ones(n, device=DEV)):
        for bad_id in (n, 2 ** 31 - 1):
            bad = ids.clone()
            bad[[0, 150, T - 1]] = bad_id
            r = mxg.lora_add(y, x, A, B, bad.to(DEV), sc)
            with pytest.raises(mxg.MXGError) as e:
                mxg.check_status()
            assert e.value.code == 11
            others = keep.clone()
            others[[0, 150, T - 1]] = False
            assert torch.equal(r[others], want[others])
    assert torch.equal(mxg.lora_add(y, x, A, B, ids.to(DEV), check=True)[keep], want[keep])  # the next call is whole again


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,N,R", [(40, 264, 520, 32), (600, 1800, 2416, 32), (400, 264, 1544, 128)])
def test_lora_bits_of_the_inner_product(T, K, N, R, dtype):
    """A x of 17 (BF16 output) or 24 (FP32) significant bits whose leading part y takes away: what is left is seen
    whole.  Every sum is exact in fp32 but the product's, which may truncate one unit of its value of about 1."""
    assert form(T, N, K, R) == ("tiles" if T > 100 else "per_token")
    n = 3
    g = torch.Generator().manual_seed(T)
    B = torch.randn(n, N, R, generator=g).to(torch.bfloat16)
    B[:, :, 0] = torch.randint(0, 2, (n, N), generator=g).to(torch.bfloat16) * 2 - 1
    ids = torch.randint(0, n, (T,), generator=g).to(torch.int32)
    sign = lambda *s: torch.randint(0, 2, s, generator=g) * 2.0 - 1  # noqa: E731
    lead = sign(T)
    b = B[ids.long(), :, 0].float()
    A = torch.zeros(n, R, K)
    x = torch.zeros(T, K)
    A[:, 0, 1], x[:, 1] = 1.0, lead
    if dtype == torch.bfloat16:  # 1 + m 2^-16, m below 128: two terms of 8 bits
        m = torch.randint(1, 128, (T,), generator=g) * sign(T)
        A[:, 0, K - 1], x[:, K - 1] = 2.0 ** -16, m
        left = m * 2.0 ** -16
    else:                        # 1 + m 2^-15 + k 2^-23: three
        m, k = torch.randint(1, 64, (T,), generator=g) * sign(T), torch.randint(1, 128, (T,), generator=g) * sign(T)
        A[:, 0, K - 1], x[:, K - 1] = 2.0 ** -15, m
        A[:, 0, 70], x[:, 70] = 2.0 ** -23, k
        left = m * 2.0 ** -15 + k * 2.0 ** -23
    to = lambda t: t.to(torch.bfloat16).to(DEV)  # noqa: E731
    got = _mxg().lora_add((-b * lead[:, None]).to(dtype).to(DEV), to(x), to(A), to(B), ids.to(DEV), check=True)
    off = (got.double().cpu() - (b * left[:, None]).double()).abs()
    assert float(off.max()) <= 2.0 ** -23


@pytest.mark.parametrize("dtype", DTYPES)
def test_tiles_write_only_their_output_and_workspace(dtype):
    mxg = _mxg()
    T, K, N, R, n = 601, 1032, 2056, 48, 7
    assert form(T, N, K, R) == "tiles"
    g = torch.Generator().manual_seed(T)
    to = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    args = (to(T, N).to(dtype), to(T, K), to(n, R, K), to(n, N, R), (torch.arange(T, device=DEV) % (n + 1) - 1).to(torch.int32))
    want = mxg.lora_add(*args, check=True)
    need, size = mxg.lora_add_workspace_size(T, K, R), T * N * args[0].element_size()
    wbuf, ws = banded(need)
    obuf, ob = banded(size)
    out = ob.view(dtype).view(T, N)
    assert torch.equal(mxg.lora_add(*args, out=out, workspace=ws, check=True), want)
    assert bands_hold(wbuf, need) and bands_hold(obuf, size) and BAND > 0
