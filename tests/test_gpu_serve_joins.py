"""The expert layer where its weights are cut into runs inside a unit, so that
units are joined from partial sums: both kernels, both formats, runs with a cut
head, whole units and a cut tail, a last row tile of 128, and 64-token tiles.

The weights and activations are small multiples of powers of two, so that the
first product is exact in any order of its sums; what is left is the rounding of
silu(g) * u to MXFP8 (a step where the 64-bit value lies within a few fp32 units
of a boundary) and the fp32 sums of the second product."""

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu

from gpu_util import i32_to_dev  # noqa: E402
from test_gpu_serve import BAND, banded, bands_hold  # noqa: E402
from test_gpu_serve_values import f64, operand, silu_rounded  # noqa: E402

DEV = "cuda:0"
KTOK, MAX_CTAS, MIN_STAGES = 64, 160, 4


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _mxg():
    import fp8_bf16_mxfp4_gb300 as mxg
    return mxg


def cut_runs(units, per_unit, tokens, ctas):
    """Bounds of the runs (in stages of 128 contraction elements) where units are cut, else None."""
    total, whole = units * per_unit, -(-units // ctas) * per_unit
    run = max(-(-total // ctas), MIN_STAGES)
    if whole <= run + (4 if run >= 2 * per_unit else 12 + tokens // 2) or per_unit == 1:
        return None
    n = min(ctas, -(-total // MIN_STAGES))
    q, r = divmod(total, n)
    return [b * q + min(b, r) for b in range(n + 1)]


def partials(bounds, per_unit):
    """The partial buffers that a kernel's cut units use, and the kinds of runs there are."""
    used, kinds = set(), set()
    for b, (s, e) in enumerate(zip(bounds, bounds[1:])):
        head, tail = s % per_unit, e % per_unit
        one = s // per_unit == (e - 1) // per_unit
        if one:
            if e - s < per_unit:
                used.add(2 * b + (head == 0))
                kinds.add("inside")
            continue
        if head:
            used.add(2 * b)
        if tail:
            used.add(2 * b + 1)
        if head and tail and e // per_unit > -(-s // per_unit):
            kinds.add("head, whole, tail")
    return used, kinds


def problem(T, E, k, H, I, fmt, seed):
    rng = np.random.default_rng(seed)
    pick = lambda v, *s: rng.choice(np.array(v), s) * rng.choice([-1.0, 1.0], s)  # noqa: E731
    x = pick([0, 0.5, 1, 2], T, H)
    w13 = pick([0, 0.5, 1, 1.5, 2, 3, 4, 6], E * 2 * I, H) / 16
    w2 = pick([0, 0.5, 1, 1.5, 2, 3, 4, 6], E * H, I) / 16
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    wts = rng.random((T, k)).astype(np.float32) - 0.25
    want, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        gu = x[t] @ w13[e * 2 * I:(e + 1) * 2 * I].T
        assert np.abs(gu).max(initial=0) < 2.0 ** 18  # multiples of 2^-6: exact in fp32
        hq, off = silu_rounded(gu[:, :I], gu[:, I:])
        W, w = w2[e * H:(e + 1) * H].T, wts[t, j].astype(np.float64)[:, None]
        np.add.at(want, t, w * (hq @ W))
        np.add.at(bound, t, np.abs(w) * (off @ np.abs(W) + (I + 8) * serve.U * ((np.abs(hq) + off) @ np.abs(W))))
    args = (torch.from_numpy(x).to(torch.bfloat16).to(DEV), i32_to_dev(ids), torch.from_numpy(wts).to(DEV),
            operand(w13, fmt, E), operand(w2, fmt, E))
    tiles = sum(-(-int((ids == e).sum()) // KTOK) for e in range(E))
    return args, want, bound, tiles, T * k // tiles


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,E,k,H,I,up,down", [
    (3, 1, 1, 4096, 256, "inside", None),
    (13, 3, 2, 4096, 512, "inside", None),
    (5, 2, 1, 384, 4096, None, "inside"),              # a row tile of 128 among the cut ones
    (1, 1, 1, 2560, 2560, "inside", "inside"),         # the kernels use the same buffers and counters
    (64, 1, 1, 6528, 128, "inside", None),             # a full token tile, joined from 13 parts
    (70, 1, 1, 128, 6528, None, "inside"),             # two token tiles of a single row tile of 128
    (1024, 1, 1, 1024, 2560, "head, whole, tail", None),
    (1024, 1, 1, 4992, 1024, None, "head, whole, tail"),
])
def test_joined_units(T, E, k, H, I, up, down, fmt):
    mxg = _mxg()
    args, want, bound, tiles, tokens = problem(T, E, k, H, I, fmt, seed=T + H)
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, MAX_CTAS)
    used = set()
    for kinds, units, per_unit in ((up, tiles * (I // 128), H // 128), (down, tiles * -(-H // 256), I // 128)):
        bounds = cut_runs(units, per_unit, tokens, ctas)
        assert (bounds is not None) == (kinds is not None)
        if bounds:
            bufs, found = partials(bounds, per_unit)
            assert kinds in found
            used |= bufs
    need = mxg.moe_experts_workspace_size(T, k, E, H, I)
    part_tok = min(KTOK, T * k)
    size = 2 * MAX_CTAS * part_tok * 256 * 4  # the partials are the workspace's end
    wbuf, ws = banded(need)
    obuf, ob = banded(T * H * 4)
    out = ob.view(torch.float32).view(T, H)
    got = mxg.moe_experts(*args, out=out, workspace=ws, check=True).clone()
    assert bands_hold(wbuf, need) and bands_hold(obuf, T * H * 4) and BAND > 0
    touched = (ws[need - size:].view(2 * MAX_CTAS, -1) != 0xA5).any(1).nonzero().flatten().tolist()
    assert set(touched) == used
    tol = bound + serve.U * (k + 1) * np.abs(want) + 2.0 ** -126
    bad = np.abs(f64(got) - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}"
    ws.fill_(0xFF)  # what is not written is not read
    for _ in range(4):
        assert torch.equal(mxg.moe_experts(*args, out_dtype=torch.float32, workspace=ws, check=True), got)
    assert torch.equal(mxg.moe_experts(*args), got.to(torch.bfloat16))
