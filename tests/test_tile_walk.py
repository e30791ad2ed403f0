"""The order of a product's tiles, compiled from the kernels' own header by the
host compiler, with traps on overflow and division by zero: every tile comes
once, inside its expert and the matrix, at every size that a call accepts."""

import os
import random
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp8_bf16_mxfp4_gb300", "csrc")


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("walk") / "walk")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error",
                    "-I", CSRC, "-o", exe, os.path.join(HERE, "tile_walk.cpp")], check=True)

    def ask(*words):
        r = subprocess.run([exe], input=" ".join(map(str, words)).encode(), capture_output=True)
        assert r.returncode == 0, f"{words[:6]}: ended with {r.returncode}"
        return np.frombuffer(r.stdout, np.int32)
    return ask


@pytest.mark.parametrize("group", [1, 3, 4096, 32768])
@pytest.mark.parametrize("mtn,ntn", [(1, 1), (7, 5), (3, 131072), (1, 131073), (2, 524288), (5, 65536 * 4), (1, 2 ** 24)])
def test_tile_order_of_any_size(ask, mtn, ntn, group):
    tiles, rng = mtn * ntn, random.Random(mtn)
    for local in {0, tiles - 1, tiles // 2, *(rng.randrange(tiles) for _ in range(20))}:
        g = min(group, mtn)
        first = local // (g * ntn) * g
        rows, idx = min(g, mtn - first), local - first * ntn
        assert ask("mn", local, tiles, ntn, group).tolist() == [first + idx % rows, idx // rows]


WALKS = [  # splits, N, K
    ([32], 33554432, 16), ([32], 33554688, 16), ([17, 0, 40], 33554432, 16), ([300], 33554432, 32), ([1], 134217728, 16),
    ([513, 0, 31, 256], 65536 * 64 + 264, 16), ([5000, 1, 0, 77], 520, 16), ([0, 129, 1000, 0], 2056, 400), ([70], 8, 16),
    ([9000, 40], 264, 32768), ([64] * 5, 776, 8208), ([1] * 512, 40, 64)]


@pytest.mark.parametrize("tok", [32, 64, 128, 256])
@pytest.mark.parametrize("splits,N,K", WALKS)
def test_every_unit_comes_once(ask, splits, N, K, tok):
    got = ask("walk", tok, N, K, len(splits), *splits).reshape(-1, 7)
    unit, k0, k1, e, tok0, n, chan0 = got.T
    chans = -(-N // 256)
    off = np.cumsum([0] + splits)
    assert len(got) == sum(-(-m // tok) for m in splits) * chans == len(np.unique(unit))
    assert (k0 == 0).all() and (k1 == -(-K // 128)).all()
    local = tok0 - off[e]
    assert (local >= 0).all() and (local % tok == 0).all() and (n == np.minimum(tok, off[e + 1] - tok0)).all() and (n > 0).all()
    assert (chan0 >= 0).all() and (chan0 < N).all() and (chan0 % 256 == 0).all()
    assert len(np.unique(tok0.astype(np.int64) * chans + chan0 // 256)) == len(got)


def check_runs(ask, pairs, tok, N, K, splits):
    out = ask("runs", pairs, tok, N, K, len(splits), *splits)
    used, parts, whole = out[:3].tolist()
    units, nk = sum(-(-m // tok) for m in splits) * -(-N // 256), -(-K // 128)
    assert used <= pairs
    of, buffers, counters = [[] for _ in range(units)], {}, {}
    for b, u, k0, k1, first, last, mine, as_read, counter in out[3:].reshape(-1, 9).tolist():
        assert 0 <= k0 < k1 <= nk and first <= b <= last
        of[u].append((k0, k1, b, first, last))
        if (k0, k1) != (0, nk):
            assert mine == as_read and 0 <= mine < 160        # what is read at the join is where it was put
            assert buffers.setdefault(mine, u) == u           # a buffer has one unit's sums
            assert counters.setdefault(counter, u) == u and 0 <= counter <= 640 - 8
    for parts_of in of:
        parts_of.sort()
        assert parts_of[0][0] == 0 and parts_of[-1][1] == nk and all(x[1] == y[0] for x, y in zip(parts_of, parts_of[1:]))
        assert [p[2] for p in parts_of] == list(range(parts_of[0][3], parts_of[0][4] + 1))
    return bool(parts), bool(whole)


def test_runs_cover_every_stage_once_and_joins_find_their_parts(ask):
    rng, kinds = random.Random(1), set()
    for _ in range(700):
        tok = rng.choice([32, 64, 128])
        splits = [rng.choice([0, 1, tok, rng.randint(0, 3 * tok)]) for _ in range(rng.choice([1, 1, 2, 5, rng.randint(1, 40)]))]
        N, K = 8 * rng.choice([1, 32, 33, rng.randint(1, 900)]), 16 * rng.choice([1, 8, 9, 128, 448, rng.randint(1, 1200)])
        kinds.add(check_runs(ask, rng.choice([76, 76, 74, 80, 79, 2, 1]), tok, N, K, splits))
    assert kinds == {(False, False), (False, True), (True, False)}


@pytest.mark.parametrize("splits,N,K", [([32], 264, 2 ** 27), ([100], 33554432, 16), ([2000] * 3, 4096, 2 ** 20), ([1] * 512, 520, 16)])
def test_runs_of_long_and_wide_products(ask, splits, N, K):
    for tok in (32, 128):
        check_runs(ask, 76, tok, N, K, splits)
