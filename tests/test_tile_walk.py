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
