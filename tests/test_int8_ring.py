"""A model of the rings of the tensor-core form of the integer products: the
producer, the warps that widen weights, the issuer and its completions as
agents that run in any order, mbarriers with their phase parity (a wait for a
parity also passes on the phase two before: what makes a lapped ring dangerous).
Every agent must find the stage it means, for every ring of the sources."""

import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_bf16_mxfp4_gb300", "csrc", "gemm_i8.cu")


def rings():
    """(slots in TMEM, stages in shared memory) of each tile, from the sources."""
    code = open(SRC).read()
    expr = re.search(r"kStages = (kTok == 32.*?);", code).group(1)
    cols = {t: 256 if t >= 128 else 128 if t >= 64 else 64 for t in (32, 64, 128, 256)}
    assert re.search(r"kACol = kTok >= 128 \? 256 : \(kTok >= 64 \? 128 : 64\)", code)
    stages = {int(t): int(n) for t, n in re.findall(r"kTok == (\d+) \? (\d+)", expr)}
    stages[256] = int(expr.rsplit(":", 1)[1])
    return [((512 - cols[t]) // 64, stages[t]) for t in (32, 64, 128, 256)]


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):  # the phase before the current one has this parity
        return (self.phase - 1) % 2 == parity


def run(slots, stages, total, seed):
    rng = random.Random(seed)
    full, empty, ready = ([Barrier(n) for _ in range(stages)] for n in (1, 1, 2))  # ready: a warp of either CTA
    smem, tmem = [None] * stages, [[None] * slots for _ in range(2)]
    landing, issued = [], []

    def producer():
        for i in range(total):
            s, phase = i % stages, i // stages % 2
            while not empty[s].passed(phase ^ 1):
                yield
            landing.append((i, s))

    def widen(cta):
        for i in range(total):
            s, phase = i % stages, i // stages % 2
            while not full[s].passed(phase):
                yield
            if slots < stages and i >= slots:
                j = i - slots
                while not empty[j % stages].passed(j // stages % 2):
                    yield
            assert smem[s] == i, (i, smem[s])          # the stage's own bytes
            assert tmem[cta][i % slots] in (None, ("done", i - slots)), (i, tmem[cta])  # the slot's MMAs have completed
            yield
            tmem[cta][i % slots] = i
            ready[s].arrive()

    def issuer():
        for i in range(total):
            s, phase = i % stages, i // stages % 2
            while not ready[s].passed(phase):
                yield
            issued.append((i, s))

    agents = [producer(), widen(0), widen(1), issuer()]
    live = len(agents)
    alive = [True] * len(agents)
    for _ in range(400 * total + 1000):
        what = rng.randrange(6)
        if what < 4 and alive[what]:
            try:
                next(agents[what])
            except StopIteration:
                alive[what] = False
                live -= 1
        elif what == 4 and landing:  # copies land in any order
            i, s = landing.pop(rng.randrange(len(landing)))
            smem[s] = i
            full[s].arrive()
        elif what == 5 and issued:   # MMAs complete in order; the commit reports their stage
            i, s = issued.pop(0)
            assert smem[s] == i
            for c in range(2):
                assert tmem[c][i % slots] == i, (i, tmem[c])
                tmem[c][i % slots] = ("done", i)
            empty[s].arrive()
        if live == 0 and not issued and not landing:
            return
    raise AssertionError("the ring stands still")


@pytest.mark.parametrize("slots,stages", sorted(set(rings())))
def test_every_agent_finds_its_stage(slots, stages):
    assert slots <= stages
    for seed in range(60):
        run(slots, stages, 5 * stages + 3, seed)


def test_waits_of_the_loops_keep_their_warps_in_step():
    """A stage is handed on by one lane, so every wait of a whole warp ends in a vote; the producer is one lane, and
    the final waits for work in flight are for one phase."""
    code = re.sub(r"//[^\n]*", "", open(SRC).read())
    body = code[code.index("int8_gemm_kernel(const"): code.index("struct I8Form")]
    plain = re.findall(r"ptx::mbar_wait\(([^,]*)", body)
    assert sorted(plain) == ["drain_bar", "empty_bar(stage)", "full_bar(s)"], plain
    assert len(re.findall(r"ptx::mbar_wait_warp\(", body)) == 7


class Runs:
    """How the kernel shares the stages of `units` units of `pu` stages out over at most `mp` pairs."""

    def __init__(self, units, pu, tokens, mp):
        self.pu, self.parts, total, c32 = pu, 0, units * pu, max((tokens + 31) // 32, 1)
        whole, run = -(-units // mp) * pu, max(-(-total // mp), 4)
        cut = run + (3 if run >= 2 * pu else 8 + c32 * (pu // run + 3) * 5 // 8)
        self.grain = pu if whole <= cut else 1
        self.pairs = min(mp, units if self.grain > 1 or pu == 1 else -(-total // 4))
        if units > 0 and 2 * units <= mp and pu > 1:
            n = min(mp // units, pu, max(2, int((1.6 * pu / c32) ** 0.5 + 0.5)))
            if pu // n + 5 + c32 * n * 5 // 8 < min(whole, cut):
                self.parts, self.grain, self.pairs = n, 1, units * n
        items, to = (pu, self.parts) if self.parts else (units if self.grain > 1 else total, self.pairs)
        self.q = items // to if to else 0
        self.r = items - self.q * to

    def run(self, b):
        u = b // self.parts if self.parts else 0
        i = b - u * self.parts
        s = u * self.pu + (i * self.q + min(i, self.r)) * self.grain
        return s, s + (self.q + (i < self.r)) * self.grain

    def owner(self, s):
        return s // (self.q + 1) if s < self.r * (self.q + 1) else self.r + (s - self.r * (self.q + 1)) // self.q

    def ends(self, u):
        return (u * self.parts, u * self.parts + self.parts - 1) if self.parts else \
            (self.owner(u * self.pu), self.owner(u * self.pu + self.pu - 1))


def pieces(s, end, pu):
    """The units of a run with their stages: the cut one at its start, the one at its end, whole ones."""
    while s < end:
        first, last = s // pu, end // pu
        head, tail = s - first * pu, end - last * pu
        if head or first == last:
            k1 = tail if first == last else pu
            yield first, head, k1
            s += k1 - head
        elif tail:
            yield last, 0, tail
            end -= tail
        else:
            yield first, 0, pu
            s += pu


def test_runs_cover_every_stage_once_and_joins_find_their_parts():
    rng = random.Random(1)
    kinds = set()
    for _ in range(4000):
        mp = rng.choice([76, 76, 74, 80, 2, 1])
        units = rng.choice([0, 1, 2, 5, 17, 25, 37, 38, 39, 75, 76, 77, 150, rng.randint(1, 600)])
        pu, tokens = rng.choice([1, 2, 5, 16, 56, 128, rng.randint(1, 200)]), rng.randint(0, 128)
        runs = Runs(units, pu, tokens, mp)
        kinds.add((runs.parts > 0, runs.grain > 1))
        assert runs.pairs <= mp
        of, buffers = [[] for _ in range(units)], {}
        for b in range(runs.pairs):
            s, end = runs.run(b)
            assert s < end
            for u, k0, k1 in pieces(s, end, pu):
                assert 0 <= k0 < k1 <= pu
                of[u].append((k0, k1, b))
                if (k0, k1) != (0, pu):
                    assert buffers.setdefault(2 * b + (k0 == 0), u) == u  # a buffer has one unit's sums
        joins = set()
        for u, parts in enumerate(of):
            parts.sort()
            assert parts[0][0] == 0 and parts[-1][1] == pu and all(x[1] == y[0] for x, y in zip(parts, parts[1:]))
            if len(parts) > 1:
                first, last = runs.ends(u)
                assert [p[2] for p in parts] == list(range(first, last + 1))
                assert all(buffers[2 * b + (b == first)] == u for b in range(first, last + 1))
                assert first not in joins  # the unit's counter is nobody else's
                joins.add(first)
    assert kinds == {(False, False), (False, True), (True, False)}
