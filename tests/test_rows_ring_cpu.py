"""The waits of the tensor-core kernel for runs of rows, stepped through on the host in many orders: its warps as small programs
over barriers that count as the hardware's do, with the kernel's own index arithmetic. A wait knows a turn of its barrier from the
next one only, so no barrier may ever be two turns ahead of a wait, nor one behind: the model says so wherever it happens, not
only in the orders that then stand still."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "serving_q8_encode_gb300", "csrc")
SHIM = r"""
#include "rows_index.cuh"
using namespace polykv;
extern "C" {
int t_stages(int d) { return rows::ring_stages(d); }
int t_pairs() { return rows::kPairs; }
uint32_t t_barrier(uint32_t pair) { return rows::pair_barrier(pair); }
uint32_t t_parity(uint32_t pair) { return rows::pair_parity(pair); }
int t_has(int nj, int i, int j) { return rows::every_other(nj, i).has(j); }
int t_any(int nj, int i) { return rows::every_other(nj, i).any(); }
}
"""


@pytest.fixture(scope="module")
def ix(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("rows_index")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run([cxx, "-shared", "-fPIC", "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    so = ctypes.CDLL(str(lib))
    for f in (so.t_barrier, so.t_parity):
        f.restype, f.argtypes = ctypes.c_uint32, [ctypes.c_uint32]
    return so


class Bar:
    """A barrier: `turn` counts the turns that are over."""

    def __init__(self, name, count):
        self.name, self.count, self.left, self.tx, self.turn = name, count, count, 0, 0

    def _check(self):
        if self.left == 0 and self.tx == 0:
            self.left, self.turn = self.count, self.turn + 1

    def arrive(self, tx=0):
        assert self.left > 0, f"{self.name}: more arrivals than its count"
        self.left, self.tx = self.left - 1, self.tx + tx
        self._check()

    def land(self):
        self.tx -= 1
        self._check()


class Missed(Exception):
    pass


class Block:
    """One block's warps over units of the given numbers of key tiles; units: [(key tiles, both row tiles hold the same rows)]."""

    def __init__(self, ix, d, units):
        self.ix, self.NS, self.P, self.units = ix, ix.t_stages(d), ix.t_pairs(), units
        self.full = [Bar(f"full {i}", 1) for i in range(self.P)]
        self.empty = [Bar(f"empty {i}", 1) for i in range(self.P)]
        self.unit_full = [Bar(f"unit_full {i}", 1) for i in range(2)]
        self.unit_free = [Bar(f"unit_free {i}", 10) for i in range(2)]
        one = lambda name, count=1: Bar(name, count)
        self.q_ready, self.q_free, self.nearly = one("q_ready"), one("q_free"), one("nearly")
        self.s_full = [one(f"s_full {i}") for i in range(2)]
        self.o_done = [one(f"o_done {i}") for i in range(2)]
        self.p_most = [one(f"p_most {i}", 4) for i in range(2)]
        self.p_ready = [one(f"p_ready {i}", 4) for i in range(2)]
        self.half_ready, self.half_free = one("half_ready", 4), one("half_free", 4)
        self.copies, self.pipe = [], []   # in flight, in any order; products and commits, in theirs
        self.slot = [None, None]

    def turns(self, k, i):
        nj, halved = self.units[k]
        return [j for j in range(nj) if (self.ix.t_has(nj, i, j) if halved else j in self.seen(k, i))]

    def seen(self, k, i):
        """A row tile of its own does not see all of a unit's key tiles, the second one of a part of them perhaps none."""
        nj = self.units[k][0]
        return range(nj - (nj > 1 and i == 0)) if k % 3 else range(nj * i, nj)

    def any(self, k, i):
        nj, halved = self.units[k]
        return self.ix.t_any(nj, i) if halved else bool(self.turns(k, i))

    def bare(self, k, i):
        """Whether a tile without key tiles has its sums announced (it has none)."""
        return False

    def pair(self, bars, n):
        """The wait for pair n's turn: the code's barrier and parity, and the turn that it means."""
        b, turn = self.ix.t_barrier(n), sum(self.ix.t_barrier(m) == self.ix.t_barrier(n) for m in range(max(0, n - 64 * self.P), n))
        assert self.ix.t_parity(n) == turn & 1
        return bars[b], turn

    def take(self, k):
        yield self.unit_full[k & 1], k >> 1
        assert self.slot[k & 1] == k, "a unit was replaced before every warp had taken it"

    # ------------------------------------------------------------ the warps
    def unit_warp(self):
        for k in range(len(self.units) + 1):
            if k >= 1:
                yield self.nearly, k - 1
            if k >= 2:
                yield self.unit_free[k & 1], (k >> 1) - 1
            self.slot[k & 1] = k
            self.unit_full[k & 1].arrive()
            if k == len(self.units):
                return
            if k >= 1:
                yield self.q_free, k - 1
            self.q_ready.arrive(tx=1)
            self.copies.append(self.q_ready)

    def producer(self):
        issued = pair = 0
        filled = {}
        for k in range(len(self.units)):
            yield from self.take(k)
            nj = self.units[k][0]
            for j in range(nj):
                if j == max(0, nj - 2):
                    self.nearly.arrive()
                for kv in range(2):
                    s = issued % self.NS
                    if issued >= self.NS:
                        yield self.pair(self.empty, filled[s])
                    filled[s] = pair
                    issued += 1
                    bar = self.full[self.ix.t_barrier(pair)]
                    if kv or j == 0:
                        bar.arrive(tx=2 if kv and j + 1 < nj else 1)
                    self.copies.append(bar)
                    if kv == 0 or j + 1 == nj:
                        pair += 1
            self.unit_free[k & 1].arrive()
        yield from self.take(len(self.units))

    def products(self):
        commit = lambda bar: self.pipe.append(bar)
        pair, pp = 0, [0, 0]
        for k in range(len(self.units)):
            yield from self.take(k)
            nj, halved = self.units[k]
            turns = [self.turns(k, i) for i in range(2)]
            scores = lambda i: commit(self.s_full[i])
            yield self.q_ready, k
            yield self.pair(self.full, pair)
            for i in range(2):
                if 0 in turns[i]:
                    scores(i)
                if self.bare(k, i):
                    commit(self.o_done[i])
            commit(self.empty[self.ix.t_barrier(pair)])
            pair += 1
            if nj == 1:
                commit(self.q_free)
            for j in range(nj):
                more = j + 1 < nj
                yield self.pair(self.full, pair)
                for i in range(2):
                    if more and j not in turns[i] and j + 1 in turns[i]:
                        scores(i)
                for i in range(2):
                    if j not in turns[i]:
                        continue
                    yield self.p_most[i], pp[i]
                    yield self.p_ready[i], pp[i]
                    pp[i] += 1
                    if more and j + 1 in turns[i]:
                        scores(i)
                    if j == turns[i][-1]:
                        commit(self.o_done[i])
                commit(self.empty[self.ix.t_barrier(pair)])
                pair += 1
                if j + 2 == nj:
                    commit(self.q_free)
            self.unit_free[k & 1].arrive()
        yield from self.take(len(self.units))

    def softmax(self, i):
        ph = sums = halves = 0
        for k in range(len(self.units)):
            yield from self.take(k)
            for _ in self.turns(k, i):
                yield self.s_full[i], ph
                ph += 1
                self.p_most[i].arrive()
                yield None
                self.p_ready[i].arrive()
            if self.any(k, i):
                yield self.o_done[i], sums
                sums += 1
            if self.units[k][1]:
                if i == 1:
                    self.half_ready.arrive()
                    yield self.half_free, halves
                else:
                    yield self.half_ready, halves
                    yield None
                    self.half_free.arrive()
                halves += 1
            self.unit_free[k & 1].arrive()
        yield from self.take(len(self.units))

    # ------------------------------------------------------------ in some order
    def run(self, rng):
        roles = [self.unit_warp(), self.producer(), self.products()] + [self.softmax(w >> 2) for w in range(8)]
        pace = [rng.choice((1.0, 1.0, 0.1, 0.01)) for _ in roles] + [rng.choice((1.0, 0.1, 0.01)) for _ in range(2)]
        at = [next(r) for r in roles]
        while any(a != "end" for a in at):
            ready = []
            for r, a in enumerate(at):
                if a == "end":
                    continue
                if a is not None:
                    bar, turn = a
                    if not turn <= bar.turn <= turn + 1:
                        raise Missed(f"{bar.name} is at turn {bar.turn} while turn {turn} of it is waited for")
                    if bar.turn == turn:
                        continue
                ready.append(r)
            ready += [len(roles)] * bool(self.copies) + [len(roles) + 1] * bool(self.pipe)
            if not ready:
                raise Missed("standing still: " + ", ".join(f"{a[0].name} turn {a[1]}" for a in at if a not in (None, "end")))
            r = rng.choices(ready, [pace[x] for x in ready])[0]
            if r == len(roles):
                self.copies.pop(rng.randrange(len(self.copies))).land()
            elif r == len(roles) + 1:
                self.pipe.pop(0).arrive()
            else:
                at[r] = next(roles[r], "end")


def units(rng, n, most, halved=0.5):
    return [(rng.randint(1, most), rng.random() < halved) for _ in range(n)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most", [1, 2, 4, 12])
def test_no_barrier_runs_ahead_of_a_wait(ix, d, most):
    """Units of 1 .. most key tiles, in orders where any of the warps, the copies and the products may be slow."""
    rng = random.Random(1000 * d + most)
    for _ in range(60):
        Block(ix, d, units(rng, rng.randint(8, 20), most, rng.choice((0.0, 0.5, 1.0)))).run(rng)


def test_a_stage_has_a_barrier_of_its_own(ix):
    for d in (64, 128):
        assert ix.t_pairs() >= ix.t_stages(d)
    assert [ix.t_barrier(n) for n in range(ix.t_pairs())] == list(range(ix.t_pairs()))


def missed(blocks, rng):
    n = 0
    for b in blocks:
        try:
            b.run(rng)
        except Missed:
            n += 1
    return n


def test_the_model_sees_a_ring_of_too_few_barriers(ix):
    """Eight barriers beside eleven stages, as a mistake in the model: a wait is missed."""
    class Few:
        t_stages, t_pairs, t_has, t_any = staticmethod(lambda d: 11), staticmethod(lambda: 8), ix.t_has, ix.t_any
        t_barrier, t_parity = staticmethod(lambda n: n % 8), staticmethod(lambda n: n // 8 & 1)

    assert missed([Block(Few, 64, [(1, True)] * 12) for _ in range(40)], random.Random(1)) > 30


def test_the_model_sees_sums_announced_for_no_key_tiles(ix):
    """The sums of a row tile without key tiles announced all the same, as a mistake in the model: their barrier runs ahead."""
    class Always(Block):
        def any(self, k, i):
            return True

        def bare(self, k, i):
            return not self.turns(k, i)

    assert missed([Always(ix, 128, [(1, True)] * 12) for _ in range(60)], random.Random(2)) > 0
