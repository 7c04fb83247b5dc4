"""Block tables planned on the GPU against a plain simulation on the host: plans, cuts, windows, refusals, graphs."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import serving_q8_encode_gb300 as pk
    return pk


class Sim:
    """The tables' state as lists, and what plan and cut say they do."""

    def __init__(self, A, M, P, page, window=0, sinks=0):
        self.A, self.M, self.P, self.page, self.window = A, M, P, page, window
        self.lead = -(-sinks // page)
        self.table = [[-1] * M for _ in range(A)]
        self.lens, self.first = [-1] * A, [self.lead] * A
        self.ring, self.head, self.tail = list(range(P)), 0, P

    def pages(self, n):
        return -(-max(0, n) // self.page)

    def give(self, s, p):
        self.ring[self.tail % self.P] = self.table[s][p]
        self.table[s][p] = -1
        self.tail += 1

    def cut(self, keep):
        for s, k in enumerate(keep):
            stay = -1 if k < 0 else min(self.lens[s], k)
            for p in range(self.pages(stay), self.pages(self.lens[s])):
                if p < self.lead or p >= self.first[s]:
                    self.give(s, p)
            self.first[s] = self.lead if stay < 0 else min(self.first[s], max(self.lead, self.pages(stay)))
            self.lens[s] = stay

    def plan(self, new, n_rows):
        free, refused, row = self.tail - self.head, False, 0
        starts, before, after, slots, places = [0], [], [], [-1] * n_rows, [-1] * n_rows
        grants = []
        for s, n in enumerate(max(0, x) for x in new):
            old = max(0, self.lens[s])
            fits = self.pages(old + n) <= self.M and row + n <= n_rows
            need = self.pages(old + n) - self.pages(old) if fits else 0
            refused = refused or need > free
            ok = n > 0 and fits and (need == 0 or not refused)
            free -= need if ok else 0
            grants.append((s, old, n, row, ok))
            row += n
            starts.append(min(row, n_rows))
            before.append(old if ok else -1)
            after.append(old + n if ok else -1)
        taken = []
        for s, old, n, at, ok in grants:
            if ok:
                for p in range(self.pages(old), self.pages(old + n)):
                    taken.append((s, p, self.ring[self.head % self.P]))
                    self.head += 1
        if self.window:
            for s in range(self.A):
                if self.lens[s] >= 0:
                    behind = min(max(0, self.lens[s] + 1 - self.window) // self.page, self.pages(self.lens[s]))
                    for p in range(max(self.first[s], self.lead), behind):
                        self.give(s, p)
                    self.first[s] = max(self.first[s], behind) if behind > max(self.first[s], self.lead) else self.first[s]
        for s, p, i in taken:
            self.table[s][p] = i
        for s, old, n, at, ok in grants:
            if ok:
                self.lens[s] = old + n
                for i in range(n):
                    places[at + i] = old + i
                    slots[at + i] = self.table[s][(old + i) // self.page] * self.page + (old + i) % self.page
        return starts, before, after, slots, places

    def check(self, t):
        assert t.lens.tolist() == self.lens
        assert t.block_table.tolist() == self.table
        assert t.first.tolist() == self.first
        assert t.counts.tolist() == [self.head, self.tail]
        free = [self.ring[i % self.P] for i in range(self.head, self.tail)]
        ring = t.ring.tolist()
        assert [ring[i % self.P] for i in range(self.head, self.tail)] == free
        held = [i for row in self.table for i in row if i >= 0]
        assert sorted(held + free) == list(range(self.P))   # every page in one place


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same(plan, want):
    for got, ref in zip(plan, want):
        assert got.tolist() == ref


@pytest.mark.parametrize("A,M,P,page,window,sinks", [
    (1, 1, 1, 16, 0, 0), (3, 9, 20, 16, 0, 0), (7, 40, 90, 16, 50, 4), (5, 12, 31, 32, 33, 40), (40, 6, 77, 64, 1, 0),
    (600, 5, 1500, 16, 17, 16), (4096, 3, 5000, 128, 0, 0), (33, 20, 300, 128, 200, 129),
])
def test_plans_and_cuts(pk, A, M, P, page, window, sinks):
    rng = random.Random(A * 31 + page)
    t, sim = pk.PageTable(A, M, P, page, window=window, sinks=sinks), Sim(A, M, P, page, window, sinks)
    last = list(sim.lens)
    for step in range(12 if A < 1000 else 4):
        most = max(1, M * page // 3)
        new = [rng.choice([0, 1, 1, rng.randint(0, most), -3]) for _ in range(A)]
        n_rows = sum(max(0, x) for x in new) + rng.choice([0, 0, 5])
        last = list(sim.lens)
        same(t.plan(ints(new), n_rows), sim.plan(new, n_rows))
        sim.check(t)
        # some end, some lose what the plan added or part of it, some stay
        keep = [rng.choice([1 << 30, 1 << 30, -1, b if b >= 0 else -1, rng.randint(max(0, b), max(0, b, n)), n])
                for b, n in zip(last, sim.lens)]
        t.cut(ints(keep))
        sim.cut(keep)
        sim.check(t)
    assert t._arrivals.item() == 0


def test_refusals_leave_no_trace(pk):
    t, sim = pk.PageTable(4, 4, 6, 16), Sim(4, 4, 6, 16)
    new = [40, 64, 3, 5]        # 3 pages; 4 that are not there; 1 behind the refusal; 1
    same(t.plan(ints(new), 112), sim.plan(new, 112))
    assert sim.lens == [40, -1, -1, -1]
    new = [5, 0, 0, 0]          # needs no page: granted
    same(t.plan(ints(new), 5), sim.plan(new, 5))
    sim.check(t)
    assert t.status() == 0      # no free pages is an ordinary thing
    # rows behind n_rows, and more tokens than a table holds, are flagged
    new = [1, 16, 16, 65]
    same(t.plan(ints(new), 20), sim.plan(new, 20))
    sim.check(t)
    with pytest.raises(pk.PolyKVError) as e:
        t.status()
    assert e.value.status == 6
    assert t.status() == 0


def test_no_rows_and_idle_slots(pk):
    t, sim = pk.PageTable(3, 4, 6, 16), Sim(3, 4, 6, 16)
    same(t.plan(ints([0, 0, 0]), 0), sim.plan([0, 0, 0], 0))
    t.cut(ints([5, 0, -1]))
    sim.cut([5, 0, -1])
    sim.check(t)


def test_long_prompts_over_many_blocks(pk):
    A, M, page, P = 20, 2048, 16, 30000
    new = [1, 0, 32767, 17, 32768] + [9000 + i for i in range(15)]
    t, sim = pk.PageTable(A, M, P, page), Sim(A, M, P, page)
    same(t.plan(ints(new), sum(new)), sim.plan(new, sum(new)))
    sim.check(t)
    keep = [i * 1000 - 1 for i in range(A)]
    t.cut(ints(keep))
    sim.cut(keep)
    sim.check(t)


def test_counters_pass_32_bits(pk):
    t, sim = pk.PageTable(3, 4, 7, 16), Sim(3, 4, 7, 16)
    at = (1 << 33) + 5
    ring = [0] * 7
    for i in range(7):
        ring[(at + i) % 7] = i
    t.restore(t.block_table.clone(), t.lens.clone(), t.first.clone(), ints(ring), torch.tensor([at, at + 7]).cuda())
    sim.ring, sim.head, sim.tail = ring, at, at + 7
    for _ in range(5):
        same(t.plan(ints([20, 3, 30]), 53), sim.plan([20, 3, 30], 53))
        t.cut(ints([-1, 0, 18]))
        sim.cut([-1, 0, 18])
        sim.check(t)


def test_broken_state_stays_inside_the_buffers(pk):
    """A state that no call left: what it names is flagged, nothing else is touched."""
    t = pk.PageTable(4, 4, 6, 16, window=8)
    t.lens.copy_(ints([1000, 64, -7, 3]))
    t.first.copy_(ints([-9, 100, 3, 0]))
    t.ring.fill_(77)
    t.counts.copy_(torch.tensor([-5, 90]).cuda())
    p = t.plan(ints([1, 1, 1, 1]), 4)
    t.cut(ints([0, 5, -1, 1]))
    assert all(x in range(-1, 6) for row in t.block_table.tolist() for x in row)
    assert all(x in range(-1, 6 * 16) for x in p.slots.tolist())
    with pytest.raises(pk.PolyKVError):
        t.status()


def test_captured_graph_follows_the_state(pk):
    t, sim = pk.PageTable(5, 30, 120, 16, window=30, sinks=3), Sim(5, 30, 120, 16, 30, 3)
    new, keep = ints([0] * 5), ints([1 << 30] * 5)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        t.plan(new, 64)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p = t.plan(new, 64)
        t.cut(keep)
    rng = random.Random(4)
    for _ in range(15):
        n = [rng.choice([0, 1, 1, 12]) for _ in range(5)]
        k = [rng.choice([1 << 30, 1 << 30, -1, (sim.lens[i] if sim.lens[i] >= 0 else -1)]) for i in range(5)]
        new.copy_(ints(n))
        keep.copy_(ints(k))
        g.replay()
        same(p, sim.plan(n, 64))
        sim.cut(k)
        sim.check(t)


def test_other_stream(pk):
    t, sim = pk.PageTable(3, 4, 9, 16), Sim(3, 4, 9, 16)
    s = torch.cuda.Stream()
    new = ints([10, 0, 17])
    s.wait_stream(torch.cuda.current_stream())
    p = t.plan(new, 27, stream=s)
    t.cut(new, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    same(p, sim.plan([10, 0, 17], 27))
    sim.cut([10, 0, 17])
    sim.check(t)
