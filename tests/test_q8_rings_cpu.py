"""The shared-memory rings of pruned_attn_q8's one-set kernel (two MMA issuers on alternate key tiles), as an event
model on the CPU: whatever load or role is late, every product must read the tile it is meant to read, and no role may
wait for good."""
import heapq
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "token_pruned_sparse_b200", "csrc",
                      "attn_q8.cu")


class Barrier:
    """An mbarrier of one arrival per phase. A wait on a parity ends when the phase before the current one has it:
    the parity tells a phase from its neighbours only."""

    def __init__(self):
        self.phase = 0

    def done(self, parity):
        return (self.phase & 1) != parity


class Model:
    """Roles of a CTA as generators that yield a time to sleep or a (barrier, parity) to wait for. Times in clocks."""
    LOAD, CONVERT, S, O, SOFTMAX, POLL = 1000, 250, 200, 260, 450, 30

    def __init__(self, k_stages, v_stages, c_stages, tiles, late=None, start=None, guard=False):
        self.nk, self.nv, self.nc, self.n = k_stages, v_stages, c_stages, tiles
        self.late, self.start, self.guard = late or {}, start or {}, guard
        self.now, self.heap, self.serial = 0, [], 0
        bars = lambda n: [Barrier() for _ in range(n)]                # noqa: E731
        self.k_full, self.k_empty, self.c_full, self.c_empty = bars(self.nk), bars(self.nk), bars(self.nc), bars(self.nc)
        self.v_full, self.v_empty = bars(self.nv), bars(self.nv)
        self.s_full, self.p_full = [bars(2), bars(2)], [bars(2), bars(2)]
        self.k_tile, self.v_tile = [None] * self.nk, [None] * self.nv
        self.pipe_free = 0
        self.wrong = []

    def at(self, when, action):
        self.serial += 1
        heapq.heappush(self.heap, (when, self.serial, action))

    def run(self):
        roles = {"tma": self.producer(), "conv": self.converters(), "mma0": self.issuer(0), "mma1": self.issuer(1),
                 "soft0": self.softmax(0), "soft1": self.softmax(1)}
        left = set(roles)

        def resume(name):
            try:
                what = next(roles[name])
            except StopIteration:
                left.discard(name)
                return
            if isinstance(what, tuple):
                poll(name, *what)
            else:
                self.at(self.now + what, lambda: resume(name))

        def poll(name, bar, parity):
            if bar.done(parity):
                resume(name)
            elif self.now < 200_000:
                self.at(self.now + self.POLL, lambda: poll(name, bar, parity))

        for name in roles:
            self.at(self.start.get(name, 0), lambda name=name: resume(name))
        while self.heap:
            self.now, _, action = heapq.heappop(self.heap)
            action()
        return self.wrong, sorted(left)

    @staticmethod
    def arrive(bar):
        bar.phase += 1

    def load(self, kind, q, slot, full):
        if kind == "k":
            self.k_tile[slot] = None

        def landed():
            if kind == "k":
                self.k_tile[slot] = q
            self.arrive(full)
        self.at(self.now + self.LOAD + self.late.get((kind, q), 0), landed)

    def producer(self):
        for q in range(self.n):
            s = q % self.nk
            if q >= self.nk:
                yield self.k_empty[s], (q // self.nk - 1) & 1
            self.load("k", q, s, self.k_full[s])
            s = q % self.nc
            if q >= self.nc:
                yield self.c_empty[s], (q // self.nc - 1) & 1
            self.load("c", q, s, self.c_full[s])
            yield 20

    def converters(self):
        for q in range(self.n):
            s, v = q % self.nc, q % self.nv
            yield self.c_full[s], (q // self.nc) & 1
            yield 60
            self.arrive(self.c_empty[s])
            if q >= self.nv:
                yield self.v_empty[v], (q // self.nv - 1) & 1
            yield self.CONVERT
            self.v_tile[v] = q
            self.arrive(self.v_full[v])

    def product(self, time, ring, slot, q, what):
        """An MMA of the pipe that both issuers share; the operand is looked at when it begins and when it ends."""
        def look():
            if ring[slot] != q:
                self.wrong.append((what, q, ring[slot]))
        begin = max(self.now, self.pipe_free)
        self.pipe_free = begin + time
        self.at(begin, look)
        self.at(self.pipe_free, look)

    def commit(self, bar):
        self.at(max(self.now, self.pipe_free), lambda: self.arrive(bar))

    def issuer(self, t):
        tiles = list(range(t, self.n, 2))

        def issue_s(u, q):
            self.product(self.S, self.k_tile, q % self.nk, q, "S")
            self.commit(self.s_full[t][u])
            if u == 1:
                self.commit(self.k_empty[q % self.nk])

        wait_k = lambda q: (self.k_full[q % self.nk], (q // self.nk) & 1)         # noqa: E731
        wait_v = lambda q: (self.v_full[q % self.nv], (q // self.nv) & 1)         # noqa: E731
        if tiles:
            yield wait_k(tiles[0])
            if self.guard and 1 - t < self.n:
                yield wait_k(1 - t)
            for u in range(2):
                issue_s(u, tiles[0])
        for j, q in enumerate(tiles):
            yield wait_v(q)
            if j + 1 < len(tiles):
                yield wait_k(tiles[j + 1])
            for u in range(2):
                yield self.p_full[t][u], j & 1
                self.product(self.O, self.v_tile, q % self.nv, q, "O")
                if u == 1:
                    self.commit(self.v_empty[q % self.nv])
                if j + 1 < len(tiles):
                    issue_s(u, tiles[j + 1])

    def softmax(self, t):
        for j in range(len(range(t, self.n, 2))):
            for u in range(2):
                yield self.s_full[t][u], j & 1
                yield self.SOFTMAX
                self.arrive(self.p_full[t][u])


DELAYS = (350, 600, 1700, 6000)


def _cases():
    yield {}, {}
    for kind in "kc":
        for q in range(7):
            for delay in DELAYS:
                yield {(kind, q): delay}, {}
                for other in range(q):
                    yield {(kind, q): delay, (kind, other): 900}, {}
    for role in ("tma", "conv", "mma0", "mma1", "soft0", "soft1"):
        for delay in (500, 3000, 9000):
            yield {}, {role: delay}
            for q in (0, 1):
                yield {("k", q): 2500}, {role: delay}


def _faults(k, v, c, **kw):
    """Every case of a ring that reads a wrong tile or does not end."""
    out = []
    for tiles in (1, 2, 3, 4, 5, 8, 13):
        for late, start in _cases():
            wrong, stuck = Model(k, v, c, tiles, late, start, **kw).run()
            if wrong or stuck:
                out.append((tiles, late, start, wrong[:2], stuck))
    return out


def _stages(name, d):
    """A ring's number of stages in the one-set layout, from the kernel's source."""
    expr = re.search(r"static constexpr int %s = ([^;]+);" % name, open(SOURCE).read()).group(1)

    def value(e):
        e = e.strip()
        while e.startswith("(") and e.endswith(")") and e[1:-1].count("(") == e[1:-1].count(")"):
            e = e[1:-1].strip()
        if "?" not in e:
            return eval(e.replace("||", " or ").replace("&&", " and "), {"D": d, "kOneSet": True})   # noqa: S307
        cond, rest = e.split("?", 1)
        depth = 0
        for i, ch in enumerate(rest):
            depth += {"(": 1, ")": -1, "?": 1}.get(ch, 0)
            if ch == ":":
                if depth == 0:
                    return value(rest[:i]) if value(cond) else value(rest[i + 1:])
                depth -= 1
        raise ValueError(e)
    return int(value(expr))


@pytest.mark.parametrize("d", [64, 128])
def test_every_product_of_the_one_set_kernel_reads_its_own_tile(d):
    rings = [_stages(n, d) for n in ("kKStages", "kVStages", "kCStages")]
    assert _faults(*rings) == []


def test_the_model_sees_a_phase_taken_for_the_one_before():
    """Three K stages pass from issuer to issuer: a wait for tile 3 ends before tile 0 has landed."""
    faults = _faults(3, 2, 4)
    assert any(w and w[0][:2] == ("S", 3) for _, _, _, w, _ in faults)
    assert _faults(2, 2, 4) == []
    # letting each issuer see the other's first tile as well does not do: an issuer that comes late finds that
    # phase gone and waits for a later one, which needs itself
    assert any(stuck for *_, stuck in _faults(3, 2, 4, guard=True))
