"""The hand-overs of the tile kernel (chunk_tile.cu) drawn up as a graph: what every warp role does with a
piece, in its order, and every barrier's arrivals before the waits for them.  What is kept in a ring (the query
rows' scales, a tile's page flags and scales) must be read before the graph lets its place be written again: a
pair of accesses without a path between them is a race, however far apart they lie in time.  CPU only; the sizes
of the rings come from the source."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "mqa_kv_cache_b200", "csrc", "chunk_tile.cu")


def _source():
    with open(SRC, encoding="utf-8") as f:
        return f.read()


def _number(name):
    return int(re.search(r"constexpr int %s = (\d+);" % name, _source()).group(1))


PIECES, RING = _number("PIECES"), _number("RING")


def _scale_places():
    """How many pieces' query scales are kept: the index that the writer and the reader both use."""
    used = set(re.findall(r"s_qs \+ \(n (&|%) (\w+)\) \* CH_ROWS", _source()) + re.findall(r"s_qs\[\(n (&|%) (\w+)\) \* CH_ROWS", _source()))
    assert len(used) == 1, used
    op, by = used.pop()
    return int(by) + 1 if op == "&" else {"PIECES": PIECES}[by]


def _slots(d, qt, fp8):
    """(16-bit K/V slots, code slots) of TCfg<d, fp8, qt>."""
    s = _source()
    assert "NS = (FP8 ? 3 : 6 - QT) * 2 / HALVES" in s and "LS = !FP8 ? 0 : QT == 2 ? 4 / HALVES : D == 128 ? 4 : 6" in s
    halves = d // 64
    if not fp8:
        return (6 - qt) * 2 // halves, 0
    return 3 * 2 // halves, 4 // halves if qt == 2 else 4 if d == 128 else 6


class Graph:
    """Nodes by name with the nodes that precede them."""

    def __init__(self):
        self.before = {}

    def node(self, name, *preds):
        self.before.setdefault(name, set()).update(p for p in preds if p is not None)
        return name

    def ancestors(self):
        """{node: bits of all that precede it}; a cycle (a deadlock) fails."""
        bit = {v: 1 << i for i, v in enumerate(self.before)}
        done, on = {}, set()
        for root in self.before:
            stack = [root]
            while stack:
                v = stack[-1]
                if v in done:
                    stack.pop()
                    continue
                assert all(p in self.before for p in self.before[v]), (v, self.before[v])
                todo = [p for p in self.before[v] if p not in done]
                if todo:
                    on.add(v)
                    assert not any(p in on for p in todo), f"deadlock at {v}"
                    stack += todo[:1]
                else:
                    m = 0
                    for p in self.before[v]:
                        m |= done[p] | bit[p]
                    done[v] = m
                    on.discard(v)
                    stack.pop()
        return bit, done


class Agent:
    """A warp role: its nodes follow one another; each may also wait for others."""

    def __init__(self, g, name):
        self.g, self.name, self.at = g, name, None

    def do(self, what, *waits):
        self.at = self.g.node((self.name,) + what, self.at, *waits)
        return self.at


def handovers(pieces, d, qt, places, fp8=True):
    """pieces: (pair, steps of buffer 0, steps of buffer 1).  -> the graph, and the pairs that have to be ordered."""
    NS, LS = _slots(d, qt, fp8)
    g = Graph()
    H, L, W, S, P = (Agent(g, x) for x in ("pieces", "loads", "widen", "scores", "values"))
    A = [Agent(g, "softmax0"), Agent(g, "softmax1")]
    takers = ("loads", "scores", "values", "softmax0", "softmax1") + (("widen",) if fp8 else ())
    landed = ("widen", "kv_full") if fp8 else ("kv_full",)  # what the products wait for
    x0, steps, joins = 0, [0, 0], 0
    commits = {"scores": None, "values": None}  # MMAs finish in the order of their issue

    def commit(agent, name):
        commits[agent.name] = g.node(name, agent.at, commits[agent.name])

    for n, (pair, n0, n1) in enumerate(pieces):
        nt, most = (n0, n1), max(n0, n1)
        tiles = (most + 1) // 2 if pair else most
        tile = lambda i: i // 2 if pair else i  # noqa: E731
        # warp 19
        H.do(("put", n), *([(t, "empty", n - PIECES) for t in takers] if n >= PIECES else []))
        if n:
            H.do(("q", n), ("q_empty", n - 1))
        g.node(("q_full", n), H.at)
        # warp 17
        L.do(("take", n), ("pieces", "put", n))
        L.do(("empty", n))
        for j in range(tiles):
            it = x0 // 2 + j
            L.do(("flags", it))
            for kv in range(2):
                x = x0 + 2 * j + kv
                if fp8:
                    L.do(("load", x), ("widen", "land_empty", x - LS) if x >= LS else None)
                else:
                    L.do(("load", x), ("kv_empty", x - NS) if x >= NS else None)
                g.node(("land_full" if fp8 else "kv_full", x), L.at)
        # the widening warps
        if fp8:
            W.do(("take", n), ("pieces", "put", n))
            W.do(("empty", n))
            W.do(("scales", n), ("q_full", n))
            W.do(("q_ready", n))
        for j in range(tiles if fp8 else 0):
            for kv in range(2):
                x = x0 + 2 * j + kv
                W.do(("use", x), ("land_full", x), ("kv_empty", x - NS) if x >= NS else None)
                W.do(("kv_full", x))
                W.do(("land_empty", x))
        # warps 16 and 18
        for agent, kv in ((S, 0), (P, 1)):
            agent.do(("take", n), ("pieces", "put", n))
            agent.do(("empty", n))
            if kv == 0:
                agent.do(("q", n), ("widen", "q_ready", n) if fp8 else ("q_full", n))
            step = list(steps)
            for i in range(most):
                x = x0 + 2 * tile(i) + kv
                if not pair or i % 2 == 0:
                    agent.do(("wait", x), landed + (x,))
                for t in range(2):
                    if i >= nt[t]:
                        continue
                    k = step[t]
                    step[t] += 1
                    if kv == 0:
                        agent.do(("mma", t, k), ("pv_done", t, k - 2) if k >= 2 else None)
                        commit(agent, ("s_full", t, k))
                    else:
                        agent.do(("mma", t, k), ("softmax%d" % t, "p_full", t, k))
                        commit(agent, ("pv_done", t, k))
                if not pair or i % 2 or i + 1 == most:
                    commit(agent, ("kv_empty", x))
            if kv == 0:
                commit(agent, ("q_empty", n))
        # the softmax groups
        for t in range(2):
            a = A[t]
            a.do(("take", n), ("pieces", "put", n))
            for k in range(nt[t]):
                a.do(("step", n, k), ("s_full", t, steps[t] + k))
                if k == 0 and fp8:
                    a.do(("read_scales", n))
                a.do(("read_tile", x0 // 2 + tile(k), k))
                a.do(("p_full", t, steps[t] + k))
            if nt[t]:
                a.do(("last", n), ("pv_done", t, steps[t] + nt[t] - 1))
            if not pair:
                a.do(("join0", joins))
                a.do(("joined0", joins), ("softmax%d" % (1 - t), "join0", joins))
            a.do(("empty", n))
            if not pair:
                a.do(("join1", joins))
                a.do(("joined1", joins), ("softmax%d" % (1 - t), "join1", joins))
        if not pair:
            joins += 1
        steps = [steps[0] + n0, steps[1] + n1]
        x0 += 2 * tiles
    order = []
    for v in list(g.before):
        if v[1] == "read_scales":
            order += [(v, ("widen", "scales", m)) for m in range(v[2] + places, len(pieces), places)]
        if v[1] == "read_tile" or (v[0] == "widen" and v[1] == "use"):
            it = v[2] if v[1] == "read_tile" else v[2] // 2
            for later in range(it + RING, x0 // 2, RING):
                order.append((v, ("loads", "flags", later)))
                if fp8:  # the keys' load brings the scales too
                    order.append((v, ("loads", "load", 2 * later)))
    return g, order


def _one_tile(r):
    halves = r.choice([1, 1, 1, 2, 2, 3, 4])
    return False, (halves + 1) // 2, halves // 2


def _two_tiles(r):
    n1 = r.choice([1, 1, 1, 2, 2, 3])
    return True, max(n1 - r.choice([0, 0, 0, 1]), 0), n1


def _unordered(pieces, d, qt, places, fp8=True):
    g, order = handovers(pieces, d, qt, places, fp8)
    bit, before = g.ancestors()
    assert order
    return [(a, b) for a, b in order if not before[b] & bit[a]]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qt", [1, 2])
def test_nothing_is_written_before_it_was_read(d, qt, fp8):
    r = random.Random(100 * d + qt)
    runs = [[(False, 1, 0)] * 14, [(False, 1, 1)] * 14, [(False, 1, 1), (False, 1, 0), (False, 1, 0)] * 5]
    if qt == 2:
        runs += [[(True, 1, 1)] * 14, [(True, 0, 1)] * 14, [(True, 2, 2), (False, 1, 0), (False, 1, 0)] * 5]
    for _ in range(40):
        runs.append([_two_tiles(r) if qt == 2 and r.random() < 0.6 else _one_tile(r) for _ in range(14)])
    for pieces in runs:
        assert not _unordered(pieces, d, qt, _scale_places(), fp8), pieces


@pytest.mark.parametrize("places", [2, 3])
def test_fewer_places_for_the_query_scales_are_a_race(places):
    """The model sees what it is there for: two places, and three where buffer 1 has no step in two pieces."""
    pieces = [(False, 1, 1), (False, 1, 0), (False, 1, 0)] * 5
    late = _unordered(pieces, 64, 1, places)
    assert any(b[1] == "scales" for _, b in late)
    assert all(b[1] == "scales" for _, b in late)
