"""Model check of the chunk attention's barrier protocol (host only, no GPU).

The kernel (csrc/cache_chunk.cu) runs one producer (Q, and K and V into a ring of two), one
MMA issuer for both query tiles, a warp that clears V rows outside the unit's keys, and two
softmax groups.  As in test_issuer_protocol.py, the protocol is replayed as a discrete-event
simulation under random schedules: loads land and products end at any time after their
issue, products of one thread in order.  Checked on every run: no deadlock, no
parity-ambiguous wait, every product reads the K, V, Q and P that it should, no S or P is
overwritten before it is read, and every tile's output adds up its steps in order.
"""
import random

import pytest

from tests.test_issuer_protocol import Barrier, ProtocolError, wait

NS = 2                                     # ring slots
THREADS = 3                                # softmax threads of a group (128 on the GPU)


def random_pieces(rng, n, one=False):
    """(j0, j1, [(a, e), (a, e)]): a piece's steps and what each query tile uses of them."""
    out = []
    for _ in range(n):
        j0 = rng.randrange(3)
        j1 = j0 + rng.randrange(1, 7)
        tiles = []
        for x in range(2):
            if (one and x == 1) or rng.random() < (0.05 if x == 0 else 0.25):
                tiles.append((j0, j0))     # a tile without a step in the piece
            else:
                a = rng.randrange(j0, j1)
                tiles.append((a, rng.randrange(a + 1, j1 + 1)))
        out.append((j0, j1, tiles))
    return out


def simulate(pieces, rng, mistake=None, one=False):
    """``one``: units of one query tile, one buffer of K and one of V that are freed apart."""
    bars, NB = {}, 1 if one else NS

    def bar(name, count=1):
        return bars.setdefault(name, Barrier(name, count))

    for x in range(2):
        for name in ("q_full", "q_empty", "s_full", "o_full"):
            bar((name, x))
        for name in ("p_half", "p_full"):
            bar((name, x), THREADS)
    for s in range(NS):
        for name in ("k_full", "v_full", "v_ready", "kv_empty", "k_empty"):
            bar((name, s))
    loads, products, commits = [], [], []  # in flight
    q, k, v = [None, None], [None] * NB, [None] * NB      # what lies in shared memory
    S, P, O = [None, None], [None, None], [[], []]        # and in TMEM
    read = [0, 0]                          # threads that have read the S of the step
    results = []

    def land(where, index, tag, barrier):
        def run():
            where[index] = tag
            barrier.arrive()
        loads.append(run)

    def producer():
        kv, uses = 0, [0, 0]
        for i, (j0, j1, tiles) in enumerate(pieces):
            for x in range(2):
                if tiles[x][0] < tiles[x][1]:
                    if uses[x]:
                        yield from wait(bar(("q_empty", x)), uses[x] - 1)
                    uses[x] += 1
                    land(q, x, i, bar(("q_full", x)))
            for j in range(j0, j1):
                st = kv % NS
                was = kv - NB              # the step whose buffers these are
                if was >= 0:
                    yield from wait(bar(("k_empty" if one else "kv_empty", was % NS)), was // NS)
                land(k, kv % NB, (i, j), bar(("k_full", st)))
                if one and was >= 0 and mistake != "early V":
                    yield from wait(bar(("kv_empty", was % NS)), was // NS)
                land(v, kv % NB, (i, j, "raw"), bar(("v_full", st)))
                kv += 1
                yield

    def cleaner():
        kv = 0
        for i, (j0, j1, _) in enumerate(pieces):
            for j in range(j0, j1):
                st = kv % NS
                yield from wait(bar(("v_full", st)), kv // NS)
                assert v[kv % NB] == (i, j, "raw")
                v[kv % NB] = (i, j, "clean")
                bar(("v_ready", st)).arrive()
                kv += 1
                yield

    def commit(name):
        products.append(("commit", bar(name)))

    def issuer():
        kv, qw, pw = 0, [0, 0], [0, 0]

        def qk(x, i, g, j, last):
            st = g % NS
            yield from wait(bar(("k_full", st)), g // NS)

            def run():
                if k[g % NB] != (i, j) or q[x] != i:
                    raise ProtocolError(f"S of {(i, j)} from K {k[g % NB]} and Q {q[x]}")
                if S[x] is not None and read[x] < THREADS:
                    raise ProtocolError("S overwritten before every thread has read it")
                if P[x] is not None:
                    raise ProtocolError("S written over a P that is still to be read")
                S[x], read[x] = (i, j), 0
            products.append(("mma", run))
            commit(("s_full", x))
            if one:
                commit(("k_empty", st))
            if last:
                commit(("q_empty", x))

        def pv(x, i, j, buffer, first):
            def run():
                if P[x] != (i, j):
                    raise ProtocolError(f"P {P[x]} for {(i, j)}")
                if v[buffer] != (i, j, "clean"):
                    raise ProtocolError(f"V {v[buffer]} for {(i, j)}")
                O[x] = [(i, j)] if first else O[x] + [(i, j)]
                P[x] = S[x] = None
            return run

        for i, (j0, j1, tiles) in enumerate(pieces):
            for x in range(2):
                if tiles[x][0] < tiles[x][1]:
                    yield from wait(bar(("q_full", x)), qw[x])
                    qw[x] += 1
            for j in range(j0, j1):
                st = kv % NS
                for x in range(2):
                    a, e = tiles[x]
                    if j == a < e:
                        yield from qk(x, i, kv, j, j == e - 1)
                yield from wait(bar(("v_ready", st)), kv // NS)
                if not any(a <= j < e for a, e in tiles):
                    if mistake != "unused K":
                        yield from wait(bar(("k_full", st)), kv // NS)
                    bar(("kv_empty", st)).arrive()
                    if one:
                        bar(("k_empty", st)).arrive()
                    kv += 1
                    continue
                for x in range(2):
                    a, e = tiles[x]
                    if not a <= j < e:
                        continue
                    if mistake != "early PV":
                        yield from wait(bar(("p_half", x)), pw[x])
                        yield from wait(bar(("p_full", x)), pw[x])
                    pw[x] += 1

                    products.append(("mma", pv(x, i, j, kv % NB, j == a)))
                    if j == e - 1:
                        commit(("o_full", x))
                    if one:
                        commit(("kv_empty", st))
                    if j == e - 1:
                        pass
                    elif mistake == "no QK":
                        pass
                    else:
                        yield from qk(x, i, kv + 1, j + 1, j + 1 == e - 1)
                if not one:
                    commit(("kv_empty", st))
                kv += 1
                yield

    def softmax(x, t):
        it, oc = 0, 0
        for i, (j0, j1, tiles) in enumerate(pieces):
            a, e = tiles[x]
            if a >= e:
                continue
            for j in range(a, e):
                yield from wait(bar(("s_full", x)), it)
                if S[x] != (i, j):
                    raise ProtocolError(f"thread of tile {x} reads S {S[x]} for {(i, j)}")
                yield
                read[x] += 1
                yield
                bar(("p_half", x)).arrive()
                yield
                if bar(("p_full", x)).arrivals == THREADS - 1:
                    P[x] = (i, j)          # complete with the last thread's half
                bar(("p_full", x)).arrive()
                it += 1
            yield from wait(bar(("o_full", x)), oc)
            oc += 1
            if O[x] != [(i, j) for j in range(a, e)]:
                raise ProtocolError(f"output of tile {x}, piece {i}: {O[x]}")
            if t == 0:
                results.append((x, i))
            yield

    agents = [producer(), cleaner(), issuer()] + [softmax(x, t) for x in range(2) for t in range(THREADS)]
    idle = 0
    slow = rng.choice((0.02, 0.1, 0.3)), rng.choice((0.02, 0.1, 0.3))      # how fast loads and products end
    while agents or loads or products:
        before = sum(b.arrivals + b.done * 1000 for b in bars.values()) + len(loads) + len(products) + len(agents)
        pick = rng.random()
        if loads and pick < slow[0]:
            loads.pop(rng.randrange(len(loads)))()
        elif products and pick < slow[0] + slow[1]:
            kind, what = products.pop(0)
            what() if kind == "mma" else what.arrive()
        elif agents:
            agent = rng.choice(agents)
            try:
                next(agent)
            except StopIteration:
                agents.remove(agent)
        after = sum(b.arrivals + b.done * 1000 for b in bars.values()) + len(loads) + len(products) + len(agents)
        idle = idle + 1 if before == after else 0
        if idle > 5000:
            raise ProtocolError("deadlock")
    assert sorted(results) == sorted((x, i) for i, p in enumerate(pieces) for x in range(2) if p[2][x][0] < p[2][x][1])


@pytest.mark.parametrize("one", [False, True])
@pytest.mark.parametrize("seed", range(60))
def test_protocol(seed, one):
    rng = random.Random(seed)
    simulate(random_pieces(rng, rng.randrange(1, 9), one), rng, one=one)


@pytest.mark.parametrize("mistake,one", [("early PV", False), ("no QK", False), ("unused K", False), ("early V", True),
                                         ("early PV", True), ("no QK", True)])
def test_planted_mistakes_are_found(mistake, one):
    found = 0
    for seed in range(60):
        rng = random.Random(1000 + seed)
        pieces = random_pieces(rng, 8, one)
        try:
            simulate(pieces, rng, mistake, one)
        except AssertionError:
            found += 1
    assert found > 0
