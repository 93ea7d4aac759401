"""The paired tiles' rings of keys and values, as a model of their protocol: two producers, the two tiles'
issuers and softmaxes, barriers waited on by parity (a wait for parity p is over unless the current
phase has parity p, as in hardware), copies that land after random times.

A task is a pair of blocks; the shorter tile passes by units that only the other attends.  Whatever
the copies' times, a tile may read a slot only once its own unit has landed there."""
import heapq
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_split_gb300", "csrc",
                      "pair_kernel.cu")


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def step(self):
        assert self.pending >= 0
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self):
        self.pending -= 1
        self.step()

    def expect(self):
        self.tx += 1
        self.pending -= 1

    def land(self):
        self.tx -= 1
        self.step()

    def over(self, parity):
        return (self.phase & 1) != (parity & 1)


def simulate(tasks, nk, nv, nb, rng, slowest):
    """tasks: (units of tile 0, units of tile 1); nk, nv: key and value slots; nb: barriers of the value loads."""
    events, now, seq = [], [0], [0]

    def at(dt, f):
        seq[0] += 1
        heapq.heappush(events, (now[0] + dt, seq[0], f))

    def latency():
        return rng.choice([rng.randint(50, 300), rng.randint(50, slowest)])

    q_full, q_empty = Bar(1), Bar(2)
    k_full, k_empty = [Bar(1) for _ in range(nk)], [Bar(2) for _ in range(nk)]
    v_full, v_empty = [Bar(1) for _ in range(nb)], [Bar(2) for _ in range(nv)]
    s_full, p_full = [[Bar(1), Bar(1)] for _ in range(2)], [[Bar(1), Bar(1)] for _ in range(2)]
    o_full, o_empty = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    keys, values = [None] * nk, [None] * nv
    pipe = [0]

    def product(duration, effect):                       # products complete in issue order
        pipe[0] = max(now[0], pipe[0]) + duration
        at(pipe[0] - now[0], effect)

    def load(ring, full, empty, item, name):
        s, b = item % len(ring), item % len(full)
        yield lambda: empty[s].over(item // len(ring) + 1)
        full[b].expect()
        ring[s] = None

        def landed():
            ring[s] = name
            full[b].land()
        at(latency(), landed)

    def key_producer():
        item = 0
        for n, task in enumerate(tasks):
            yield lambda: q_empty.over(n + 1)
            q_full.expect()
            at(latency(), q_full.land)
            for u in range(max(task)):
                yield from load(keys, k_full, k_empty, item, (n, u))
                item += 1

    def value_producer():
        item = 0
        for n, task in enumerate(tasks):
            for u in range(max(task)):
                yield from load(values, v_full, v_empty, item, (n, u))
                item += 1

    def issuer(t):
        item = done = blocks = 0
        for n, task in enumerate(tasks):
            nu, other, item0 = task[t], task[1 - t], item
            item += max(task)
            yield lambda: q_full.over(n)
            if nu == 0:
                q_empty.arrive()
                continue

            def score(u):
                s = (item0 + u) % nk
                yield lambda: k_full[s].over((item0 + u) // nk)
                assert keys[s] == (n, u), "keys read before they landed"

                def end(full=s_full[t][(done + u) & 1], last=u == nu - 1, both=u >= other):
                    full.arrive()
                    if last:
                        q_empty.arrive()
                    for _ in range(2 if both else 1):
                        k_empty[s].arrive()
                product(50, end)

            def output(u):
                if u == 0:
                    yield lambda: o_empty[t].over(blocks + 1)
                yield lambda: p_full[t][(done + u) & 1].over((done + u) >> 1)
                s = (item0 + u) % nv

                def end(both=u >= other):
                    for _ in range(2 if both else 1):
                        v_empty[s].arrive()
                product(30, end)

            yield from score(0)
            for u in range(nu):
                if u + 1 < nu:
                    yield from score(u + 1)
                yield from output(u)
            product(0, o_full[t].arrive)
            done += nu
            blocks += 1

    def softmax(t):
        item = done = blocks = 0
        for n, task in enumerate(tasks):
            item0 = item
            item += max(task)
            for u in range(task[t]):
                yield lambda: s_full[t][done & 1].over(done >> 1)
                until = now[0] + rng.randint(20, 300)
                at(until - now[0], lambda: None)
                yield lambda: now[0] >= until
                i = item0 + u
                yield lambda: v_full[i % nb].over(i // nb)
                assert values[i % nv] == (n, u), "values read before they landed"
                p_full[t][done & 1].arrive()
                done += 1
            if task[t]:
                yield lambda: o_full[t].over(blocks)
                blocks += 1
                o_empty[t].arrive()

    agents = [key_producer(), value_producer(), issuer(0), issuer(1), softmax(0), softmax(1)]
    waits = [None] * len(agents)
    live = set(range(len(agents)))
    while live:
        moved = True
        while moved:
            moved = False
            for a in rng.sample(sorted(live), len(live)):
                if waits[a] is None or waits[a]():
                    moved = True
                    try:
                        waits[a] = next(agents[a])
                    except StopIteration:
                        live.discard(a)
        if live:
            assert events, "every agent waits"
            now[0], _, f = heapq.heappop(events)
            f()


def value_barriers(nv):
    with open(SOURCE) as f:
        found = re.search(r"v_full\[([^\]]+)\], v_empty\[NV\];", f.read())
    return eval(found.group(1), {"NV": nv})      # the ring's own expression


def task_list(rng):
    tasks = []
    for _ in range(rng.randint(2, 7)):
        long = rng.randint(1, 14)
        short = rng.choice([0, rng.randint(0, long), rng.randint(0, long), max(0, long - 1), long])
        tasks.append((long, short) if rng.random() < 0.5 else (short, long))
    return tasks


@pytest.mark.parametrize("nk,nv", [(3, 2), (6, 6), (2, 2), (4, 3)])     # head dims 128 and 64, and smaller rings
def test_a_tile_reads_only_units_that_have_landed(nk, nv):
    for seed in range(400):
        rng = random.Random(seed)
        simulate(task_list(rng), nk, nv, value_barriers(nv), rng, rng.choice([300, 3000, 20000]))
