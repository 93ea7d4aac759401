"""assign_pages against a plain restatement, request by request; all whole numbers."""
import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv

pytestmark = pytest.mark.gpu


class Pool:
    def __init__(self, held, spare, max_pages, page, seed=0, capacity=None):
        g = np.random.default_rng(seed)
        total = sum(held) + spare
        perm = g.permutation(total).astype(np.int32)
        self.page, self.max_pages = page, max_pages
        self.table = np.full((len(held), max_pages), -7, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.free = np.full(capacity or total, -9, np.int32)
        self.free[:spare] = perm[at:]
        self.count, self.held = spare, list(held)

    def step(self, seq, qo=None, num_slots=0):
        """The state after the call, its slots, and whether something is reported."""
        bad, P, cap = False, self.page, len(self.free)
        need = [-(-max(0, n) // P) for n in seq]
        bad |= any(n < 0 for n in seq)
        back = []
        for b, n in enumerate(need):
            if n < self.held[b] and n <= self.max_pages:
                back += list(self.table[b, n:self.held[b]])
        if self.count + len(back) > cap:
            bad, back = True, back[:cap - self.count]
        self.free[self.count:self.count + len(back)] = back
        avail = self.count + len(back)
        at, asked = avail, 0
        held = list(self.held)
        for b, n in enumerate(need):
            if n > self.max_pages:
                bad = True
                continue
            if n > self.held[b]:
                asked += n - self.held[b]
                if asked > avail:
                    bad = True
                    continue
                for j in range(self.held[b], n):
                    at -= 1
                    self.table[b, j] = self.free[at]
            held[b] = n
        self.count, self.held = at, held
        slots = np.full(num_slots, -5, np.int64)
        if qo is not None:
            for b, n in enumerate(seq):
                lo, hi = int(qo[b]), int(qo[b + 1])
                if not (0 <= lo <= hi <= num_slots) or hi - lo > max(0, n):
                    bad = True
                    slots[max(lo, 0):min(hi, num_slots)] = -1
                    continue
                for r in range(lo, hi):
                    pos = n - (hi - r)
                    slots[r] = self.table[b, pos // P] * P + pos % P if pos // P < held[b] else -1
        return slots, bad


class Device:
    def __init__(self, pool):
        to = lambda x: torch.from_numpy(np.array(x, np.int32)).cuda()  # noqa: E731
        self.table, self.free, self.held, self.count = to(pool.table), to(pool.free), to(pool.held), to([pool.count])
        self.page, self.err = pool.page, torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, seq, qo=None, num_slots=0, **over):
        slots = None if qo is None else torch.full((num_slots,), -5, dtype=torch.int64, device="cuda")
        i32 = lambda v: torch.tensor(np.array(v), dtype=torch.int32, device="cuda")  # noqa: E731
        skv.assign_pages(self.table, self.held, i32(seq), self.free, self.count, page_size=self.page,
                         qo_indptr=None if qo is None else i32(qo), slots=slots, dev_error_word=self.err, **over)
        st, _ = skv.read_device_error(self.err, clear=True)
        return None if slots is None else slots.cpu().numpy(), st == skv.ERR_DEVICE_CHECK


def compare(pool, dev, seq, new, extra=0):
    qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(qo[-1]) + extra
    want, bad = pool.step(seq, qo, n)
    got, reported = dev.step(seq, qo, n)
    assert np.array_equal(dev.held.cpu().numpy(), pool.held)
    assert int(dev.count) == pool.count
    assert np.array_equal(dev.table.cpu().numpy(), pool.table)
    assert np.array_equal(dev.free.cpu().numpy(), pool.free)
    assert np.array_equal(got, want)
    assert reported == bad
    return bad


@pytest.mark.parametrize("page", [1, 16, 64, 100])
@pytest.mark.parametrize("batch", [1, 3, 33, 1024, 1500])
def test_steps_of_a_serving_batch(batch, page):
    """Prompts, decode steps, ends and refused drafts, each step on what the last one left."""
    g = np.random.default_rng(batch * 7 + page)
    most = 20 * page
    pool = Pool([0] * batch, 25 * batch, 25, page, seed=batch)
    dev = Device(pool)
    seq = [0] * batch
    for step in range(6):
        new = []
        for b in range(batch):
            kind = g.integers(0, 6)
            if seq[b] == 0 or kind == 0:
                seq[b] = int(g.integers(1, most)) if step % 2 == 0 else 0        # a new prompt, or an end
                new.append(seq[b])
            elif kind == 1:
                seq[b] = max(1, seq[b] - int(g.integers(0, min(seq[b], 2 * page) + 1)))   # refused drafts
                new.append(min(seq[b], 1))
            else:
                n = int(g.integers(1, 5))
                seq[b] = min(most, seq[b] + n)
                new.append(min(n, seq[b]))
        compare(pool, dev, seq, new, extra=3)


def test_long_prompts_and_many_slots():
    pool = Pool([0, 3, 0, 50], 3000, 1100, 16, seed=1)
    compare(pool, Device(pool), [17000, 40, 16000, 0], [17000, 7, 9999, 0], extra=11)


def test_not_enough_pages():
    """Requests are served in order until the list runs out; later ones that need none are untouched."""
    pool = Pool([1, 2, 1, 4, 1], 3, 16, 16, seed=2)
    dev = Device(pool)
    assert compare(pool, dev, [3 * 16, 2 * 16, 3 * 16 + 1, 4 * 16, 2 * 16], [32, 1, 33, 1, 16])
    assert pool.held == [3, 2, 1, 4, 1]          # the fifth asks after the third, which did not fit
    # an end in the same call makes room
    assert not compare(pool, dev, [3 * 16, 2 * 16, 2 * 16, 0, 2 * 16], [1, 1, 16, 0, 16])


def test_refusals_are_reported():
    pool = Pool([1, 2, 1], 10, 4, 16, seed=3)
    dev = Device(pool)
    assert compare(pool, dev, [5 * 16, -3, 16], [1, 0, 2])       # more than a row holds; a negative length
    assert compare(pool, dev, [16, 16, 8], [1, 1, 9])            # more new tokens than the request has
    pool = Pool([4, 1], 2, 8, 16, seed=4, capacity=4)            # no room for all pages given back
    assert compare(pool, Device(pool), [0, 16], [0, 1])


def test_slots_of_wrong_bounds():
    pool = Pool([2, 2, 2], 5, 8, 16, seed=5)
    for qo in ([0, 4, 2, 6], [0, 3, 6, 40], [-2, 3, 6, 8]):
        dev = Device(pool)
        got, reported = dev.step([30, 30, 30], qo, 10)
        assert reported and got[:0].size == 0 and got.shape == (10,)


def test_held_and_count_out_of_range_are_clipped():
    pool = Pool([2, 2], 5, 8, 16, seed=6)
    dev = Device(pool)
    dev.held[0], dev.count[0] = 100, 10 ** 6
    _, reported = dev.step([8 * 16, 16])
    assert reported and int(dev.held[0]) == 8 and int(dev.held[1]) == 1


def test_separate_outputs_and_no_slots():
    pool = Pool([1, 4, 0], 9, 8, 16, seed=7)
    dev = Device(pool)
    held_out, count_out = torch.empty_like(dev.held), torch.empty_like(dev.count)
    before = dev.held.clone(), dev.count.clone()
    dev.step([40, 10, 70], held_out=held_out, free_count_out=count_out)
    pool.step([40, 10, 70])
    assert torch.equal(dev.held, before[0]) and torch.equal(dev.count, before[1])
    assert held_out.tolist() == pool.held and int(count_out) == pool.count
    assert np.array_equal(dev.table.cpu().numpy(), pool.table)


def test_replayed_graph_follows_lengths():
    pool = Pool([0] * 40, 600, 20, 16, seed=8)
    dev = Device(pool)
    seq = torch.zeros(40, dtype=torch.int32, device="cuda")
    qo = torch.arange(41, dtype=torch.int32, device="cuda")
    slots = torch.empty(40, dtype=torch.int64, device="cuda")

    def call():
        skv.assign_pages(dev.table, dev.held, seq, dev.free, dev.count, page_size=16, qo_indptr=qo, slots=slots,
                         dev_error_word=dev.err)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()                                    # (lengths of 0: nothing changes)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    pool.step([0] * 40, np.arange(41), 40)
    g = np.random.default_rng(9)
    for _ in range(5):
        lens = g.integers(1, 250, 40)
        seq.copy_(torch.from_numpy(lens.astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = pool.step(list(map(int, lens)), np.arange(41), 40)
        assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(dev.table.cpu().numpy(), pool.table)
        assert dev.held.tolist() == pool.held and int(dev.count) == pool.count
