"""assign_pages in steps without new tokens, and slots under row bounds that are wrong."""
import numpy as np
import pytest

from tests.test_gpu_pages import Device, Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seq", [[0, 16, 0, 30], [0, 0, 0, 0], [40, 16, 64, 30]])
def test_a_step_without_new_tokens(seq):
    """An empty slots tensor: pages are given back (and taken) all the same, and nothing is reported."""
    pool = Pool([3, 1, 4, 2], 6, 8, 16, seed=10)
    dev = Device(pool)
    pool.step(seq)
    got, reported = dev.step(seq, [0, 0, 0, 0, 0], 0)
    assert got.size == 0 and not reported
    assert dev.held.tolist() == pool.held and int(dev.count) == pool.count
    assert np.array_equal(dev.table.cpu().numpy(), pool.table) and np.array_equal(dev.free.cpu().numpy(), pool.free)


def allowed(pool, seq, qo, num_slots):
    """The values that each slot may have: of a row that one request claims, its slot or -1 where the request's bounds are
    refused; of a row that several claim (bounds that decrease in between), the value of any of them; the rows
    behind qo_indptr[batch] as they were."""
    may = [set() for _ in range(num_slots)]
    for b, n in enumerate(seq):
        lo, hi = int(qo[b]), int(qo[b + 1])
        ok = 0 <= lo <= hi <= num_slots and hi - lo <= n
        for r in range(max(lo, 0), min(hi, num_slots)):
            pos = n - (hi - r)
            may[r].add(int(pool.table[b, pos // pool.page]) * pool.page + pos % pool.page if ok else -1)
    end = max(0, min(num_slots, int(qo[-1])))
    return [m or {-1} for m in may[:end]] + [{-5}] * (num_slots - end)


BOUNDS = [[0, 4, 2, 6], [0, 8, 3, 9], [0, 3, 6, 40], [-2, 3, 6, 8], [2, 5, 5, 9], [0, 9, 9, 4], [0, 3, 6, -1], [0, 1, 32, 33], [0, 0, 0, 10]]


@pytest.mark.parametrize("num_slots", [10, 34, 5000])
@pytest.mark.parametrize("bounds", range(len(BOUNDS)))
def test_slots_of_wrong_bounds(bounds, num_slots):
    """Few slots (within the call's first launch) and many (in its second)."""
    qo = BOUNDS[bounds]
    pool = Pool([2, 2, 2], 5, 8, 16, seed=11)
    dev = Device(pool)
    seq = [30, 30, 30]
    got, reported = dev.step(seq, qo, num_slots)
    pool.step(seq, qo, num_slots)
    refused = [not (0 <= qo[b] <= qo[b + 1] <= num_slots and qo[b + 1] - qo[b] <= 30) for b in range(3)]
    assert reported == any(refused)
    may = allowed(pool, seq, qo, num_slots)
    assert len(got) == len(may)
    for r, (g, m) in enumerate(zip(got, may)):
        assert int(g) in m, (r, int(g), m)


@pytest.mark.parametrize("num_slots", [4096, 6000])
def test_one_request_of_wrong_bounds_among_many(num_slots):
    """The other requests' slots are right; the refused one's are all -1."""
    batch, page = 300, 16
    pool = Pool([2] * batch, 5, 8, page, seed=12)
    dev = Device(pool)
    seq = [20] * batch
    seq[100] = 9                                            # 10 new tokens of 9
    qo = np.arange(batch + 1, dtype=np.int32) * 10
    got, reported = dev.step(seq, qo, num_slots)
    want, bad = pool.step(seq, qo, num_slots)
    assert reported and bad
    assert np.array_equal(got, want) and (got[1000:1010] == -1).all() and (got[1010:3000] >= 0).all() and (got[3000:] == -5).all()
