"""assign_pages in steps without new tokens."""
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
