"""Split attention over block scales with bf16 partial outputs, held to what the rounding of the partial outputs
can do to each output (and not to the largest value of the cache)."""
import numpy as np
import pytest

import long_context_split_gb300 as skv
from tests.block_util import BlockBatch, check_attention

pytestmark = pytest.mark.gpu


def reference(batch):
    """``batch.attention()`` with 2^-8 A more in the bound, A = sum p |v| per element: a split's output is rounded by at
    most 2^-8 of itself, which is at most its own sum p |v|, and the splits' weights sum to 1."""
    out, lse, bound, lse_bound = batch.attention()
    q = batch.q.double().numpy()
    for b, (L, t) in enumerate(zip(batch.seq, batch.new)):
        kk, vv = batch.values(batch.k, batch.ks, b, 0, L), np.abs(batch.values(batch.v, batch.vs, b, 0, L))
        for i in range(t):
            n, r = L - t + i + 1, int(batch.qo[b]) + i
            for h in range(batch.heads * batch.group):
                s = kk[:n, h // batch.group] @ q[r, h] * batch.scale
                p = np.exp(s - s.max())
                bound[r, h] += 2.0 ** -8 * (p / p.sum()) @ vv[:n, h // batch.group]
    return out, lse, bound, lse_bound


CASES = [([300, 64, 1000], [1, 1, 3], 4, dict(uniform_splits=4)), ([300, 64, 1000], [1, 1, 3], 4, dict(uniform_splits=5, interleave=1)),
         ([700, 1300], [7, 8], 8, dict(uniform_splits=3)), ([1500, 300, 2100], [40, 1, 17], 8, dict(uniform_splits=4))]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_bf16_partials(case):
    seq, new, group, params = CASES[case]
    batch = BlockBatch(seq, new, heads=2, group=group, page=64, block=32, seed=90 + case, spread=2.0, poison=True)
    att = skv.SplitKVAttention(batch.problem, skv.plan_params("uniform", partial_dtype=skv.BF16, **params))
    ref = reference(batch)
    # the bound tells outputs from others: from 0, and from those of another head
    o, _, bound, _ = ref
    assert (np.abs(o) > bound).mean() > 0.9
    assert (np.abs(o - np.roll(o, 1, axis=1)) > bound).mean() > 0.9
    check_attention(batch, *att.decode(), ref=ref)
    check_attention(batch, *att.two_stage(), ref=ref)
    att.check_device_error()
