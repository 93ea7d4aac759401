"""Expanded latent attention over histories whose keys and values of all heads are not held at once: groups of
heads, expanded and attended one after the other in the same workspace.  Bounds as in test_gpu_latent."""
import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv
from tests.test_gpu_latent import SCALE, Case

IMAGES = 8 << 30            # bytes of keys and values that a workspace holds at most (two heads at least)


def _plan(seq, new, heads):
    """A plan from lengths alone (host only)."""
    qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    table = torch.zeros(1, dtype=torch.int32).expand(len(seq), -(-max(seq) // 64))
    return skv.LatentPlan(skv.AttentionProblem(
        q=torch.zeros(0, dtype=torch.bfloat16), k_cache=torch.zeros(1, 64, 576, dtype=torch.bfloat16), v_cache=None,
        page_table=table.contiguous(), seq_lens=t(len(seq)), qo_indptr=t(len(seq) + 1), num_q_heads=heads, num_kv_heads=1,
        head_dim_qk=576, head_dim_v=512, page_size=64, scale=SCALE, kind="mla", seq_lens_host=seq, qo_indptr_host=qo))


@pytest.mark.parametrize("seq,new,heads", [
    ([1 << 20] * 4, [512] * 4, 128),            # four requests of a million tokens
    ([1 << 20], [2048], 128), ([1 << 17] * 2, [1, 1], 128), ([1 << 20] * 20, [1] * 20, 16), ([3 << 20], [7], 3), ([3 << 22], [7], 1),
])
def test_the_workspace_is_bounded(seq, new, heads):
    p = _plan(seq, new, heads)
    units = sum(-(-n // 64) for n in seq)
    images = max(IMAGES, 2 * units * 32768)
    tokens, total = 64 * units, sum(new)
    states = int((p.splits() * np.array(new)).sum()) * heads * (512 + 4 + 4)
    small = 40 * p.num_tasks + 48 * len(seq) + 8 * units + images // 4096 + (1 << 16) + 4 * total * heads
    assert p.workspace_bytes <= images + 1152 * tokens + states + small


def test_groups_are_used_only_where_they_are_needed():
    one, two = _plan([1 << 17], [1], 128), _plan([(1 << 17) + 64], [1], 128)
    assert one.workspace_bytes > IMAGES         # 8 GiB of keys and values exactly: all heads at once
    assert two.workspace_bytes < IMAGES // 2 + (256 << 20)      # a unit more: two groups of 64 heads
    for p in (one, two):
        assert p.num_tasks == 128 * int(p.splits()[0])
    odd = _plan([1 << 20] * 2, [300] * 2, 11)   # groups of 4, 4 and 3 heads
    assert odd.num_tasks == 2 * 2 * int(odd.splits()[0]) * 11


def test_a_batch_of_few_tasks_is_not_split_into_more_than_one_round():
    """Tasks run one per SM: a task more than SMs would leave a second round nearly empty."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152
    # (lengths, tasks of a group before splits, groups)
    for seq, new, heads, tasks, groups in (([1 << 20], [1], 16, 16, 1), ([1 << 16] * 3, [1, 200, 40], 7, 21, 1),
                                           ([1 << 20], [512], 128, 32, 8), ([1 << 17], [1], 100, 100, 1),
                                           ([50000, 30000], [300, 1], 32, 96, 1)):
        p = _plan(seq, new, heads)
        assert (p.splits() == sms // tasks).all()
        assert p.num_tasks <= groups * sms


@pytest.mark.gpu
@pytest.mark.parametrize("seq,new,heads,fp8", [
    ([140000, 200, 65], [70, 200, 65], 128, False),      # two heads per task in the long request's groups
    ([140000], [2], 128, True),                          # split histories
    ([300000, 64, 5000], [130, 1, 300], 63, False),      # an odd last group
])
def test_groups_of_heads(seq, new, heads, fp8):
    c = Case(seq, new, heads, 64, fp8, seed=41)
    att, out, lse = c.run("expanded")
    _, again, _ = c.run("expanded", lse=False)
    assert torch.equal(out, again)
    keep = [0, 1, 63, 64, 127] if heads == 128 else [0, 31, 32, 62]
    c.w, c.q, c.heads = c.w[keep], c.q[:, keep], len(keep)
    c.check("expanded", out[:, keep], lse[:, keep])
