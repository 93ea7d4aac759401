"""Attention over block scales at the ends of their range, and with scores so far apart that weights leave
float32's range: every output finite and within ``block_util``'s bound."""
import math

import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv
from tests.block_util import VALUES, BlockBatch, check_attention, encode

pytestmark = pytest.mark.gpu

P100, M100, ZEROS = 2.0 ** 100, 2.0 ** -100, 2.0 ** -126


class RangeBatch(BlockBatch):
    def attention(self, codes=None):
        """``block_util``'s, with 2^-133 more: an output below the normal numbers is rounded by half of bf16's step there,
        2^-134, and each float32 product behind it by 2^-150 (fewer than 2^16 of them here)."""
        out, lse, bound, lse_bound = super().attention(codes)
        return out, lse, bound + 2.0 ** -133, lse_bound


class FarBatch(RangeBatch):
    """Block j of 16 tokens has blocks[j % len(blocks)] = (score, value scale): queries of ones and keys of plus or minus
    one under a key scale that makes every score of the block `score` binary orders.  What a float32
    weight cannot hold counts for nothing: a key more than 126 binary orders below its row's largest may be lost, so that
    its share is added to the bound (one order more, for the exponent's own rounding)."""

    def __init__(self, seq, new, blocks, seed=0, page=64, **kw):
        super().__init__(seq, new, page=page, block=16, seed=seed, **kw)
        self.q.fill_(1.0)
        self.q_dev.copy_(self.q)
        one = int(encode(np.array([1.0]))[0])
        for b, n in enumerate(self.seq):
            for j in range(-(-n // 16)):
                score, scale = blocks[j % len(blocks)]
                p, t = int(self.table[b, j * 16 // page]), j * 16 % page // 16
                self.k[p, :, 16 * t:16 * t + 16] = one | (0x80 if score < 0 else 0)
                self.ks[p, :, t] = abs(score) * math.log(2.0) / (self.dim * self.scale)
                self.vs[p, :, t] = scale
        for dev, host in ((self.k_dev, self.k), (self.ks_dev, self.ks), (self.vs_dev, self.vs)):
            dev.copy_(torch.from_numpy(host))

    def attention(self, codes=None):
        out, lse, bound, lse_bound = super().attention(codes)
        for b, (L, t) in enumerate(zip(self.seq, self.new)):
            kk, vv = self.values(self.k, self.ks, b, 0, L), np.abs(self.values(self.v, self.vs, b, 0, L))
            for i in range(t):
                n, r = L - t + i + 1, int(self.qo[b]) + i
                for h in range(self.heads * self.group):
                    s = kk[:n, h // self.group].sum(1) * self.scale
                    p = np.exp(s - s.max())
                    bound[r, h] += np.where(p < 2.0 ** -125, p, 0.0) @ vv[:n, h // self.group] / p.sum()
        return out, lse, bound, lse_bound


# a dominant block with a value scale far below that of a block whose weights leave float32's range
FAR = [[(0, M100), (-g, P100)] for g in (100, 127, 130, 160, 220)] + [[(0, 0.0), (-g, 4.0)] for g in (100, 140, 200)] + \
      [[(0, ZEROS), (-g, 8.0)] for g in (100, 128, 180)] + [[(0, 2.0 ** -70), (-130, 2.0 ** 60)], [(0, ZEROS), (-150, 2.0 ** 120)]]
# requests of one new token; blocks of 16 to 64 query rows per KV head; more rows, on the chunk tiles
FORMS = [("one", [200, 64, 17], [1, 1, 1], 4), ("block", [200, 40], [16, 5], 4), ("tiles", [300, 200], [40, 33], 8)]


@pytest.mark.parametrize("form,seq,new,group", FORMS, ids=[f[0] for f in FORMS])
@pytest.mark.parametrize("blocks", range(len(FAR)))
def test_scores_and_scales_far_apart(blocks, form, seq, new, group):
    batch = FarBatch(seq, new, FAR[blocks], heads=2, group=group, seed=blocks)
    att = skv.SplitKVAttention(batch.problem)
    assert att.plan.kernel_path == 1 and (att.plan.num_chunk_tasks > 0) == (form == "tiles")
    check_attention(batch, *att.decode())
    att.check_device_error()


@pytest.mark.parametrize("blocks", range(len(FAR)))
def test_scores_and_scales_far_apart_on_the_float32_path(blocks):
    batch = FarBatch([100, 40], [1, 20], FAR[blocks], heads=2, group=2, dim=64, seed=blocks)
    att = skv.SplitKVAttention(batch.problem)
    assert att.plan.kernel_path == 0
    check_attention(batch, *att.decode())


@pytest.mark.parametrize("scales", [(0.0, 16.0), (ZEROS, 16.0), (M100, P100), (0.0, 2.0 ** 110)])
@pytest.mark.parametrize("group,seq,new,first", [(4, 24, 15, 16), (2, 40, 31, 16), (8, 40, 33, 16), (8, 120, 70, 64)])
def test_later_blocks_that_a_row_may_not_see(group, seq, new, first, scales):
    """The first rows see blocks of the first scale alone (0: they are 0), whatever the scale of the new tokens behind them."""
    blocks = [(0, scales[0])] * (first // 16) + [(0, scales[1])] * 8
    batch = FarBatch([seq], [new], blocks, heads=2, group=group, seed=group)
    att = skv.SplitKVAttention(batch.problem)
    assert (att.plan.num_chunk_tasks > 0) == (group * new > 64)
    out, lse = att.decode()
    check_attention(batch, out, lse)
    if scales[0] == 0.0:
        assert (out[:first - (seq - new)] == 0).all()


@pytest.mark.parametrize("form,seq,new,group", FORMS, ids=[f[0] for f in FORMS])
@pytest.mark.parametrize("reach", [20.0, 90.0, 200.0])
@pytest.mark.parametrize("seed", range(3))
def test_random_scores_and_scales(seed, reach, form, seq, new, group):
    """Scores and value scales of every block drawn from ranges wider and narrower than float32's, some scales 0."""
    g = np.random.default_rng(seed)
    blocks = [(float(g.uniform(-reach, reach)), 0.0 if g.random() < 0.2 else 2.0 ** float(g.uniform(max(-126.0, -reach), min(100.0, reach))))
              for _ in range(13)]
    batch = FarBatch(seq, new, blocks, heads=2, group=group, seed=50 + seed)
    for params in (None, dict(uniform_splits=3)):
        att = skv.SplitKVAttention(batch.problem, skv.plan_params("uniform", **params) if params else None)
        check_attention(batch, *att.decode())
        att.check_device_error()


# the largest score at a block of scale 0, after blocks of small scales and beside one that decides the output
LATE = [[(0, M100)] * 4 + [(30, 0.0), (5, M100), (0, 0.0), (0, 0.0)], [(0, M100)] * 4 + [(60, 0.0), (7, M100), (0, 0.0), (-9, M100)],
        [(0, ZEROS)] * 4 + [(9, 0.0), (6, ZEROS), (0, 0.0), (2, ZEROS)]]


@pytest.mark.parametrize("form,seq,new,group", FORMS, ids=[f[0] for f in FORMS])
@pytest.mark.parametrize("blocks", range(len(LATE)))
def test_the_largest_score_under_a_scale_of_zero(blocks, form, seq, new, group):
    batch = FarBatch(seq, new, LATE[blocks], heads=2, group=group, seed=20 + blocks)
    check_attention(batch, *skv.SplitKVAttention(batch.problem).decode())


@pytest.mark.parametrize("form,seq,new,group", FORMS + [("long", [4000], [40], 8)], ids=[f[0] for f in FORMS] + ["long"])
@pytest.mark.parametrize("scale", [ZEROS, 2.0 ** -110, 2.0 ** 110])
def test_scales_at_the_ends_of_the_range(scale, form, seq, new, group):
    batch = FarBatch(seq, new, [(0, scale), (-1, scale), (2, scale / 2 if scale > 1 else 2 * scale)], heads=2, group=group, seed=30)
    check_attention(batch, *skv.SplitKVAttention(batch.problem).decode())


def test_half_a_million_tokens_of_the_smallest_scale():
    """On the chunk tiles: the sum of weights (after a first unit of scores 7.5 binary orders lower, which they do not
    rescale for) times 2^126 is far beyond float32's normal numbers.  Every query is alike, so that a token's rows are."""
    n, new, group, page = 516224, 5, 16, 64
    g = torch.Generator(device="cuda").manual_seed(31)
    v = torch.randint(0x20, 0x70, (n // page, 1, page, 128), generator=g, device="cuda", dtype=torch.uint8)
    ks = torch.full((n // page, 1, 4), 7.5 * math.log(2.0) / math.sqrt(128.0), device="cuda")
    ks[0] = 0.0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    problem = skv.AttentionProblem(
        q=torch.ones(new, group, 128, dtype=torch.bfloat16, device="cuda"), k_cache=torch.full_like(v, 0x38), v_cache=v,
        page_table=torch.arange(n // page, dtype=torch.int32, device="cuda")[None].contiguous(), seq_lens=i32([n]), qo_indptr=i32([0, new]),
        num_q_heads=group, num_kv_heads=1, head_dim_qk=128, head_dim_v=128, page_size=page, scale=1.0 / math.sqrt(128.0),
        seq_lens_host=[n], qo_indptr_host=[0, new], k_scale=ks, v_scale=torch.full_like(ks, ZEROS))
    att = skv.SplitKVAttention(problem, skv.plan_params("uniform", uniform_splits=1))
    assert att.plan.num_chunk_tasks > 0
    out, _ = att.decode()
    x = torch.from_numpy(VALUES).cuda()[v.view(n, 128).long()]                     # (in units of the scale)
    w = torch.exp2(torch.where(torch.arange(n, device="cuda") < 64, -7.5, 0.0).double())
    for i in range(new):
        m = n - new + i + 1
        want = (w[:m] @ x[:m]) / w[:m].sum()
        # bf16's rounding, f16's of the weights and 2^-11 for the scores' and the float32 sums' errors (all values positive)
        assert ((out[i].double() * 2.0 ** 126 - want).abs() <= want * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11)).all()


@pytest.mark.parametrize("group,new", [(4, 9), (4, 16), (8, 40)])
def test_attention_over_what_the_append_writes(group, new):
    """Rows of zeros (a scale of 2^-126), of the smallest and of large finite numbers beside ordinary ones, appended and attended over."""
    batch = RangeBatch([90, 16 + new, new, new], [new] * 4, heads=2, group=group, page=64, block=16, seed=40)
    g = torch.Generator().manual_seed(41)
    k, v = (torch.randn(4 * new, 2, 128, generator=g) for _ in range(2))
    k *= 0.05
    v[:new // 2] = 0.0
    v[new // 2:new] *= 2.0 ** 100
    v[2 * new:2 * new + 16] = 0.0                  # a block of zeros, the next one (if any) of large values
    v[2 * new + 16:3 * new] *= 2.0 ** 40
    v[3 * new:] *= 2.0 ** -120
    k, v = k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda()
    skv.kv_append(batch.problem, k, v)
    batch.k, batch.ks, batch.v, batch.vs = (t.cpu().numpy() for t in (batch.k_dev, batch.ks_dev, batch.v_dev, batch.vs_dev))
    assert (batch.vs == ZEROS).any() and batch.vs.max() > 2.0 ** 90
    check_attention(batch, *skv.SplitKVAttention(batch.problem).decode())
