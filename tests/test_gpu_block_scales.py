"""The E4M3 cache with block scales: appended rows (every byte of the cache and every scale against a
restatement in float64), gathered rows, and attention over it against float64 with bounds
counted from the roundings (``block_util.attention``)."""
import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv
from tests.block_util import VALUES, BlockBatch, check_attention, encode

pytestmark = pytest.mark.gpu


def pow2_of(a):
    """The smallest power of two (from 2^-126) whose 448-fold is not below a."""
    if a == 0:
        return 2.0 ** -126
    e = int(np.floor(np.log2(a / 448.0))) - 1
    while 448.0 * 2.0 ** e < a:
        e += 1
    return 2.0 ** max(e, -126)


def quotient(x, s):
    """x / s as a float32 (float64's quotient of float32 numbers rounds to the same float32)."""
    with np.errstate(all="ignore"):
        return (x.astype(np.float32) / np.float32(s)).astype(np.float64)


def expected(batch, k_new, v_new):
    """(k, ks, v, vs) after an append, block by block."""
    res = []
    for codes, scales, new in ((batch.k, batch.ks, k_new), (batch.v, batch.vs, v_new)):
        codes, scales, x = codes.copy(), scales.copy(), new.float().cpu().numpy()
        S = batch.block
        for b, (L, t) in enumerate(zip(batch.seq, batch.new)):
            at = L - t
            while at < L:
                lo, end = at // S * S, min(at // S * S + S, L)
                page, slot = int(batch.table[b, at // batch.page]), at % batch.page
                j, first = slot // S, slot // S * S
                for h in range(batch.heads):
                    r = int(batch.qo[b]) + at - (L - t)
                    rows = x[r:r + end - at, h]
                    mag = np.abs(rows[np.isfinite(rows)]).astype(np.float64)
                    top = float(mag.max()) if mag.size else 0.0
                    was = float(scales[page, h, j])
                    if lo < at and was > 0 and top <= float(np.float32(448.0) * np.float32(was)):
                        now = was
                    else:
                        now = pow2_of(top)
                        if lo < at:
                            old = VALUES[codes[page, h, first:slot]].astype(np.float32) * np.float32(was)
                            codes[page, h, first:slot] = encode(quotient(old, now))
                        scales[page, h, j] = now
                    codes[page, h, slot:slot + end - at] = encode(quotient(rows, now))
                at = end
        res += [codes, scales]
    return res


def same_codes(a, b):
    nan = lambda c: np.where((c & 0x7F) == 0x7F, 0x7F, c)  # noqa: E731
    return np.array_equal(nan(a), nan(b))


def check_append(batch, k_new, v_new, err=None):
    want = expected(batch, k_new, v_new)
    skv.kv_append(batch.problem, k_new, v_new, dev_error_word=err)
    got = [t.cpu().numpy() for t in (batch.k_dev, batch.ks_dev, batch.v_dev, batch.vs_dev)]
    for name, g, w in zip(("k", "k scales", "v", "v scales"), got, want):
        if g.dtype == np.uint8:
            assert same_codes(g, w), name
        else:
            assert np.array_equal(g, w, equal_nan=True), name
    batch.k, batch.ks, batch.v, batch.vs = got


def rows_of(batch, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    T = int(batch.qo[-1])
    mk = lambda: (torch.randn(T, batch.heads, batch.dim, generator=g) * size *  # noqa: E731
                  torch.exp2(torch.randn(T, 1, 1, generator=g) * 2)).to(dtype).cuda()
    return mk(), mk()


LENGTHS = [([1], [1]), ([300], [300]), ([65, 1, 64, 200], [1, 1, 64, 137]), ([17, 33, 128, 129, 31], [2, 1, 1, 1, 15]),
           ([5, 700, 16], [0, 650, 16])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
def test_append_writes_codes_and_scales(lengths, page, block, dtype):
    seq, new = LENGTHS[lengths]
    for heads, dim in ((2, 128), (3, 64)):
        batch = BlockBatch(seq, new, heads=heads, dim=dim, page=page, block=block, seed=lengths)
        check_append(batch, *rows_of(batch, dtype, seed=lengths))


def test_append_token_by_token_into_one_block():
    """Scales grow with the tokens; each step starts from the cache that the last one left."""
    batch = BlockBatch([1], [1], heads=2, dim=128, page=64, block=64, seed=3)
    for n in range(1, 65):
        batch.seq, batch.new, batch.qo = [n], [1], np.array([0, 1], np.int32)
        batch.seq_dev.fill_(n)
        batch.problem = batch.make()
        check_append(batch, *rows_of(batch, torch.bfloat16, seed=n, size=2.0 ** (n % 7 - 3)))


def test_append_infinities_nan_zeros_and_subnormals():
    batch = BlockBatch([40, 20], [40, 3], heads=2, dim=64, page=64, block=16, seed=4)
    k, v = rows_of(batch, torch.float32, seed=5)
    k[0, 0, 3], k[1, 0, 5], k[2, 1, 0], k[17, 0, 0] = float("inf"), float("-inf"), float("nan"), 3.4e38
    k[32:40] = 0.0                                   # a block of zeros
    v[16:32] = 1e-42                                 # subnormal rows
    v[33, 0], v[41] = float("nan"), float("inf")     # (the second row of a block with older tokens: its scale stays)
    check_append(batch, k, v)


def test_append_older_scales_that_are_zero_or_nan():
    batch = BlockBatch([20, 20, 20], [1, 1, 1], heads=1, dim=64, page=64, block=64, seed=6)
    for b, s in enumerate((0.0, float("nan"), 2.0 ** -20)):
        batch.ks[batch.table[b, 0]] = s
    batch.ks_dev.copy_(torch.from_numpy(batch.ks))
    check_append(batch, *rows_of(batch, torch.bfloat16, seed=7))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_strided_and_odd_rows(dtype):
    seq, new = [70, 200, 9], [64, 3, 9]
    for heads, dim, block in ((2, 128, 16), (2, 128, 64), (1, 60, 16), (5, 6, 64)):
        batch = BlockBatch(seq, new, heads=heads, dim=dim, page=64, block=block, seed=8)
        T = int(batch.qo[-1])
        fused = torch.randn(T, 3 * heads, dim, device="cuda").to(dtype)
        check_append(batch, fused[:, heads:2 * heads], fused[:, 2 * heads:])
        batch = BlockBatch(seq, new, heads=heads, dim=dim, page=64, block=block, seed=9)
        wide = torch.randn(heads, T, dim + 1, device="cuda").to(dtype)          # head-major, odd rows
        check_append(batch, wide.transpose(0, 1)[..., :dim], wide.transpose(0, 1)[..., 1:])


def test_append_follows_lengths_on_the_device_and_leaves_other_rows():
    """The device's lengths and row bounds count: a request's rows moved by 5 tokens, and rows behind the
    device's last request left alone."""
    batch = BlockBatch([50, 60], [10, 20], heads=2, dim=64, page=64, block=16, seed=10)
    k, v = rows_of(batch, torch.bfloat16, seed=11)
    problem = batch.problem
    batch.seq, batch.new, batch.qo = [45, 60], [10, 12], np.array([0, 10, 22], np.int32)
    batch.seq_dev.copy_(torch.tensor(batch.seq, dtype=torch.int32))
    batch.qo_dev.copy_(torch.from_numpy(batch.qo))
    want = expected(batch, k, v)
    skv.kv_append(problem, k, v)
    assert same_codes(batch.k_dev.cpu().numpy(), want[0]) and same_codes(batch.v_dev.cpu().numpy(), want[2])
    assert np.array_equal(batch.ks_dev.cpu().numpy(), want[1])


def test_append_refuses_pages_out_of_range_and_reports():
    batch = BlockBatch([70, 40], [70, 40], heads=1, dim=64, page=64, block=64, seed=12)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    batch.table_dev[1, 0] = batch.num_pages
    k, v = rows_of(batch, torch.bfloat16, seed=13)
    other = batch.k[[p for p in range(batch.num_pages) if p not in batch.table[0]]].copy()
    skv.kv_append(batch.problem, k, v, dev_error_word=err)
    assert skv.read_device_error(err)[0] == skv.ERR_DEVICE_CHECK
    got = batch.k_dev.cpu().numpy()
    assert np.array_equal(got[[p for p in range(batch.num_pages) if p not in batch.table[0]]], other)
    batch.table[1, 0] = 0
    batch.seq, batch.new, batch.qo = [70], [70], np.array([0, 70], np.int32)
    want = expected(batch, k, v)
    for p in batch.table[0, :2]:
        assert same_codes(got[p], want[0][p])


@pytest.mark.parametrize("rows", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,block,dim", [(64, 16, 128), (128, 128, 128), (16, 16, 64), (64, 32, 60)])
def test_gather_returns_scaled_values(page, block, dim, rows):
    batch = BlockBatch([1, 300, 64, 129], [1, 1, 1, 1], heads=3, dim=dim, page=page, block=block, seed=14, spread=6.0)
    begin, count = [0, 17, 60, 0], [1, 200, 4, 129]
    at = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    k = torch.full((int(at[-1]) + 2, 3, dim), 7.0, dtype=rows, device="cuda")
    v = torch.full_like(k, 7.0)
    skv.kv_gather(batch.problem, torch.from_numpy(at).cuda(), k, v, torch.tensor(begin, dtype=torch.int32, device="cuda"))
    for codes, scales, got in ((batch.k, batch.ks, k), (batch.v, batch.vs, v)):
        for b in range(4):
            page_, slot = batch.slots(b, begin[b], begin[b] + count[b])
            x = VALUES[codes[page_, :, slot]].astype(np.float32) * scales[page_, :, slot // block][..., None]
            assert torch.equal(got[at[b]:at[b + 1]].cpu(), torch.from_numpy(x).to(rows))
        assert (got[int(at[-1]):] == 7.0).all()


# ---- attention ----------------------------------------------------------------------
DECODE = [([1, 63, 64, 65, 300, 1000], [1] * 6), ([4097], [1]), ([129, 257], [2, 4])]


@pytest.mark.parametrize("poison", [False, True])
@pytest.mark.parametrize("page,block,heads,group", [(64, 16, 2, 8), (64, 64, 1, 16), (128, 128, 2, 1), (128, 32, 1, 5),
                                                    (128, 16, 8, 2), (64, 32, 1, 12)])
@pytest.mark.parametrize("lengths", range(len(DECODE)))
def test_decode_against_float64(lengths, page, block, heads, group, poison):
    seq, new = DECODE[lengths]
    batch = BlockBatch(seq, new, heads=heads, group=group, page=page, block=block, seed=20 + lengths, spread=2.0, poison=poison)
    att = skv.SplitKVAttention(batch.problem)
    assert att.plan.kernel_path == 1
    ref = batch.attention()
    check_attention(batch, *att.decode(), ref=ref)
    att.check_device_error()


@pytest.mark.parametrize("group,new", [(1, [33, 64, 17]), (8, [5, 8, 7]), (16, [3, 4, 2]), (5, [7, 12, 1])])
@pytest.mark.parametrize("heads", [1, 24])
def test_blocks_of_up_to_64_rows(group, new, heads):
    """17 to 64 query rows of a KV head in one block: more rows than lanes where states are combined; split
    (few heads) and unsplit requests."""
    batch = BlockBatch([700, 64, 1300], new, heads=heads, group=group, page=64, block=32, seed=25, spread=2.0, poison=True)
    att = skv.SplitKVAttention(batch.problem)
    assert att.plan.num_chunk_tasks == 0
    check_attention(batch, *att.decode())
    att.check_device_error()


@pytest.mark.parametrize("spread", [12.0])
def test_scales_far_apart_keep_their_bits(spread):
    """Value scales from 2^-40 to 2^40 of one another: rows that weigh a block of tiny values alone
    keep them to the bound (which is relative to what the row sums)."""
    batch = BlockBatch([200, 512, 64], [1, 1, 1], heads=2, group=4, page=64, block=16, seed=30, spread=spread)
    check_attention(batch, *skv.SplitKVAttention(batch.problem).decode())


def test_blocks_of_scale_zero():
    batch = BlockBatch([200, 90], [1, 1], heads=2, group=4, page=64, block=16, seed=31)
    batch.vs[::2, :, ::2] = 0.0
    batch.vs[batch.table[1, :2]] = 0.0                      # every value of a request: the output is 0
    batch.ks[1::2] = 0.0
    batch.vs_dev.copy_(torch.from_numpy(batch.vs))
    batch.ks_dev.copy_(torch.from_numpy(batch.ks))
    out, lse = skv.SplitKVAttention(batch.problem).decode()
    check_attention(batch, out, lse)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("page,block,group,seq,new", [(64, 16, 8, [300, 90], [37, 5]), (128, 128, 4, [700], [150]),
                                                      (64, 64, 1, [200, 333], [200, 70]), (64, 32, 16, [260, 64], [9, 64]),
                                                      (128, 64, 8, [900, 40], [300, 33])])
@pytest.mark.parametrize("poison", [False, True])
def test_chunks_of_new_tokens(page, block, group, seq, new, poison):
    batch = BlockBatch(seq, new, heads=2, group=group, page=page, block=block, seed=40, spread=2.0, poison=poison)
    att = skv.SplitKVAttention(batch.problem)
    check_attention(batch, *att.decode())
    att.check_device_error()


@pytest.mark.parametrize("params", [dict(mode="uniform", uniform_splits=3), dict(mode="uniform", uniform_splits=5, interleave=1),
                                    dict(mode="uniform", uniform_splits=4, partial_dtype=skv.BF16)])
def test_splits_interleaved_and_two_stage(params):
    batch = BlockBatch([300, 64, 1000], [1, 1, 3], heads=2, group=4, page=64, block=32, seed=50, spread=2.0, poison=True)
    att = skv.SplitKVAttention(batch.problem, skv.plan_params(**params))
    o, l, bound, lse_bound = batch.attention()
    if params.get("partial_dtype") == skv.BF16:
        # each split's output is rounded once more: by at most 2^-8 of its own values, whose weighted sum A covers
        worst = np.abs(VALUES[np.isfinite(VALUES)]).max() * np.nanmax(batch.vs)
        bound = bound + 2.0 ** -8 * worst
    check_attention(batch, *att.decode(), ref=(o, l, bound, lse_bound))
    check_attention(batch, *att.two_stage(), ref=(o, l, bound, lse_bound))


@pytest.mark.parametrize("params", [dict(), dict(mode="uniform", uniform_splits=3), dict(mode="uniform", uniform_splits=4, partial_dtype=skv.BF16),
                                    dict(mode="uniform", uniform_splits=30)])
def test_split_chunks(params):
    """Chunk tiles whose histories are split (by the planner, where there are few of them), beside decoding requests."""
    batch = BlockBatch([1500, 300, 2100], [40, 1, 17], heads=2, group=8, page=64, block=32, seed=51, spread=2.0, poison=True)
    att = skv.SplitKVAttention(batch.problem, skv.plan_params(**params) if params else None)
    assert att.plan.num_chunk_tasks > 0 and att.plan.splits()[0] > 1 and att.plan.overlap_ctas == 0
    o, l, bound, lse_bound = batch.attention()
    if params.get("partial_dtype") == skv.BF16:
        bound = bound + 2.0 ** -8 * 448.0 * np.nanmax(batch.vs)
    check_attention(batch, *att.decode(), ref=(o, l, bound, lse_bound))
    check_attention(batch, *att.two_stage(), ref=(o, l, bound, lse_bound))
    att.check_device_error()


@pytest.mark.parametrize("page,block,dim,heads,group", [(16, 16, 128, 2, 4), (64, 32, 64, 1, 8), (128, 64, 64, 2, 2), (32, 16, 128, 1, 3)])
def test_other_shapes_on_the_float32_path(page, block, dim, heads, group):
    batch = BlockBatch([1, 100, 333], [1, 3, 20], heads=heads, group=group, dim=dim, page=page, block=block, seed=60, spread=3.0,
                       poison=True)
    att = skv.SplitKVAttention(batch.problem)
    assert att.plan.kernel_path == 0
    check_attention(batch, *att.decode())


def test_graph_replays_follow_the_cache():
    batch = BlockBatch([300, 65], [1, 1], heads=2, group=8, page=64, block=16, seed=70)
    att = skv.SplitKVAttention(batch.problem)
    out, lse = att.out_like()
    k, v = rows_of(batch, torch.bfloat16, seed=71)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        skv.kv_append(batch.problem, k, v)
        att.decode(out, lse)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        skv.kv_append(batch.problem, k, v)
        att.decode(out, lse)
    for seed in (72, 73):
        batch.k, batch.ks, batch.v, batch.vs = (t.cpu().numpy() for t in (batch.k_dev, batch.ks_dev, batch.v_dev, batch.vs_dev))
        k2, v2 = rows_of(batch, torch.bfloat16, seed=seed, size=4.0)
        k.copy_(k2)
        v.copy_(v2)
        want = expected(batch, k2, v2)
        graph.replay()
        torch.cuda.synchronize()
        assert same_codes(batch.k_dev.cpu().numpy(), want[0]) and same_codes(batch.v_dev.cpu().numpy(), want[2])
        check_attention(batch, out, lse, ref=batch.attention(want))


def test_chunk_tiles_beside_decoding_requests():
    """Enough chunk tasks for all SMs and decoding requests: the two kernels run side by side on streams of their own."""
    batch = BlockBatch([2000] * 8 + [700], [1] * 8 + [640], heads=8, group=8, page=64, block=16, seed=52, spread=2.0, poison=True)
    att = skv.SplitKVAttention(batch.problem)
    assert att.plan.overlap_ctas > 0 and att.plan.num_chunk_tasks >= 152
    out, lse = att.out_like()
    for _ in range(3):
        att.decode(out, lse)
    att.check_device_error()
    # every decoding row, and chunk rows spread over the request
    some = BlockBatch([2000] * 8, [1] * 8, heads=8, group=8, page=64, block=16, seed=52, spread=2.0, poison=True)
    for name in ("k", "v", "ks", "vs", "table"):
        setattr(some, name, getattr(batch, name))
    some.q = batch.q[:8]
    check_attention(some, out[:8], lse[:8])
    for i in (0, 1, 63, 300, 639):
        one = BlockBatch([61 + i], [1], heads=8, group=8, page=64, block=16, seed=52, spread=2.0)
        for name in ("k", "v", "ks", "vs"):
            setattr(one, name, getattr(batch, name))
        one.table, one.q = batch.table[8:], batch.q[8 + i:9 + i]
        check_attention(one, out[8 + i:9 + i], lse[8 + i:9 + i])


@pytest.mark.parametrize("seq,new,chunks", [([300, 1000, 65], [1, 1, 1], False), ([600, 90], [40, 1], True)])
def test_withheld_tasks_time_out_and_the_context_survives(seq, new, chunks):
    """The test hook withholds every task: the bounded waits of the engine and of the chunk tiles run out into an error
    status, and the next launch is right."""
    batch = BlockBatch(seq, new, heads=2, group=8, page=64, block=16, seed=55)
    att = skv.SplitKVAttention(batch.problem, skv.plan_params("uniform", uniform_splits=2))
    assert (att.plan.num_chunk_tasks > 0) == chunks
    skv.debug_set_inject(1)
    try:
        att.decode()
        torch.cuda.synchronize()
    finally:
        skv.debug_set_inject(0)
    assert skv.read_device_error(att.error_word, clear=True)[0] == skv.ERR_TIMEOUT
    check_attention(batch, *att.decode())
    att.check_device_error()


def test_bad_pages_are_reported_and_do_not_reach_other_requests():
    """A page id outside the pool: its request's rows are undefined, the others' right, in the engine and the tiles."""
    for new in ([1, 1], [40, 40]):
        batch = BlockBatch([300, 500], new, heads=2, group=4, page=64, block=16, seed=56)
        ref = batch.attention()
        batch.table_dev[0, 2] = batch.num_pages + 7
        att = skv.SplitKVAttention(batch.problem)
        out, lse = att.decode()
        assert skv.read_device_error(att.error_word, clear=True)[0] == skv.ERR_DEVICE_CHECK
        t = new[0]
        o, l, bound, lse_bound = ref
        assert (np.abs(out[t:].double().cpu().numpy() - o[t:]) <= bound[t:]).all()


def test_decode_without_a_workspace_of_its_own():
    batch = BlockBatch([300, 1000, 65], [1, 2, 1], heads=2, group=8, page=64, block=32, seed=57)
    plan = skv.splitkv_plan(batch.problem)
    out = torch.empty(4, 16, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(4, 16, device="cuda")
    skv.splitkv_decode_static(batch.problem, plan, out, lse)
    check_attention(batch, out, lse)
    assert skv.read_static_device_error()[0] == skv.OK


def test_two_batches_on_two_streams():
    """Append and attention of two batches at once, each on its own stream."""
    pair = [BlockBatch([700, 900], [30, 1], heads=2, group=8, page=64, block=16, seed=s) for s in (58, 59)]
    rows = [rows_of(b, torch.bfloat16, seed=s) for b, s in zip(pair, (58, 59))]
    want = [expected(b, *r) for b, r in zip(pair, rows)]
    atts = [skv.SplitKVAttention(b.problem) for b in pair]
    outs = [a.out_like() for a in atts]
    streams = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, r, a, o, s in zip(pair, rows, atts, outs, streams):
            skv.kv_append(b.problem, *r, stream=s)
            a.decode(*o, stream=s)
    torch.cuda.synchronize()
    for b, w, o in zip(pair, want, outs):
        assert same_codes(b.k_dev.cpu().numpy(), w[0]) and np.array_equal(b.vs_dev.cpu().numpy(), w[3])
        check_attention(b, *o, ref=b.attention(w))


def test_pages_beyond_two_to_the_31_bytes():
    """Pages whose codes lie more than 2^31 bytes into the cache, and their scales."""
    pages, heads, page, dim = 20000, 16, 64, 128                      # 2.6 GB of codes each
    k = torch.zeros(pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    small = BlockBatch([150], [1], heads=heads, group=1, page=page, block=16, seed=80)
    ids = [19999, 17000, 19998]
    ks, vs = torch.ones(pages, heads, 4, device="cuda"), torch.ones(pages, heads, 4, device="cuda")
    for j, p in enumerate(ids):
        src = int(small.table[0, j])
        k[p], v[p] = small.k_dev[src], small.v_dev[src]
        ks[p], vs[p] = small.ks_dev[src], small.vs_dev[src]
    table = torch.tensor([ids + [-1]], dtype=torch.int32, device="cuda")
    problem = small.make(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, page_table=table)
    check_attention(small, *skv.SplitKVAttention(problem).decode())
    kn, vn = rows_of(small, torch.bfloat16, seed=81)
    want = expected(small, kn, vn)
    skv.kv_append(problem, kn, vn)
    for j, p in enumerate(ids):
        src = int(small.table[0, j])
        assert same_codes(k[p].cpu().numpy(), want[0][src]) and np.array_equal(vs[p].cpu().numpy(), want[3][src])
