"""sample_tokens against a restatement in float64: the kept tokens and the drawn token exactly, the
distributions to half a step of float32 and the errors of the weights behind them.

A drawn token can differ from float64's only where sample_u times the total lies within the sums' error of a
border between two tokens.  A weight is rounded to a unit of at most 2^-43 of the largest (half of that: 2^-44, for
each of V tokens) after an exponential whose error is below 2^-40 of itself (of the total, for all together; the
product with top_p or sample_u doubles it), and float64's own sums stay below 2^-40 of the total too.  The rows here are few
and their numbers fixed, and each test asserts that no border is that near."""
import math

import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv

pytestmark = pytest.mark.gpu
F32_STEP = 2.0 ** -24


def reference(x, t=1.0, k=0, p=1.0, mp=0.0, u=None):
    """(probabilities in float64, token, how near a border the draw or a cut is and the total, in units of the largest
    weight) of one row."""
    x = np.asarray(x, np.float64)
    V = x.size
    none = np.zeros(V)
    x = np.where(np.isnan(x), -np.inf, x)
    if not t >= 0 or x.max() == -np.inf:
        return none, -1, np.inf, 0.0
    top = x.max()
    if t == 0:
        probs = none.copy()
        probs[np.argmax(x)] = 1.0
        return probs, int(np.argmax(x)), np.inf, 1.0
    if np.isinf(top):
        z = np.where(x == top, 0.0, -np.inf)
    else:
        with np.errstate(over="ignore", invalid="ignore"):
            z = np.where(x == -np.inf, -np.inf, (x - top) / t)
    keep = x > -np.inf
    if mp > 0 and not np.isinf(top):
        keep &= x - top >= (t * math.log(mp) if mp < 1 else 0.0)
    keep &= z > -np.inf
    order = np.lexsort((np.arange(V), -z))
    order = order[keep[order]]
    near = np.inf
    if k > 0:
        order = order[:k]
    w = np.exp(z[order])
    total = w.sum()
    if p <= 0:
        order = order[:1]
    elif p < 1:
        cum = np.cumsum(w)
        reach = float(np.float32(p)) * cum[-1]
        n = int(np.searchsorted(cum, reach, side="left")) + 1
        near = min(near, np.abs(cum - reach)[np.abs(cum - reach) > 0].min(initial=np.inf))
        order = order[:n]
    weights = none.copy()
    weights[order] = np.exp(z[order])
    cum = np.cumsum(weights)
    token = None
    if u is not None:
        at = float(np.float32(u)) * cum[-1]
        hit = np.nonzero((cum > at) & (weights > 0))[0]
        token = int(hit[0]) if hit.size else int(np.nonzero(weights)[0][-1])
        gaps = np.abs(cum[weights > 0] - at)
        near = min(near, gaps[gaps > 0].min(initial=np.inf))
    return weights / cum[-1], token, near, total


def check(x, u, t=None, k=None, p=None, mp=None):
    """x [rows, V] (float32 or bfloat16, on the device); settings lists or None."""
    rows, V = x.shape
    dev = lambda v, dt: None if v is None else torch.tensor(v, dtype=dt, device="cuda")  # noqa: E731
    probs = torch.full((rows, V), -1.0, device="cuda")
    kw = dict(temperature=dev(t, torch.float32), top_k=dev(k, torch.int32), top_p=dev(p, torch.float32), min_p=dev(mp, torch.float32))
    ud = torch.tensor(u, dtype=torch.float32, device="cuda")
    tokens = skv.sample_tokens(x, ud, probs_out=probs, **kw)
    alone = skv.sample_tokens(x, ud, **kw)
    only = torch.full((rows, V), -1.0, device="cuda")
    assert skv.sample_tokens(x, None, probs_out=only, **kw) is None
    assert torch.equal(tokens, alone) and torch.equal(only, probs)
    host = x.double().cpu().numpy()
    got = probs.double().cpu().numpy()
    f32 = lambda v, r, off: off if v is None else float(np.float32(v[r]))  # noqa: E731
    for r in range(rows):
        want, token, near, total = reference(host[r], f32(t, r, 1.0), 0 if k is None else k[r], f32(p, r, 1.0), f32(mp, r, 0.0), u[r])
        assert near > V * 2.0 ** -44 + 4 * 2.0 ** -40 * total, f"row {r}: a border within {near:.2e} (total {total:.3g})"
        # (probabilities below float32's normal numbers may be 0)
        assert ((got[r] > 0) == (want > 0))[(want == 0) | (want > 1e-37)].all(), f"row {r}: kept tokens differ"
        # half a step of the result, half of one of each rounded factor, and the weights' 2^-40
        assert (np.abs(got[r] - want) <= want * (3 * F32_STEP + 2.0 ** -39) + 1e-37).all(), f"row {r}"
        assert int(tokens[r]) == token, f"row {r}: token {int(tokens[r])}, expected {token}"
    return tokens


def logits_of(rows, V, seed=0, slope=1.5, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = -torch.log1p(-torch.rand(rows, V, generator=g)) * slope + torch.randn(rows, V, generator=g) * 0.3 - 3.0
    return x.to(dtype).cuda()


def uniform(rows, seed):
    return [float(np.float32(v)) for v in np.random.default_rng(seed).random(rows)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 128, 1000, 4096, 4097, 32000, 100003])
def test_without_filters(V, dtype):
    check(logits_of(5, V, seed=V, dtype=dtype), uniform(5, V))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 9, 513, 5000, 32000])
@pytest.mark.parametrize("slope", [0.0, 0.05, 0.7, 1.5, 6.0])
def test_filters_alone_and_together(V, slope, dtype):
    """slope 0.05: everything in a few histogram bins; 0: noise of 0.3 alone."""
    t = [1.0, 0.7, 1.3, 0.0, 0.01, 1.0, 2.0, 0.5, 1.0, 0.9, 100.0, 1e-6]
    k = [0, 50, 0, 3, 0, 1, 3000, 7, 2500, 1 << 30, 40, 5]
    p = [1.0, 1.0, 0.9, 0.5, 0.95, 0.3, 0.8, 0.99, 1.0, 0.999, 0.5, 0.7]
    mp = [0.0, 0.0, 0.0, 0.1, 0.05, 0.0, 0.02, 0.3, 0.0, 1e-4, 0.0, 0.0]
    n = len(t)
    x = logits_of(n, V, seed=int(V + 1000 * slope), slope=slope, dtype=dtype)
    u = uniform(n, V)
    check(x, u, t=t, k=k, p=p, mp=mp)
    check(x, u, k=k)
    check(x, u, p=p)
    check(x, u, mp=mp, t=t)


@pytest.mark.parametrize("V", [8, 3000, 50000])
def test_equal_logits(V):
    """All tokens alike: what is kept are the lowest ones, whose number the borders give exactly."""
    x = torch.full((6, V), 1.25, device="cuda")
    x[3] = 0.0
    x[3, ::2] = -0.0
    k = [0, V // 2, 0, V // 4, 5, 0]
    p = [1.0, 1.0, 0.5, 1.0, 0.25, 0.125]
    check(x, [0.9999, 0.1, 0.5, 0.75, 0.3, 0.77], k=k, p=p)


def test_many_equal_logits_at_the_cut():
    """The cut falls among thousands of equal logits, below a few larger ones and above smaller ones."""
    x = torch.full((4, 40000), -2.0, device="cuda")
    x[:, 1000:9000] = 1.0
    x[:, 20000:20003] = 3.0
    check(x, uniform(4, 5), k=[4003, 0, 6000, 9000], p=[1.0, 0.4, 0.7, 0.9])
    check(x.bfloat16(), uniform(4, 6), k=[3000, 0, 2, 20000], p=[0.9, 0.8, 0.7, 0.999])


@pytest.mark.parametrize("V", [50, 20000])
def test_infinities_and_nan(V):
    x = logits_of(8, V, seed=9)
    inf, nan = float("inf"), float("nan")
    x[0, ::3] = -inf
    x[1, 1::2] = nan
    x[2] = -inf
    x[3] = nan
    x[4, [4, 17, 30]] = inf
    x[5] = -inf
    x[5, 11] = -1e38
    x[6, 3] = 3e38
    x[6, 7] = -3e38
    x[7, V - 1] = nan
    for kw in (dict(), dict(k=[3] * 8), dict(p=[0.6] * 8), dict(mp=[0.2] * 8, t=[0.5] * 8), dict(t=[0.0] * 8)):
        tokens = check(x, [0.5, 0.2, 0.3, 0.4, 0.5, 0.6, 0.7, 0.8], **kw)
        assert tokens[2] == -1 and tokens[3] == -1


def test_random_numbers_at_their_ends():
    x = logits_of(1, 3000, seed=11).expand(6, -1).contiguous()
    x[:, 0] = -float("inf")
    u = [0.0, 1.0 - 2.0 ** -24, 2.0 ** -149, 1.0, 2.0, -0.5]
    tokens = skv.sample_tokens(x, torch.tensor(u, device="cuda"))
    assert tokens.tolist() == [1, 2999, 1, 2999, 2999, 1]
    assert int(skv.sample_tokens(x[:1], torch.tensor([float("nan")], device="cuda"))[0]) == 1


def test_settings_at_their_ends():
    nan = float("nan")
    x = logits_of(8, 5000, seed=12)
    check(x, uniform(8, 12), k=[-5, 0, 1, 5000, 4999, 2 ** 31 - 1, -2 ** 31, 2], p=[0.0, -1.0, 2.0, 1.0, 1e-30, 0.9999999, 0.5, 1e-42],
          mp=[0.0, -1.0, 0.0, 0.0, 0.0, 0.0, 1e-30, 0.0])
    check(x, uniform(8, 13), mp=[1.0, 0.999, 5.0, 1e-45, 0.0, 0.5, 1.0, 0.1], t=[1.0, 1e-3, 1.0, 30.0, 1e-20, 1e20, 0.0, 1e30])
    off = skv.sample_tokens(x, torch.full((8,), 0.4, device="cuda"))
    same = skv.sample_tokens(x, torch.full((8,), 0.4, device="cuda"), top_p=torch.full((8,), nan, device="cuda"),
                             min_p=torch.full((8,), nan, device="cuda"))
    assert torch.equal(off, same)


def test_wrong_temperatures_are_reported():
    x = logits_of(3, 400, seed=14)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    probs = torch.ones(3, 400, device="cuda")
    t = torch.tensor([-1.0, float("nan"), 1.0], device="cuda")
    tokens = skv.sample_tokens(x, torch.full((3,), 0.5, device="cuda"), temperature=t, probs_out=probs, dev_error_word=err)
    assert skv.read_device_error(err)[0] == skv.ERR_DEVICE_CHECK
    assert tokens[:2].tolist() == [-1, -1] and tokens[2] >= 0 and (probs[:2] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_rows(dtype):
    wide = logits_of(6, 5003, seed=15, dtype=dtype)
    for a, b in ((0, 5000), (1, 5001), (3, 803)):
        check(wide[:, a:b], uniform(6, a), k=[0, 40, 0, 9, 0, 0], p=[1.0, 0.9, 0.5, 0.8, 1.0, 0.99])
    probs = torch.full((6, 5011), -1.0, device="cuda")
    skv.sample_tokens(wide, None, probs_out=probs[:, 3:5006])
    assert (probs[:, :3] == -1).all() and (probs[:, 5006:] == -1).all() and (probs[:, 3:5006] > 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset,V", [(3, 5003), (4, 5003), (4, 5008), (8, 4097), (4, 3), (8, 70001)])
def test_few_kept_tokens_in_strided_distributions(offset, V, dtype):
    """Rows that keep few tokens, at bases and lengths that are multiples of a vector or not: what lies
    beside the rows stays, what is not kept is zero."""
    rows = 5
    x = logits_of(rows, V, seed=21, dtype=dtype)
    for kw in (dict(temperature=torch.zeros(rows, device="cuda")),
               dict(top_k=torch.full((rows,), 3, dtype=torch.int32, device="cuda")),
               dict(top_k=torch.full((rows,), 150, dtype=torch.int32, device="cuda")),
               dict(top_p=torch.full((rows,), 0.3, device="cuda"))):
        want = torch.full((rows, V), float("nan"), device="cuda")
        skv.sample_tokens(x, None, probs_out=want, **kw)
        wide = torch.full((rows, (V + offset + 9) // 4 * 4), -1.0, device="cuda")
        skv.sample_tokens(x, None, probs_out=wide[:, offset:offset + V], **kw)
        assert torch.equal(wide[:, offset:offset + V], want)
        assert (wide[:, :offset] == -1).all() and (wide[:, offset + V:] == -1).all()
        assert ((want > 0).sum(1) >= 1).all() and torch.allclose(want.double().sum(1), torch.ones(rows, device="cuda").double(), atol=1e-5)
        if "top_k" in kw:
            assert ((want > 0).sum(1) <= int(kw["top_k"][0])).all()


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_row_counts_take_other_cluster_sizes(rows):
    x = logits_of(rows, 20000, seed=rows)
    check(x[:12], uniform(12, 1)[:min(12, rows)], k=[0, 5, 900, 3000] * 3, p=[0.9] * 12) if rows >= 12 else None
    u = torch.tensor(uniform(rows, 2), device="cuda")
    kw = dict(top_k=torch.full((rows,), 60, dtype=torch.int32, device="cuda"), top_p=torch.full((rows,), 0.9, device="cuda"))
    whole = skv.sample_tokens(x, u, **kw)
    one = torch.cat([skv.sample_tokens(x[i:i + 1], u[i:i + 1], top_k=kw["top_k"][:1], top_p=kw["top_p"][:1]) for i in range(rows)])
    assert torch.equal(whole, one)


def test_two_calls_at_once():
    """Two batches of rows on two streams, and the same rows again: equal to each alone."""
    x = [logits_of(20, 30000, seed=s, slope=slope) for s, slope in ((30, 1.6), (31, 0.7))]
    u = torch.tensor(uniform(20, 32), device="cuda")
    kw = dict(top_p=torch.full((20,), 0.95, device="cuda"))
    alone = [skv.sample_tokens(y, u, **kw) for y in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            out = torch.empty(20, dtype=torch.int32, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            skv.sample_tokens(x[i], u, out_tokens=out, stream=s, **kw)
            got[i].append(out)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in got[i])


def test_largest_vocabulary_and_many_rows():
    """2^19 tokens, all alike but for a few (the sums come near their 64 bits), and more rows than CTAs."""
    V = 1 << 19
    x = torch.zeros(3, V, device="cuda")
    x[1, 77], x[1, V - 1] = 1.0, 1.0
    x[2] = -5.0
    got = skv.sample_tokens(x, torch.tensor([0.5, 0.25, 1.0 - 2.0 ** -24], device="cuda"))
    assert int(got[0]) == V // 2 and int(got[2]) == V - 1
    check(x[1:2], [0.25])
    check(x[:2], [0.5, 0.9], p=[0.75, 0.5], k=[0, 400000])
    rows = logits_of(5000, 600, seed=33)
    u = uniform(5000, 33)
    many = skv.sample_tokens(rows, torch.tensor(u, device="cuda"), top_k=torch.full((5000,), 20, dtype=torch.int32, device="cuda"))
    host = rows.cpu().numpy()
    for r in range(0, 5000, 97):
        assert int(many[r]) == reference(host[r], k=20, u=u[r])[1]


def test_frequencies_follow_the_distribution():
    """1 / n of evenly spread numbers give each token its probability, within 1 / n."""
    n = 20000
    x = logits_of(1, 12, seed=16).expand(n, -1).contiguous()
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tokens = skv.sample_tokens(x, u.float())
    want = torch.softmax(x[0].double(), 0)
    got = torch.bincount(tokens, minlength=12).double() / n
    assert (got - want).abs().max() <= 1.5 / n


def test_replayed_graph_and_probabilities_for_verification():
    """The distributions are what verify_drafts takes: with certain drafts equal to tokens of probability 1
    all are accepted, and a captured pair of calls follows its inputs."""
    V, T = 3000, 4
    x = torch.empty(T, V, device="cuda")
    u = torch.empty(T, device="cuda")
    temp = torch.empty(T, device="cuda")
    probs = torch.empty(T, V, device="cuda")
    fed = torch.zeros(T, dtype=torch.int32, device="cuda")
    qo = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out, acc = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    tokens = torch.empty(T, dtype=torch.int32, device="cuda")

    def call():
        skv.sample_tokens(x, u, temperature=temp, out_tokens=tokens, probs_out=probs)
        skv.verify_drafts(fed, qo, probs, None, u, u[:1], out, acc)

    x.copy_(logits_of(T, V, seed=17))
    u.fill_(0.5)
    temp.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (18, 19):
        x.copy_(logits_of(T, V, seed=seed))
        best = x.argmax(1).int()
        fed[1:] = best[:-1]
        graph.replay()
        torch.cuda.synchronize()
        assert tokens.tolist() == best.tolist() and out.tolist() == best.tolist() and int(acc) == T - 1
