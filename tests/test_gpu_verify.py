"""verify_drafts against a float64 restatement.  The outputs are whole numbers and must be
equal.  Weights that are multiples of 2^-20 make every sum exact in any order, so draws that
meet a border of the cumulative distribution exactly are tested too; with other weights the
two sides' sums agree to about 2^-45 of the total, far below the distance of a random draw
from the nearest border."""
import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv

BELOW_ONE = float(np.nextafter(np.float32(1), np.float32(0)))


def reference(tokens, qo, p, q, accept_u, sample_u, seq_lens):
    out = np.full(len(tokens), -1, np.int32)
    acc = np.zeros(len(qo) - 1, np.int32)
    lens = np.array(seq_lens, np.int32)
    for b in range(len(qo) - 1):
        r0, r1 = qo[b], qo[b + 1]
        if r1 <= r0:
            continue
        n = a = 0
        n = r1 - r0 - 1
        while a < n:
            x = tokens[r0 + a + 1]
            qx = 1.0 if q is None else float(q[r0 + a, x])
            if not float(accept_u[r0 + a]) * qx < float(p[r0 + a, x]):
                break
            out[r0 + a] = x
            a += 1
        acc[b] = a
        lens[b] = seq_lens[b] - n + a
        row = p[r0 + a].astype(np.float64)
        w = row.copy()
        if a < n:
            if q is None:
                w[tokens[r0 + a + 1]] = 0.0
            else:
                w = w - q[r0 + a].astype(np.float64)
        w = np.where(w > 0, w, 0.0)
        if not w.sum() > 0:
            w = np.where(row > 0, row, 0.0)
        if not w.sum() > 0:
            continue
        cdf = np.cumsum(w)
        hit = np.nonzero((cdf > float(sample_u[b]) * cdf[-1]) & (w > 0))[0]
        out[r0 + a] = hit[0] if len(hit) else np.nonzero(w > 0)[0][-1]
    return out, acc, lens


def run(tokens, qo, p, q, accept_u, sample_u, seq_lens, pad=0):
    """The kernel on the same inputs; pad > 0 gives rows a stride of vocab + pad."""
    def dev(x):
        t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
        if pad and t.dim() == 2:
            wide = torch.full((t.shape[0], t.shape[1] + pad), 9.0, device="cuda")
            wide[:, :t.shape[1]] = t
            t = wide[:, :t.shape[1]]
        return t

    lens_out = torch.full((len(qo) - 1,), -7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, acc = skv.verify_drafts(dev(tokens), dev(qo), dev(p), None if q is None else dev(q), dev(accept_u), dev(sample_u),
                                 seq_lens=dev(np.asarray(seq_lens, np.int32)), seq_lens_out=lens_out, dev_error_word=err)
    return out.cpu().numpy(), acc.cpu().numpy(), lens_out.cpu().numpy(), skv.read_device_error(err)


def check(*args, pad=0):
    out, acc, lens, st = run(*args, pad=pad)
    want = reference(*args)
    assert st == (skv.OK, 0)
    np.testing.assert_array_equal(acc, want[1])
    np.testing.assert_array_equal(out, want[0])
    np.testing.assert_array_equal(lens, want[2])
    return acc


def make(rows, vocab, seed, near=0.4, cut=0.0, dyadic=False):
    """qo, tokens, p, q, u: drafts drawn from q, q a perturbation of p."""
    rng = np.random.default_rng(seed)
    qo = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    T = int(qo[-1])
    logit = rng.standard_normal((T, vocab)) * 2
    def soft(z):
        e = np.exp(z - z.max(1, keepdims=True))
        e[e < cut] = 0.0
        return e / e.sum(1, keepdims=True)
    p, q = soft(logit), soft(logit + near * rng.standard_normal((T, vocab)))
    tokens = np.zeros(T, np.int32)
    for r in range(T - 1):
        tokens[r + 1] = rng.choice(vocab, p=q[r])
    if dyadic:
        p, q = np.round(p * 2 ** 20) / 2 ** 20, np.round(q * 2 ** 20) / 2 ** 20
        u = rng.integers(0, 2 ** 10, T) / 2 ** 10
        s = rng.integers(0, 2 ** 10, len(rows)) / 2 ** 10
    else:
        u, s = rng.random(T), rng.random(len(rows))
    f = lambda x: x.astype(np.float32)  # noqa: E731
    return tokens, qo, f(p), f(q), f(u), f(s), [50] * len(rows)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [1, 2, 5, 127, 128, 1000, 4096, 4099, 32000, 70001])
@pytest.mark.parametrize("pad", [0, 3])
def test_matches_the_restatement(vocab, pad):
    rows = [1, 4, 0, 16, 2, 7, 1]
    if vocab <= 4099:
        rows.append(70)                           # more drafts than a warp tests at once
    check(*make(rows, vocab, seed=vocab, near=0.1), pad=pad)
    check(*make(rows, vocab, seed=vocab + 1, near=1.0, cut=1e-2), pad=pad)


@pytest.mark.gpu
def test_accepts_and_refuses():
    args = make([16] * 40, 1000, seed=3, near=0.3)
    acc = check(*args)
    assert acc.min() < 3 and acc.max() > 10       # both ends occur
    check(args[0], args[1], args[2], args[3], np.zeros_like(args[4]), args[5], args[6])                # u = 0
    check(args[0], args[1], args[2], args[3], np.full_like(args[4], BELOW_ONE), args[5], args[6])


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [64, 1024, 20000])
def test_draws_that_meet_a_border_exactly(vocab):
    tokens, qo, p, q, u, s, lens = make([3] * 64, vocab, seed=5, near=0.5, dyadic=True)
    check(tokens, qo, p, q, u, s, lens)
    # rows of equal weights: u = k / 64 is the border below token k * vocab / 64
    p[:] = 1.0 / 2 ** 20
    q[:] = 0.0
    s = (np.arange(64) / 64).astype(np.float32)
    check(tokens, qo, p, q, np.ones_like(u), s, lens)


@pytest.mark.gpu
def test_certain_drafts_without_a_draft_distribution():
    tokens, qo, p, q, u, s, lens = make([5, 1, 9, 2] * 8, 501, seed=6)
    check(tokens, qo, p, None, u, s, lens)
    acc = check(tokens, qo, p, None, np.zeros_like(u), s, lens)     # u = 0 accepts every draft with weight
    np.testing.assert_array_equal(acc, np.diff(qo) - 1)


@pytest.mark.gpu
def test_the_ends_of_the_distribution():
    tokens, qo, p, q, u, s, lens = make([2] * 32, 3000, seed=7, cut=1e-1)
    for v in (0.0, BELOW_ONE):
        check(tokens, qo, p, q, u, np.full_like(s, v), lens)
    # all weight on one token, first, last and in the middle
    for x in (0, 2999, 1111):
        p[:] = 0.0
        p[:, x] = 1.0
        out, acc, _, _ = run(tokens, qo, p, q, np.ones_like(u), s, lens)
        assert (out[qo[:-1] + acc] == x).all()
        check(tokens, qo, p, q, np.ones_like(u), s, lens)


@pytest.mark.gpu
def test_rows_without_weight():
    tokens, qo, p, q, u, s, lens = make([3] * 6, 700, seed=8)
    one = np.ones_like(u)
    check(tokens, qo, p, p.copy(), one, s, lens)       # p - q zero everywhere: the draw is from p
    p[qo[2]:qo[4]] = 0.0                               # requests 2 and 3: no weight at all
    out, acc, _, st = run(tokens, qo, p, q, one, s, lens)
    assert st == (skv.OK, 0) and out[qo[2]] == -1 and out[qo[3]] == -1
    check(tokens, qo, p, q, one, s, lens)
    p[qo[4], ::2] = np.nan                             # NaN and negative weigh nothing
    p[qo[4], 1] = -1.0
    check(tokens, qo, p, np.zeros_like(q), one, s, lens)


@pytest.mark.gpu
def test_a_draft_outside_the_vocabulary_is_refused_and_reported():
    tokens, qo, p, q, u, s, lens = make([4, 4], 300, seed=9)
    u[:] = 0.0
    tokens[2], tokens[6] = 300, -1
    out, acc, _, st = run(tokens, qo, p, q, u, s, lens)
    assert st[0] == skv.ERR_DEVICE_CHECK
    assert list(acc) == [1, 1] and out[1] >= 0 and out[2] == -1


@pytest.mark.gpu
def test_replays_from_a_graph_with_new_numbers():
    args = make([4] * 5, 5000, seed=10)
    dev = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in args[:6]]
    lens = torch.full((5,), 50, dtype=torch.int32, device="cuda")
    out, acc = torch.empty(20, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        skv.verify_drafts(*dev, out, acc, seq_lens=lens, seq_lens_out=lens)     # lengths in place
    lens.fill_(50)
    for seed in (11, 12):
        other = make([4] * 5, 5000, seed=seed)
        for d, x in zip(dev, other[:6]):
            d.copy_(torch.from_numpy(np.ascontiguousarray(x)))
        before = lens.cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        want = reference(*other[:6], before)
        np.testing.assert_array_equal(out.cpu().numpy(), want[0])
        np.testing.assert_array_equal(acc.cpu().numpy(), want[1])
        np.testing.assert_array_equal(lens.cpu().numpy(), want[2])


@pytest.mark.gpu
def test_rows_past_32_bit_offsets():
    vocab, rows = 120001, 18000                      # 2.2e9 probabilities (8.6 GB)
    p = torch.zeros(rows, vocab, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    p[rows - 3, 7] = 1.0                             # the draft after this row is accepted
    p[rows - 2, 100] = 0.5                           # and refused after this one: the draw
    p[rows - 2, 120000] = 0.5
    tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    tokens[rows - 2], tokens[rows - 1] = 7, 5
    qo = i32([0, 1, rows - 3, rows])
    u = torch.zeros(rows, device="cuda")
    out, acc = skv.verify_drafts(tokens, qo, p, None, u, torch.tensor([0.0, 0.0, 0.75], device="cuda"))
    torch.cuda.synchronize()
    assert acc.tolist() == [0, 0, 1]
    assert out[rows - 3:].tolist() == [7, 120000, -1]
    assert out[0] == -1                              # a row without weight


# ------------------------------------------------------------------ refusals (no GPU needed)
def _host():
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    return dict(tokens=i(4), qo_indptr=i(3), target_probs=torch.zeros(4, 10), draft_probs=torch.zeros(4, 10),
                accept_u=torch.zeros(4), sample_u=torch.zeros(2))


@pytest.mark.parametrize("over", [
    dict(tokens=torch.zeros(4)), dict(qo_indptr=torch.zeros(3)), dict(target_probs=torch.zeros(4, 10).double()),
    dict(target_probs=torch.zeros(3, 10)), dict(draft_probs=torch.zeros(4, 11)), dict(draft_probs=torch.zeros(10, 4).T),
    dict(accept_u=torch.zeros(3)), dict(sample_u=torch.zeros(3)), dict(accept_u=torch.zeros(4).half()),
])
def test_types_and_shapes_are_checked(over):
    a = _host()
    a.update(over)
    with pytest.raises(TypeError):
        skv.verify_drafts(**a)


def test_arguments_are_checked_on_the_host():
    def status(**over):
        a = _host()
        a.update(over)
        with pytest.raises(skv.SplitKVError) as e:
            skv.verify_drafts(**a)
        return e.value.status, str(e.value)

    assert status()[0] == skv.ERR_INVALID_ARG                       # host memory
    assert "come together" in status(seq_lens=torch.zeros(2, dtype=torch.int32))[1]
    a = _host()
    assert "overlap" in status(tokens=a["tokens"], out_tokens=a["tokens"])[1]
    flat = torch.zeros(41)
    assert "stride" in status(target_probs=flat.as_strided((4, 10), (5, 1)))[1]
