"""Latent attention (expanded and absorbed forms) against the formula in float64.

Two checks.  (1) Every element lies within a bound built from the roundings that the form makes,
each taken at its half step, by arithmetic on the case itself:
  expanded  E = scale * 2^-8 * sum_d |q_d k_d| over the latent columns (keys rounded to bf16) bounds
            every score's error, so a weight changes by a factor within exp(+-2E); probabilities and
            values are rounded to f16 (2^-11 each); the result to bf16 (2^-8).
  absorbed  the same with E from the absorbed query's rounding, sum_c |q_lat,c c_c|; probabilities
            as a bf16 pair (2^-15), the latent output as another: 2^-15 sum_c |o_c w_c|.
A further 2^-13 of sum p|v| covers float32 sums, the exponential's approximation and products with
up to 2^11 terms.
(2) The whole output's relative error (2-norm).  A rounding at half step h is uniform in
[-h, h] at worst: rms h / sqrt(3), 2.3e-3 for bf16.  The roundings are independent and the scores'
spread here is about 1, so either form's two bf16 roundings stay within 2.3e-3 * sqrt(2) = 3.2e-3; 4e-3 is
allowed.  (A key left out of a history of
1000 equal weights shows as 3e-2.)"""
import math

import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv

SCALE = 1.0 / math.sqrt(192.0)
NORM = 4e-3


class Case:
    def __init__(self, seq, new, heads, page=64, fp8=False, seed=0, dev="cuda", stale=float("nan")):
        g = torch.Generator().manual_seed(seed)
        self.seq, self.new, self.heads, self.page, self.fp8 = list(seq), list(new), heads, page, fp8
        self.k_scale = 0.0625 if fp8 else None
        self.qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = self.T = int(self.qo[-1])
        pages = [-(-n // page) for n in seq]
        N = sum(pages) + 1
        perm = torch.randperm(N, generator=g, dtype=torch.int32)
        self.table = torch.full((len(seq), max(pages)), -1, dtype=torch.int32)
        at = 0
        # slots that no token owns hold NaN: they must not reach any result
        cache = torch.full((N, page, 576), stale)
        self.rows = []
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
            x = torch.randn(seq[b], 576, generator=g)
            j = torch.arange(seq[b])
            cache[self.table[b].long()[j // page], j % page] = x / 0.0625 if fp8 else x
        cache = cache.to(torch.float8_e4m3fn) if fp8 else cache.bfloat16()
        values = cache.double()
        for b in range(len(seq)):
            j = torch.arange(seq[b])
            r = values[self.table[b].long()[j // page], j % page]
            self.rows.append(r * (0.0625 if fp8 else 1.0))
        self.cache = (cache.view(torch.uint8) if fp8 else cache).to(dev)
        self.w = (torch.randn(heads, 256, 512, generator=g) / math.sqrt(512)).bfloat16()
        self.q = torch.randn(T, heads, 192, generator=g).bfloat16()
        self.kw = dict(k_cache=self.cache, w_kv_b=self.w.to(dev), page_table=self.table.to(dev),
                       seq_lens=torch.tensor(self.seq, dtype=torch.int32).to(dev), qo_indptr=torch.from_numpy(self.qo).to(dev),
                       scale=SCALE, seq_lens_host=self.seq, qo_indptr_host=self.qo, k_scale=self.k_scale)

    def reference(self, form, q=None):
        """out, lse, and the bound on every element of out and lse, in float64."""
        q_all = (self.q if q is None else q).double()
        out = torch.zeros(self.T, self.heads, 128, dtype=torch.float64)
        lse = torch.zeros(self.T, self.heads, dtype=torch.float64)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        w = self.w.double()
        for b, c in enumerate(self.rows):
            lo, hi = self.qo[b], self.qo[b + 1]
            if hi == lo:
                continue
            L, T = self.seq[b], hi - lo
            hide = torch.arange(L)[None] > L - T + torch.arange(T)[:, None]
            for h in range(self.heads):
                qh = q_all[lo:hi, h]
                kn, v = c[:, :512] @ w[h, :128].T, c[:, :512] @ w[h, 128:].T
                s = (qh[:, :128] @ kn.T + qh[:, 128:] @ c[:, 512:].T) * SCALE
                s = s.masked_fill(hide, -math.inf)
                p = torch.softmax(s, 1)
                o = p @ v
                if form == "expanded":
                    e = qh[:, :128].abs() @ kn.abs().T
                else:
                    e = (qh[:, :128] @ w[h, :128]).abs() @ c[:, :512].abs().T
                E = (SCALE * 2.0 ** -8 * e).masked_fill(hide, 0.0).amax(1)
                pv = p @ v.abs()
                rounding = 2.0 ** -10 if form == "expanded" else 2.0 ** -15
                t = ((torch.exp(2 * E) - 1)[:, None] + rounding + 2.0 ** -13) * pv + 2.0 ** -8 * o.abs() + 2.0 ** -24
                if form == "absorbed":
                    t = t + 2.0 ** -15 * (p @ c[:, :512]).abs() @ w[h, 128:].abs().T
                out[lo:hi, h], lse[lo:hi, h] = o, torch.logsumexp(s, 1)
                tol[lo:hi, h], ltol[lo:hi, h] = t, E + 1e-5 + 2.0 ** -20 * lse[lo:hi, h].abs()
        return out, lse, tol, ltol

    def check(self, form, out, lse=None, q=None):
        ref, rl, tol, ltol = self.reference(form, q)
        got = out.cpu().double()
        assert torch.isfinite(got).all()
        over = (got - ref).abs() - tol
        assert (over <= 0).all(), f"{int((over > 0).sum())} elements out of bound, worst by {float(over.max()):.3e}"
        rel = float((got - ref).norm() / ref.norm())
        assert rel <= NORM, f"relative error {rel:.2e}"
        if lse is not None:
            assert ((lse.cpu().double() - rl).abs() <= ltol).all()

    def run(self, form, q=None, lse=True, params=None):
        att = skv.LatentAttention(form=form, params=params, **self.kw)
        lse = torch.full((self.T, self.heads), float("nan"), device="cuda") if lse else None
        out = torch.full((self.T, self.heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        att((self.q if q is None else q).cuda() if not (q is not None and q.is_cuda) else q, out=out, lse=lse)
        torch.cuda.synchronize()
        att.check_device_error()
        return att, out, lse


BATCHES = {
    "one_token": ([1], [1]),
    "edges": ([1, 2, 63, 64, 65, 127, 128, 129], [1, 2, 63, 64, 65, 127, 128, 129]),
    "chunks": ([300, 700, 257], [44, 200, 256]),
    "long_rows": ([513, 900], [513, 300]),
    "no_rows": ([50, 200, 90], [50, 0, 1]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("heads,page,fp8", [(2, 64, False), (3, 16, True), (1, 48, False), (16, 128, False)])
def test_expanded(batch, heads, page, fp8):
    c = Case(*BATCHES[batch], heads, page, fp8, seed=heads + page)
    _, out, lse = c.run("expanded")
    c.check("expanded", out, lse)


@pytest.mark.gpu
def test_expanded_splits_long_histories_of_few_tasks():
    c = Case([9000, 3000, 40], [3, 300, 40], 2, seed=5)
    att, out, lse = c.run("expanded")
    n = att.plan.splits()
    assert n[0] > 4 and n[1] > 1 and n[2] == 1
    c.check("expanded", out, lse)
    _, out2, _ = c.run("expanded", lse=False)
    assert torch.equal(out, out2)                # the merge's order is fixed


@pytest.mark.gpu
def test_expanded_many_heads_and_tasks():
    c = Case([400, 130], [400, 70], 128, seed=6)
    att, out, lse = c.run("expanded")
    assert att.plan.num_tasks > 300 and (att.plan.splits() == 1).all()
    c.check("expanded", out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("seq,new,heads,fp8", [
    ([700, 64, 65, 300, 128, 1, 190], [128, 64, 1, 100, 128, 1, 127], 33, False),   # odd heads: a last task of one
    ([500, 390, 129, 64], [300, 70, 129, 64], 64, True),                            # beside requests of two tiles
    ([257] * 5, [3, 0, 128, 129, 17], 65, False),
])
def test_expanded_two_heads_per_task(seq, new, heads, fp8):
    c = Case(seq, new, heads, 32, fp8, seed=len(seq))
    att, out, lse = c.run("expanded")
    assert att.plan.num_tasks == sum((-(-heads // 2) if n <= 128 else -(-n // 256) * heads) for n in new if n)
    c.check("expanded", out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [128, 16, 1])
@pytest.mark.parametrize("fp8", [False, True])
def test_absorbed(heads, fp8):
    seq, new = ([200, 64, 1, 777], [1, 3, 1, 2]) if heads == 128 else ([200, 64, 1], [1, 3, 1])
    c = Case(seq, new, heads, 64, fp8, seed=7)
    _, out, lse = c.run("absorbed")
    c.check("absorbed", out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("seq,new", [([3000], [1]), ([3000, 100], [2, 1]), ([700] * 9, [1] * 9), ([300] * 20, [2] * 20)])
def test_absorbed_merges_many_splits(seq, new):
    c = Case(seq, new, 128, seed=17)
    for params in (skv.plan_params("uniform", uniform_splits=37), skv.plan_params("uniform", uniform_splits=3, partial_dtype=skv.BF16)):
        att, out, lse = c.run("absorbed", params=params)
        assert att.plan.splits()[0] in (37, 3)
        if att.plan.partial_dtype == torch.float32:
            c.check("absorbed", out, lse)
        else:                                    # the states' own rounding to bf16: 2^-8 of every |o_s| more
            ref, rl, tol, ltol = c.reference("absorbed")
            assert float((out.cpu().double() - ref).norm() / ref.norm()) <= NORM + 2.3e-3
            assert ((lse.cpu().double() - rl).abs() <= ltol).all()


@pytest.mark.gpu
def test_absorbed_single_token_and_more_tokens_than_a_tile():
    for seq, new in (([500], [1]), ([65] * 67, [2] * 67)):
        c = Case(seq, new, 128 if len(seq) == 1 else 8, seed=8)
        _, out, _ = c.run("absorbed", lse=False)
        c.check("absorbed", out)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_queries_sliced_from_a_wider_projection(form):
    c = Case([90, 30], [5, 2], 4, seed=9)
    wide = torch.full((7, 4 * 192 + 64), float("nan"), dtype=torch.bfloat16)
    wide[:, :768] = c.q.view(7, 768)
    q = wide.cuda()[:, :768].view(7, 4, 192)
    assert not q.is_contiguous()
    _, out, lse = c.run(form, q=q)
    c.check(form, out, lse)


@pytest.mark.gpu
def test_auto_takes_the_form_that_the_lengths_make_cheaper():
    prompt, decode = Case([900], [900], 128, seed=10), Case([900], [1], 128, seed=10)
    for c, form in ((prompt, "expanded"), (decode, "absorbed")):
        att, out, _ = c.run("auto", lse=False)
        assert att.form == form
        if c is decode:
            c.check(form, out)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_replays_from_a_graph(form):
    c = Case([300, 70], [40, 1], 128, seed=11)
    att, out, lse = c.run(form)
    q = c.q.cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        att(q, out=out, lse=lse)
    q2 = torch.flip(c.q, dims=[0])
    q.copy_(q2)
    for _ in range(2):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
    att.check_device_error()
    c.check(form, out, lse, q=q2)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_waits_that_run_out_are_reported(form):
    # the loads are withheld (a host-side hook): every wait ends by its limit, the error word tells,
    # and the same object works again after its plan is uploaded
    c = Case([300], [20], 128, seed=14)
    att, out, lse = c.run(form)
    q = c.q.cuda()
    skv.debug_set_inject(1)
    try:
        att(q, out=out, lse=lse)
        st, raw = skv.read_device_error(att.error_word, clear=True)
    finally:
        skv.debug_set_inject(0)
    assert st == skv.ERR_TIMEOUT and raw != 0
    if form == "expanded":
        skv.latent_upload(att.plan, att.workspace)
    else:
        skv.splitkv_plan_upload(att.plan, att.workspace)
    out.fill_(float("nan"))
    att(q, out=out, lse=lse)
    torch.cuda.synchronize()
    att.check_device_error()
    c.check(form, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_a_batch_without_query_rows(form):
    c = Case([30, 7], [0, 0], 128, seed=15)
    att = skv.LatentAttention(form=form, **c.kw)
    assert att(c.q.cuda()).shape == (0, 128, 128)
    torch.cuda.synchronize()
    att.check_device_error()


@pytest.mark.gpu
def test_a_bad_page_and_a_value_beyond_f16_are_reported():
    c = Case([300], [300], 2, seed=12)
    att = skv.LatentAttention(form="expanded", **c.kw)
    c.kw["page_table"][0, 2] = 10 ** 6
    q = c.q.cuda()
    att(q)
    st, raw = skv.read_device_error(att.error_word, clear=True)
    assert st == skv.ERR_DEVICE_CHECK and raw != 0
    c.kw["page_table"].copy_(c.table)
    c.kw["w_kv_b"][1, 130, 0] = 3e38                 # values far beyond 65504, still finite in float32
    c.cache[int(c.table[0, 0]), 5, 0] = 0.001
    c.cache[int(c.table[0, 0]), 6:, 0] = 0.0
    att(q)
    st, _ = skv.read_device_error(att.error_word, clear=True)
    assert st == skv.ERR_DEVICE_CHECK
    c.kw["w_kv_b"].copy_(c.w)
    out = att(q)
    torch.cuda.synchronize()
    att.check_device_error()
    assert torch.isfinite(out.float()).all()


@pytest.mark.gpu
def test_nan_in_a_visible_row_is_not_hidden():
    c = Case([200], [100], 1, seed=13)
    j = 150                                          # token 150 is seen by query rows 50 .. 99
    c.cache[int(c.table[0, j // 64]), j % 64, 3] = float("nan")
    _, out, _ = c.run("expanded")
    assert torch.isnan(out.float()).any(-1)[50:, 0].all()


@pytest.mark.gpu
def test_expanded_rows_that_see_nothing_of_a_later_split():
    c = Case([4096, 1100], [4000, 5], 2, seed=18)
    att, out, lse = c.run("expanded")
    assert att.plan.splits()[0] >= 3             # rows up to 1000 see the first split only
    c.check("expanded", out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_projection_of_states_without_weight(rows, dtype):
    """States of lse -inf contribute nothing, whatever they hold, a row of none but those is 0 with
    lse -inf, and a NaN log-sum-exp is not hidden: rows r of 3 states, by r % 3."""
    c = Case([rows], [rows], 2, seed=19)
    p, R = _problem(c, k_cache=c.cache, q=torch.zeros(rows, 2, 576, dtype=torch.bfloat16, device="cuda"),
                    page_table=c.kw["page_table"]), rows * 2
    g = torch.Generator().manual_seed(1)
    states = torch.randn(R, 3, 512, generator=g).to(dtype)
    lse = torch.randn(R, 3, generator=g)
    kind = torch.arange(R) // 2 % 3              # 0: one empty state, 1: all empty, 2: a NaN lse
    lse[kind == 0, 1] = -math.inf
    lse[kind == 1] = -math.inf
    lse[kind == 2, 0] = float("nan")
    lse[kind == 2, 1:] = -math.inf
    states[lse == -math.inf] = float("nan")
    out = torch.full((rows, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse_out = torch.zeros(rows, 2, device="cuda")
    layer = skv.latent_layer(p, c.q.cuda(), c.kw["w_kv_b"], out, lse_out)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.latent_project(p, layer, states.view(-1, 512).cuda(), lse.view(-1).cuda(),
                       torch.arange(0, 3 * R + 1, 3, dtype=torch.int32, device="cuda"), err)
    torch.cuda.synchronize()
    assert int(err) == 0
    kind, got = kind.view(rows, 2), out.cpu().double()
    assert (got[kind == 1] == 0).all() and (lse_out.cpu()[kind == 1] == -math.inf).all()
    assert torch.isnan(got[kind == 2]).all() and torch.isnan(lse_out.cpu()[kind == 2]).all()
    # the others: the merge in float32 (three terms), the merged output as a bf16 pair (2^-15), one bf16 rounding
    w = torch.softmax(lse.double(), 1).view(rows, 2, 3)
    o = torch.einsum("rhs,rhsc->rhc", w, torch.nan_to_num(states.double(), nan=0.0).view(rows, 2, 3, 512))
    ref = torch.einsum("rhc,hvc->rhv", o, c.w.double()[:, 128:])
    tol = torch.einsum("rhc,hvc->rhv", o.abs(), c.w.double()[:, 128:].abs()) * 2.0 ** -13 + 2.0 ** -8 * ref.abs()
    assert ((got - ref).abs() <= tol)[kind == 0].all()


# ------------------------------------------------------------------ refusals (no GPU needed)
def _status(call):
    with pytest.raises(skv.SplitKVError) as e:
        call()
    return e.value.status


def _problem(c, **over):
    kw = dict(q=torch.zeros(c.T, c.heads, 576, dtype=torch.bfloat16), k_cache=c.cache, v_cache=None, page_table=c.table,
              seq_lens=c.kw["seq_lens"], qo_indptr=c.kw["qo_indptr"], num_q_heads=c.heads, num_kv_heads=1, head_dim_qk=576,
              head_dim_v=512, page_size=c.page, scale=SCALE, kind="mla", seq_lens_host=c.seq, qo_indptr_host=c.qo)
    kw.update(over)
    return skv.AttentionProblem(**kw)


def test_problems_that_are_not_latent_attention_are_refused():
    c = Case([20], [3], 2, dev="cpu")
    assert skv.LatentPlan(_problem(c)).num_tasks == 2
    assert _status(lambda: skv.LatentPlan(_problem(c, scale=0.0))) == skv.ERR_UNSUPPORTED
    assert _status(lambda: skv.LatentPlan(_problem(c, head_dim_v=448))) == skv.ERR_UNSUPPORTED
    assert _status(lambda: skv.LatentPlan(_problem(c, q=torch.zeros(3, 2, 576), k_cache=c.cache.float()))) == skv.ERR_UNSUPPORTED
    gqa = _problem(c, kind="gqa", v_cache=c.cache, head_dim_v=576)
    assert _status(lambda: skv.LatentPlan(gqa)) == skv.ERR_INVALID_ARG
    with pytest.raises(skv.SplitKVError):
        skv.latent_prefers_expanded(gqa)


def test_the_preferred_form_follows_lengths_and_shape():
    def prefers(seq, new, heads, page=64):
        c = Case(seq, new, heads, page, dev="cpu")
        return skv.latent_prefers_expanded(_problem(c))

    assert not prefers([900], [1], 128) and not prefers([900] * 3, [16, 1, 32], 128)
    assert prefers([300], [300], 128) and prefers([900], [200], 128)
    # where the absorbed form would attend on the CUDA cores
    assert prefers([900], [1], 16) and prefers([90], [1], 128, page=16)


def test_layers_are_checked():
    c = Case([20], [3], 2, dev="cpu")
    p = _problem(c)
    out = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    for q, w, o in ((c.q[:2], c.w, out), (c.q.float(), c.w, out), (c.q, c.w[:1], out), (c.q, c.w, out.float()),
                    (c.q.transpose(0, 1).contiguous().transpose(0, 1), c.w, out),
                    (c.q, c.w.transpose(1, 2).contiguous().transpose(1, 2), out)):
        with pytest.raises(TypeError):
            skv.latent_layer(p, q, w, o)
    flat = torch.zeros(3 * 389, dtype=torch.bfloat16)
    odd = flat.as_strided((3, 2, 192), (389, 192, 1))       # rows off the 16-byte grid
    layer = skv.latent_layer(p, odd, c.w, out)
    q_abs = torch.zeros(3, 2, 576, dtype=torch.bfloat16)
    assert _status(lambda: skv.latent_absorb_query(p, layer, q_abs)) == skv.ERR_INVALID_ARG
    layer = skv.latent_layer(p, c.q, c.w, out)
    assert _status(lambda: skv.latent_absorb_query(p, layer, q_abs)) == skv.ERR_INVALID_ARG       # host memory
    states, lse = torch.zeros(6, 512), torch.zeros(6)
    ind = torch.arange(7, dtype=torch.int32)
    assert _status(lambda: skv.latent_project(p, layer, states, lse, ind)) == skv.ERR_INVALID_ARG


def test_the_ends_of_the_absorbed_form_check_their_buffers():
    c = Case([20], [3], 2, dev="cpu")
    p = _problem(c)
    layer = skv.latent_layer(p, c.q, c.w, torch.zeros(3, 2, 128, dtype=torch.bfloat16))
    for q_abs in (torch.zeros(2, 2, 576, dtype=torch.bfloat16), torch.zeros(3, 2, 576), torch.zeros(3, 2, 1152, dtype=torch.bfloat16)[..., ::2]):
        with pytest.raises(TypeError):
            skv.latent_absorb_query(p, layer, q_abs)
    o, lse, ind = torch.zeros(12, 512), torch.zeros(12), torch.arange(0, 14, 2, dtype=torch.int32)
    for bad in ((o.double(), lse, ind), (o[:, :256], lse, ind), (o, lse[:11], ind), (o, lse.double(), ind), (o, lse, ind[:6]),
                (o, lse, ind.long())):
        with pytest.raises(TypeError):
            skv.latent_project(p, layer, *bad)


def test_the_expanded_call_checks_its_plan_and_workspace():
    c = Case([20, 30], [3, 2], 2, dev="cpu")
    p = _problem(c)
    plan = skv.LatentPlan(p)
    layer = skv.latent_layer(p, c.q, c.w, torch.zeros(5, 2, 128, dtype=torch.bfloat16))
    ws = torch.zeros(plan.workspace_bytes + 512, dtype=torch.uint8)
    ws = ws[(-ws.data_ptr()) % 256:]
    assert _status(lambda: skv.latent_expanded(p, plan, layer, ws[:plan.workspace_bytes - 256])) == skv.ERR_WORKSPACE
    assert _status(lambda: skv.latent_expanded(p, plan, layer, ws[1:])) == skv.ERR_WORKSPACE
    assert _status(lambda: skv.latent_upload(plan, ws[:256])) == skv.ERR_WORKSPACE
    longer = _problem(c, seq_lens_host=[20, 31])
    assert _status(lambda: skv.latent_expanded(longer, plan, layer, ws)) == skv.ERR_INVALID_ARG
    none = Case([20], [0], 2, dev="cpu")
    q0 = _problem(none)
    skv.latent_expanded(q0, skv.LatentPlan(q0), skv.latent_layer(q0, none.q, none.w, torch.zeros(0, 2, 128, dtype=torch.bfloat16)), ws)


def test_the_wrapper_checks_its_arguments():
    c = Case([20], [3], 2, dev="cpu")
    for over in (dict(k_cache=c.cache[..., :512].contiguous()), dict(k_cache=c.cache.float()), dict(k_scale=1.0)):
        with pytest.raises(TypeError):
            skv.LatentAttention(**{**c.kw, **over})
    with pytest.raises(ValueError):
        skv.LatentAttention(form="both", **c.kw)
