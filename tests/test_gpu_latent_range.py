"""Expanded latent attention where magnitudes are far from 1: values that f16 alone would lose, and many small
weights.

The bound on every element is test_gpu_latent's (keys' roundings through the scores, 2^-11 each for values
and probabilities, 2^-13 for sums, 2^-8 for the result), relative to sum p|v| with nothing absolute that could
hide a small value: results are compared times the power of two that brings them back to 1."""
import math

import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv
from tests.test_gpu_latent import SCALE, Case


def _scale_values(c, powers):
    """W_uv of head h times 2^powers[h] on the device (exact in bf16); the reference keeps the unscaled weights."""
    w = c.w.clone()
    for h, e in enumerate(powers):
        w[h, 128:] *= 2.0 ** e
    c.kw["w_kv_b"] = w.cuda()


def _unscaled(out, powers):
    return out.double() * torch.tensor([2.0 ** -e for e in powers], dtype=torch.float64, device=out.device)[:, None]


@pytest.mark.gpu
@pytest.mark.parametrize("seq,new,heads", [
    ([300, 65, 1], [300, 65, 1], 2),            # prompts
    ([5000, 90], [3, 90], 2),                   # split histories
    ([130] * 3, [128, 1, 100], 128),            # two heads per task
])
@pytest.mark.parametrize("fp8", [False, True])
def test_values_scaled_by_powers_of_two(seq, new, heads, fp8):
    c = Case(seq, new, heads, 64, fp8, seed=31)
    powers = [(-16, -24, -40, 3, 0)[h % 5] for h in range(heads)]
    keep = [0, 1, 2, 63, 64, 127] if heads > 2 else list(range(heads))      # (a few heads against the reference)
    _scale_values(c, powers)
    _, out, lse = c.run("expanded")
    out = _unscaled(out, powers)[:, keep]
    c.w, c.q, c.heads = c.w[keep], c.q[:, keep], len(keep)
    c.check("expanded", out, lse[:, keep])


@pytest.mark.gpu
def test_latent_rows_scaled_by_powers_of_two():
    for e in (-16, -24):
        c = Case([200, 700], [200, 80], 3, seed=32)
        c.cache *= 2.0 ** e
        c.rows = [r * 2.0 ** e for r in c.rows]
        _, out, lse = c.run("expanded")
        c.w = c.w.float()
        c.w[:, 128:] *= 2.0 ** -e               # the reference's values at 1
        c.check("expanded", out.double() * 2.0 ** -e, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("first,later", [(-24, 0), (0, -24), (-30, -50), (-56, -3)])
@pytest.mark.parametrize("heads,seq,new", [(2, [320], [320]), (1, [6400], [40])])
def test_units_of_different_magnitude(first, later, heads, seq, new):
    """Tokens of the first 64 (and of the last split's first units) times 2^first, the others times 2^later: rows that
    see only the first ones, and rows whose sum meets both.  The rotary columns keep their size, so scores vary."""
    c = Case(seq, new, heads, seed=33)
    n = seq[0]
    scale = torch.full((n,), 2.0 ** later, dtype=torch.float64)
    scale[:64] = 2.0 ** first
    scale[n - n // 4:n - n // 8] = 2.0 ** first
    j = torch.arange(n)
    where = c.table[0].long()[j // 64], j % 64
    c.cache[where[0].cuda(), where[1].cuda(), :512] *= scale.bfloat16().cuda()[:, None]
    c.rows[0][:, :512] *= scale[:, None]
    _, out, lse = c.run("expanded")
    c.w = c.w.float()
    c.w[:, 128:] *= 2.0 ** -min(first, later)   # the smallest values at 1: the bound's absolute floor is far below them
    ref, rl, tol, ltol = c.reference("expanded")
    got = out.cpu().double() * 2.0 ** -min(first, later)
    assert torch.isfinite(got).all()
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{int((over > 0).sum())} elements out of bound, worst by {float(over.max()):.3e}"
    assert ((lse.cpu().double() - rl).abs() <= ltol).all()
    rel = (got - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert float(rel.max()) <= 2.0 ** -6


@pytest.mark.gpu
def test_tokens_of_different_magnitude_within_a_unit():
    """Token j times 2^-(j mod 40): a row of a few small values among a unit of values at 1 keeps an
    absolute error of 2^-39 of the largest (half a step of the smallest f16 numbers) per unit of weight."""
    c = Case([64, 130], [64, 130], 2, seed=34)
    for b, n in enumerate(c.seq):
        j = torch.arange(n)
        scale = 2.0 ** -((j + 39) % 40).double()
        c.cache[c.table[b].long()[j // 64].cuda(), (j % 64).cuda(), :512] *= scale.bfloat16().cuda()[:, None]
        c.rows[b][:, :512] *= scale[:, None]
    _, out, lse = c.run("expanded")
    ref, rl, tol, ltol = c.reference("expanded")
    most = max(float((c.rows[b][:, :512] @ c.w.double()[h, 128:].T).abs().max()) for b in range(2) for h in range(2))
    tol = tol - 2.0 ** -24 + 2.0 ** -39 * most
    over = (out.cpu().double() - ref).abs() - tol
    assert (over <= 0).all(), f"{int((over > 0).sum())} elements out of bound, worst by {float(over.max()):.3e}"


@pytest.mark.gpu
def test_units_without_values():
    """Tokens whose latent columns are all zero (only rotary columns): zero values, weights that count."""
    c = Case([256, 40], [256, 40], 2, seed=35)
    zero = torch.arange(64, 192)
    c.cache[c.table[0].long()[zero // 64].cuda(), (zero % 64).cuda(), :512] = 0
    c.rows[0][zero, :512] = 0
    j = torch.arange(40)
    c.cache[c.table[1].long()[j // 64].cuda(), (j % 64).cuda(), :512] = 0
    c.rows[1][:, :512] = 0
    _, out, lse = c.run("expanded")
    assert (out[256:] == 0).all()
    c.check("expanded", out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1 << 17, 1 << 20])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_many_small_weights_beside_a_large_one(n, at):
    """One key holds 98 % of a row's weight and n - 1 equal ones share the rest; the large key's values are 0, so
    the result is the small ones' share.  Each small weight is off by at most 2^-32 of the largest (an f16
    half step of 2^-25 under a largest of 2^7), all of them together by n 2^-32; the other bounds as
    above.  Enough requests of one token keep the history in one task."""
    others = 160
    pages = n // 64
    cache = torch.zeros(pages + 1, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache[:pages, :, 0] = 1.0
    big = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[at]
    cache[big // 64, big % 64, 0] = 0.0
    cache[big // 64, big % 64, 512] = 16.0
    q_rope = 13.375 if n == 1 << 17 else 15.375          # scores of 0 and of 16 q_rope / sqrt(192)
    q = torch.zeros(1 + others, 1, 192, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 128] = q_rope
    w = torch.zeros(1, 256, 512, dtype=torch.bfloat16)
    w[0, 128:, 0] = torch.rand(128, generator=torch.Generator().manual_seed(3)) * 0.5 + 0.5
    table = torch.full((1 + others, pages), pages, dtype=torch.int32)
    table[0] = torch.arange(pages)
    lens, qo = [n] + [1] * others, list(range(2 + others))
    att = skv.LatentAttention(form="expanded", k_cache=cache, w_kv_b=w.cuda(), page_table=table.cuda(),
                              seq_lens=torch.tensor(lens, dtype=torch.int32).cuda(), scale=SCALE, seq_lens_host=np.array(lens, np.int32),
                              qo_indptr=torch.tensor(qo, dtype=torch.int32).cuda(), qo_indptr_host=np.array(qo, np.int32))
    assert (att.plan.splits() == 1).all()
    lse = torch.zeros(1 + others, 1, device="cuda")
    out = att(q, lse=lse)
    torch.cuda.synchronize()
    att.check_device_error()
    small = (n - 1) * math.exp(-16 * q_rope * SCALE)
    share, v = small / (1 + small), w[0, 128:, 0].double()
    assert 0.0195 < share < 0.0255
    tol = v * (n * 2.0 ** -32 + share * (2.0 ** -10 + 2.0 ** -13 + n / 64 * 2.0 ** -24 + 2.0 ** -8))
    err = (out[0, 0].cpu().double() - share * v).abs()
    assert (err <= tol).all(), f"{float((err / v).max()):.3e} of {share:.3e}"
    # n / 64 float32 additions of a unit's sum to one that is already 1 / share times all the others': half a
    # step of up to 2^-23 each, always to the same side where the addends are equal
    assert abs(float(lse[0, 0]) - (16 * q_rope * SCALE + math.log1p(small))) < n / 64 * 2.0 ** -24 + 1e-5
