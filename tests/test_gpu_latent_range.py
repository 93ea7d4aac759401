"""Expanded latent attention where magnitudes are far from 1: values that f16 alone would lose.

The bound on every element is test_gpu_latent's (keys' roundings through the scores, 2^-11 each for values
and probabilities, 2^-13 for sums, 2^-8 for the result), relative to sum p|v| with nothing absolute that could
hide a small value: results are compared times the power of two that brings them back to 1."""
import pytest
import torch

from tests.test_gpu_latent import Case


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
