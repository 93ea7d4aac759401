"""A batch over a paged E4M3 cache with block scales, on the host in float64 and on the device."""
import math

import numpy as np
import torch

import long_context_split_gb300 as skv


def e4m3_values():
    """The value of every code (NaN for 0x7F, 0xFF)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0)) * np.where(c & 0x80, -1.0, 1.0)
    return np.where((c & 0x7F) == 0x7F, np.nan, v)


VALUES = e4m3_values()
_POS = VALUES[:0x7F]


def encode(x):
    """Codes of float64 values: nearest, ties to the even code, saturated at 448; NaN -> 0x7F."""
    a = np.minimum(np.abs(x), 448.0)
    i = np.searchsorted(_POS, np.nan_to_num(a), side="left").clip(0, 0x7E)
    lo = np.maximum(i - 1, 0)
    d_lo, d_hi = np.abs(a - _POS[lo]), np.abs(_POS[i] - a)
    pick = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, i)
    return np.where(np.isnan(x), 0x7F, pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


class BlockBatch:
    """seq / new: lengths per request.  The cache is full of random codes and scales, those of unused
    slots and blocks included (NaN codes and NaN scales there with `poison`)."""

    def __init__(self, seq, new, heads=2, group=1, dim=128, page=64, block=16, seed=0, spread=1.0, poison=False, dev="cuda",
                 extra=2):
        g = np.random.default_rng(seed)
        self.seq, self.new, self.heads, self.group, self.dim = list(seq), list(new), heads, group, dim
        self.page, self.block, self.dev = page, block, dev
        self.qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pages = [-(-n // page) for n in seq]
        self.num_pages = sum(pages) + extra
        perm = g.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((len(seq), max(pages) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        N, per = self.num_pages, page // block
        normal = lambda shape: np.clip(g.standard_normal(shape) * 60.0, -448, 448)  # noqa: E731
        self.k, self.v = encode(normal((N, heads, page, dim))), encode(normal((N, heads, page, dim)))
        self.ks = (np.exp2(g.standard_normal((N, heads, per)) * 0.3) / 60.0).astype(np.float32)
        self.vs = (np.exp2(g.standard_normal((N, heads, per)) * spread) / 60.0).astype(np.float32)
        if poison:
            used = np.zeros((N, page), bool)
            for b, n in enumerate(self.seq):
                j = np.arange(n)
                used[self.table[b, j // page], j % page] = True
            for c in (self.k, self.v):
                c[np.broadcast_to(~used[:, None, :, None], c.shape)] = 0x7F
            dead = ~used.reshape(N, per, block).any(2)
            for s in (self.ks, self.vs):
                s[np.broadcast_to(dead[:, None], s.shape)] = np.nan
        self.q = torch.from_numpy(g.standard_normal((max(1, int(self.qo[-1])), heads * group, dim)).astype(np.float32)).to(torch.bfloat16)
        self.scale = 1.0 / math.sqrt(dim)
        to = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)  # noqa: E731
        self.k_dev, self.v_dev, self.ks_dev, self.vs_dev = to(self.k), to(self.v), to(self.ks), to(self.vs)
        self.table_dev, self.qo_dev = to(self.table), to(self.qo)
        self.seq_dev = torch.tensor(self.seq, dtype=torch.int32, device=dev)
        self.q_dev = self.q.to(dev)
        self.problem = self.make()

    def make(self, **over):
        kw = dict(q=self.q_dev, k_cache=self.k_dev, v_cache=self.v_dev, page_table=self.table_dev, seq_lens=self.seq_dev,
                  qo_indptr=self.qo_dev, num_q_heads=self.heads * self.group, num_kv_heads=self.heads, head_dim_qk=self.dim,
                  head_dim_v=self.dim, page_size=self.page, scale=self.scale, seq_lens_host=self.seq, qo_indptr_host=self.qo,
                  k_scale=self.ks_dev, v_scale=self.vs_dev)
        kw.update(over)
        return skv.AttentionProblem(**kw)

    def slots(self, b, lo, hi):
        j = np.arange(lo, hi)
        return self.table[b][j // self.page], j % self.page

    def values(self, codes, scales, b, lo, hi):
        """float64 [hi - lo, heads, dim] of tokens lo .. hi-1 of request b."""
        page, slot = self.slots(b, lo, hi)
        return VALUES[codes[page, :, slot]] * scales[page, :, slot // self.block].astype(np.float64)[..., None]

    def attention(self, codes=None):
        """(out, lse, bound, lse_bound) in float64 over the host's cache, or over (k, ks, v, vs) `codes`.

        The bound of an output counts, with p the row's weights and A = sum p |v| per element:
          2^-8 |out|   the rounding to bf16;
          A (2^-11 + 3 d + 2^-18)   weights times scales rounded to f16 (half a step), an error d of the scores and the
                       approximate exponentials (2^-22) and float32 sums behind them;
          448 n 2^-24 max(p vs)   f16's subnormals: 2^-25 of a unit that is at most twice the row's largest product, for n keys;
        d: products of 128 terms accumulated in float32, each of at most (dim + 8) roundings of 2^-23 (accumulators may
        truncate) of the sum of magnitudes; queries below 2^-14 lose at most 2^-25 each."""
        k, ks, v, vs = codes or (self.k, self.ks, self.v, self.vs)
        T, H, g = int(self.qo[-1]), self.heads, self.group
        out, bound = np.zeros((T, H * g, self.dim)), np.zeros((T, H * g, self.dim))
        lse, lse_bound = np.full((T, H * g), -np.inf), np.zeros((T, H * g))
        q = self.q.double().numpy()
        for b, (L, t) in enumerate(zip(self.seq, self.new)):
            kk, vv = self.values(k, ks, b, 0, L), self.values(v, vs, b, 0, L)
            page, slot = self.slots(b, 0, L)
            sv = vs[page, :, slot // self.block].astype(np.float64)            # [L, heads]
            for i in range(t):
                n = L - t + i + 1
                r = int(self.qo[b]) + i
                for h in range(H * g):
                    s = kk[:n, h // g] @ q[r, h] * self.scale
                    mag = (np.abs(kk[:n, h // g]) @ (np.abs(q[r, h]) + 0.0)).max() * self.scale
                    small = np.abs(kk[:n, h // g]).sum(1).max() * self.scale * 2.0 ** -25
                    d = mag * (self.dim + 8) * 2.0 ** -23 + small
                    m = s.max()
                    p = np.exp(s - m)
                    L1 = p.sum()
                    lse[r, h], lse_bound[r, h] = m + np.log(L1), d + 2.0 ** -20 * (1 + abs(m + np.log(L1)))
                    p /= L1
                    o = p @ vv[:n, h // g]
                    A = p @ np.abs(vv[:n, h // g])
                    out[r, h] = o
                    bound[r, h] = 2.0 ** -8 * np.abs(o) + A * (2.0 ** -11 + 3 * d + 2.0 ** -18) \
                        + 448.0 * n * 2.0 ** -24 * (p * sv[:n, h // g]).max()
        return out, lse, bound, lse_bound


def check_attention(batch, out, lse, ref=None):
    o, l, bound, lse_bound = ref or batch.attention()
    got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy().reshape(l.shape)
    assert np.isfinite(got).all()
    err = np.abs(got - o) - bound
    assert (err <= 0).all(), f"worst {err.max():.3e} over a bound of {bound[np.unravel_index(err.argmax(), err.shape)]:.3e}"
    assert (np.abs(got_l - l) <= lse_bound).all(), np.abs(got_l - l).max()
