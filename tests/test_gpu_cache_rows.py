"""kv_append and kv_gather against a plain restatement: every byte of the cache (written
slots and untouched ones) and every gathered row must match.

The quantisation is restated in float64 from its definition: the quotient x / scale is a
float32 (one rounding, as documented), then the nearest E4M3 number, ties to even, saturated
at 448; codes are compared exactly, so no tolerance is involved.  Gathered values are
code * scale in float32, rounded once to the row type: exact too."""
import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv

ROW = {"f32": torch.float32, "bf16": torch.bfloat16}
CACHE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}
K_SCALE, V_SCALE = 0.0625, 0.05


def e4m3_decode(codes):
    c = codes.astype(np.int64)
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    return np.where((c & 0x7F) == 0x7F, np.nan, sign * v)


_ALL = e4m3_decode(np.arange(0x7F, dtype=np.uint8))     # the non-negative numbers, ascending


def e4m3_encode(x):
    """Codes of float64 values: nearest, ties to the even code, saturated; NaN -> 0x7F."""
    a = np.minimum(np.abs(x), 448.0)
    i = np.searchsorted(_ALL, np.nan_to_num(a), side="left").clip(0, 0x7E)
    lo = np.maximum(i - 1, 0)
    d_lo, d_hi = np.abs(a - _ALL[lo]), np.abs(_ALL[i] - a)
    pick = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, i)
    code = np.where(np.isnan(x), 0x7F, pick | np.where(np.signbit(x), 0x80, 0))
    return code.astype(np.uint8)


def encode(x, cache, scale):
    """Cache entries (torch, CPU) of rows x (torch, CPU)."""
    if cache == "e4m3":
        with np.errstate(all="ignore"):
            quot = x.float().numpy() / np.float32(scale)
        return torch.from_numpy(e4m3_encode(quot.astype(np.float64)))
    return x.to(CACHE[cache])


def decode(codes, cache, scale, rows):
    if cache == "e4m3":
        v = e4m3_decode(codes.numpy()).astype(np.float32) * np.float32(scale)
        return torch.from_numpy(v).to(ROW[rows])
    return codes.to(ROW[rows])


def same(a, b):
    """Equal, NaN equal to NaN."""
    a, b = a.cpu(), b.cpu()
    if a.dtype.is_floating_point:
        return torch.equal(torch.nan_to_num(a.float(), nan=12345.0), torch.nan_to_num(b.float(), nan=12345.0))
    return torch.equal(a, b)


def same_codes(a, b):
    nan = lambda t: torch.where((t & 0x7F) == 0x7F, torch.full_like(t, 0x7F), t)  # noqa: E731
    return torch.equal(nan(a.cpu()), nan(b.cpu()))


class Batch:
    def __init__(self, seq, new, kind="gqa", heads=2, dim=64, page=16, cache="bf16", seed=0, dev="cuda", extra_pages=2):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.heads, self.dim, self.page, self.cache = kind, heads, dim, page, cache
        self.seq, self.new = list(seq), list(new)
        self.qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pages = [-(-n // page) for n in seq]
        self.num_pages = sum(pages) + extra_pages
        perm = torch.randperm(self.num_pages, generator=g, dtype=torch.int32)
        self.table = torch.full((len(seq), max(pages) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (self.num_pages, heads, page, dim) if kind == "gqa" else (self.num_pages, page, dim)
        dt = CACHE[cache]

        def fill():
            if dt == torch.uint8:
                return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
            return torch.randn(shape, generator=g).to(dt)

        self.k, self.v = fill(), fill() if kind == "gqa" else None
        self.k_dev, self.v_dev = self.k.to(dev), None if self.v is None else self.v.to(dev)
        self.seq_dev = torch.tensor(self.seq, dtype=torch.int32, device=dev)
        self.qo_dev = torch.from_numpy(self.qo).to(dev)
        self.table_dev = self.table.to(dev)
        self.problem = self.make_problem()

    def make_problem(self, **over):
        fp8 = self.cache == "e4m3"
        q = torch.empty(max(1, int(self.qo[-1])), self.heads, self.dim, device=self.k_dev.device,
                        dtype=torch.float32 if self.cache == "f32" else torch.bfloat16)
        kw = dict(q=q, k_cache=self.k_dev, v_cache=self.v_dev, page_table=self.table_dev, seq_lens=self.seq_dev,
                  qo_indptr=self.qo_dev, num_q_heads=self.heads, num_kv_heads=self.heads, head_dim_qk=self.dim,
                  head_dim_v=self.dim if self.kind == "gqa" else self.dim - 64, page_size=self.page, scale=0.1,
                  kind=self.kind, seq_lens_host=self.seq, qo_indptr_host=self.qo,
                  k_scale=K_SCALE if fp8 else None, v_scale=V_SCALE if fp8 else None)
        kw.update(over)
        return skv.AttentionProblem(**kw)

    def slots(self, b, lo, hi):
        j = torch.arange(lo, hi)
        return self.table[b].long()[j // self.page], j % self.page

    def write(self, k_rows, v_rows):
        """The expected caches after an append of CPU rows."""
        k, v = self.k.clone(), None if self.v is None else self.v.clone()
        for b in range(len(self.seq)):
            lo, hi = self.qo[b], self.qo[b + 1]
            page, slot = self.slots(b, self.seq[b] - (hi - lo), self.seq[b])
            if self.kind == "gqa":
                k[page, :, slot] = encode(k_rows[lo:hi], self.cache, K_SCALE)
                v[page, :, slot] = encode(v_rows[lo:hi], self.cache, V_SCALE)
            else:
                k[page, slot] = encode(torch.cat([k_rows, v_rows], 1)[lo:hi] if v_rows is not None else k_rows[lo:hi],
                                       self.cache, K_SCALE)
        return k, v

    def check(self, k, v):
        cmp = same_codes if self.cache == "e4m3" else same
        assert cmp(self.k_dev, k)
        if v is not None:
            assert cmp(self.v_dev, v)


def awkward(t):
    """Zeros, infinities, NaN, values past 448 * scale, halfway points and tiny values among normal ones."""
    f = t.reshape(-1)
    special = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 28.0, 29.0, -1000.0, 1e-6, 2.0 ** -13,
                            -(2.0 ** -14), 0.0625 * 17 / 16, 0.0625 * 19 / 16, 3e38], dtype=torch.float32).to(t.dtype)
    n = min(len(special), f.numel())
    f[:n] = special[:n]
    return t


def layout(rows, shape, how, gen, dtype):
    """Row tensor of `shape` on the device with another layout; returns (device view, CPU copy)."""
    x = awkward(torch.randn(shape, generator=gen).to(dtype))
    if how == "plain":
        d = x.cuda()
    elif how == "fused":          # a slice of a wider projection
        wide = torch.randn((shape[0], 3 * shape[1]) + tuple(shape[2:]), generator=gen).to(dtype)
        wide[:, shape[1]:2 * shape[1]] = x
        d = wide.cuda()[:, shape[1]:2 * shape[1]]
    elif how == "odd":            # rows off by one element: no 16-byte alignment
        flat = torch.zeros(x.numel() + 1, dtype=dtype)
        flat[1:] = x.reshape(-1)
        d = flat.cuda()[1:].view(shape)
    else:                         # "heads": head-major storage
        d = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    assert same(d, x)
    return d, x


SHAPES = [
    dict(heads=2, dim=64, page=16), dict(heads=8, dim=128, page=64), dict(heads=1, dim=128, page=128),
    dict(heads=3, dim=20, page=5),                 # nothing a multiple of 8 or 16
]


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["plain", "fused", "odd", "heads"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("cache,rows", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "f32"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_append_gqa(cache, rows, shape, how):
    s = SHAPES[shape]
    B = Batch([1, 40, 17, 200, 64, 9], [1, 3, 17, 70, 0, 9], cache=cache, seed=shape, **s)
    g = torch.Generator().manual_seed(7)
    T = int(B.qo[-1])
    kd, k = layout(T, (T, s["heads"], s["dim"]), how, g, ROW[rows])
    vd, v = layout(T, (T, s["heads"], s["dim"]), how, g, ROW[rows])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.kv_append(B.problem, kd, vd, err)
    assert skv.read_device_error(err) == (skv.OK, 0)
    B.check(*B.write(k, v))


@pytest.mark.gpu
@pytest.mark.parametrize("cache,rows", [("bf16", "bf16"), ("e4m3", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("split", [True, False])
def test_append_latent(cache, rows, split):
    B = Batch([65, 1, 128, 300], [65, 1, 0, 37], kind="mla", heads=1, dim=576, page=64, cache=cache, seed=3)
    g = torch.Generator().manual_seed(8)
    x = awkward(torch.randn(int(B.qo[-1]), 576, generator=g).to(ROW[rows]))
    xd = x.cuda()
    if split:
        skv.kv_append(B.problem, xd[:, :512], xd[:, 512:])
    else:
        skv.kv_append(B.problem, xd)
    torch.cuda.synchronize()
    B.check(*B.write(x, None))


@pytest.mark.gpu
def test_append_a_broadcast_row_and_a_large_batch():
    # one row for every token (stride 0); 1100 requests: the owner search takes several steps
    n = 1100
    new = [(i * 7) % 3 for i in range(n)]
    B = Batch([5 + (i % 13) for i in range(n)], new, heads=2, dim=64, page=16, cache="e4m3", seed=4)
    T = int(B.qo[-1])
    row = torch.randn(1, 2, 64).bfloat16()
    kd = row.cuda().expand(T, 2, 64)
    skv.kv_append(B.problem, kd, kd)
    torch.cuda.synchronize()
    B.check(*B.write(row.expand(T, 2, 64), row.expand(T, 2, 64)))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.05, 0.0625, 1.0 / 3.0, 1e-3, 7.77, 1.0, 448.0, 1e-30, 2.0 ** -126, 3e38])
def test_every_bf16_value_quantises_as_the_quotient(scale):
    # all 65,536 bit patterns (infinities and NaN among them), for scales whose quotient takes a
    # reciprocal and for extreme ones: codes equal those of the float32 quotient
    B = Batch([64], [64], cache="e4m3", heads=8, dim=128, page=64, seed=40)
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(64, 8, 128)
    problem = B.make_problem(k_scale=scale, v_scale=scale)
    skv.kv_append(problem, x.cuda(), x.cuda())
    torch.cuda.synchronize()
    page, slot = B.slots(0, 0, 64)
    k = B.k.clone()
    k[page, :, slot] = encode(x, "e4m3", scale)
    assert same_codes(B.k_dev, k)
    # float32 rows next to every border between two codes
    at = torch.from_numpy((_ALL[1:] + _ALL[:-1]) / 2 * np.float32(scale)).float()
    near = torch.stack([torch.nextafter(at, torch.zeros(())), at, torch.nextafter(at, torch.full((), 3e38))]).reshape(-1)
    f = torch.zeros(64 * 8 * 128)
    f[:len(near)], f[1000:1000 + len(near)] = near, -near
    f = f.view(64, 8, 128)
    skv.kv_append(problem, f.cuda(), f.cuda())
    torch.cuda.synchronize()
    k[page, :, slot] = encode(f, "e4m3", scale)
    assert same_codes(B.k_dev, k)


@pytest.mark.gpu
def test_append_refuses_bad_pages_and_reports_them():
    B = Batch([40, 40], [20, 20], cache="bf16", seed=5)
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(40, 2, 64, generator=g).bfloat16() for _ in range(2))
    want_k, want_v = B.write(k, v)
    # request 1's page 1 (tokens 16 .. 31) gets an id outside the pool: those rows stay unwritten
    page = int(B.table[1, 1])
    B.table_dev[1, 1] = B.num_pages
    want_k[page], want_v[page] = B.k[page], B.v[page]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.kv_append(B.problem, k.cuda(), v.cuda(), err)
    st, raw = skv.read_device_error(err, clear=True)
    assert st == skv.ERR_DEVICE_CHECK and raw != 0
    B.check(want_k, want_v)
    # without an error word the same rows are skipped silently
    skv.kv_append(B.problem, k.cuda(), v.cuda())
    torch.cuda.synchronize()
    B.check(want_k, want_v)


@pytest.mark.gpu
def test_append_in_a_graph_follows_the_device_lengths():
    B = Batch([33, 100], [1, 1], cache="e4m3", heads=2, dim=128, page=64, seed=6)
    kd, vd = torch.zeros(2, 2, 128, device="cuda").bfloat16(), torch.zeros(2, 2, 128, device="cuda").bfloat16()
    stream = torch.cuda.Stream()
    B.seq_dev.copy_(torch.tensor([30, 97], dtype=torch.int32))
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        skv.kv_append(B.problem, kd, vd)
        B.seq_dev.add_(1)
    want_k, want_v = B.k.clone(), B.v.clone()
    g = torch.Generator().manual_seed(10)
    for step in range(4):                       # tokens 29 .. 32 and 96 .. 99
        k, v = (torch.randn(2, 2, 128, generator=g).bfloat16() for _ in range(2))
        kd.copy_(k), vd.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for b, first in ((0, 29), (1, 96)):
            page, slot = B.slots(b, first + step, first + step + 1)
            want_k[page, :, slot] = encode(k[b:b + 1], "e4m3", K_SCALE)
            want_v[page, :, slot] = encode(v[b:b + 1], "e4m3", V_SCALE)
    B.check(want_k, want_v)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["plain", "fused", "odd", "heads"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("cache,rows", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "f32"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_gather_gqa(cache, rows, shape, how):
    s = SHAPES[shape]
    B = Batch([1, 40, 17, 200, 64, 9], [1, 1, 1, 1, 1, 1], cache=cache, seed=20 + shape, **s)
    begin = [0, 3, 16, 130, 64, 0]
    count = [1, 37, 1, 70, 0, 9]
    at = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    rows_out = int(at[-1]) + 3                  # three rows behind the last request
    g = torch.Generator().manual_seed(21)
    kd, k = layout(rows_out, (rows_out, s["heads"], s["dim"]), how, g, ROW[rows])
    vd, v = layout(rows_out, (rows_out, s["heads"], s["dim"]), how, g, ROW[rows])
    for b in range(6):
        page, slot = B.slots(b, begin[b], begin[b] + count[b])
        k[at[b]:at[b + 1]] = decode(B.k[page, :, slot], cache, K_SCALE, rows)
        v[at[b]:at[b + 1]] = decode(B.v[page, :, slot], cache, V_SCALE, rows)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.kv_gather(B.problem, torch.from_numpy(at).cuda(), kd, vd,
                  torch.tensor(begin, dtype=torch.int32, device="cuda"), err)
    assert skv.read_device_error(err) == (skv.OK, 0)
    assert same(kd, k) and same(vd, v)


@pytest.mark.gpu
@pytest.mark.parametrize("cache,rows", [("bf16", "f32"), ("e4m3", "bf16"), ("f32", "bf16")])
def test_gather_latent_without_begin(cache, rows):
    B = Batch([65, 1, 128, 300], [1, 1, 1, 1], kind="mla", heads=1, dim=576, page=64, cache=cache, seed=30)
    at = np.concatenate([[0], np.cumsum(B.seq)]).astype(np.int32)
    ind = torch.from_numpy(at).cuda()
    n = int(at[-1])
    lat, rope = torch.empty(n, 512, dtype=ROW[rows], device="cuda"), torch.empty(n, 64, dtype=ROW[rows], device="cuda")
    whole = torch.empty(n, 576, dtype=ROW[rows], device="cuda")
    skv.kv_gather(B.problem, ind, lat, rope)
    skv.kv_gather(B.problem, ind, whole)
    torch.cuda.synchronize()
    want = torch.cat([decode(B.k[B.slots(b, 0, B.seq[b])], cache, K_SCALE, rows) for b in range(4)])
    assert same(whole, want) and same(lat, want[:, :512]) and same(rope, want[:, 512:])


@pytest.mark.gpu
def test_gather_refuses_positions_past_the_length():
    B = Batch([20, 20], [1, 1], cache="bf16", seed=31)
    at = torch.tensor([0, 21, 41], dtype=torch.int32, device="cuda")   # one token more than request 0 has
    k, v = (torch.full((41, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.kv_gather(B.problem, at, k, v, None, err)
    st, _ = skv.read_device_error(err)
    assert st == skv.ERR_DEVICE_CHECK
    page, slot = B.slots(0, 0, 20)
    assert same(k[:20], B.k[page, :, slot]) and (k[20] == 0).all()
    page, slot = B.slots(1, 0, 20)
    assert same(v[21:], B.v[page, :, slot])


@pytest.mark.gpu
def test_append_then_gather_on_another_stream():
    B = Batch([300, 41], [300, 41], heads=4, dim=64, page=16, cache="e4m3", seed=32)
    k, v = (torch.randn(341, 4, 64).bfloat16() for _ in range(2))
    kd, vd = k.cuda(), v.cuda()
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    ind = torch.from_numpy(np.array([0, 300, 341], np.int32)).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    skv.kv_append(B.problem, kd, vd, stream=s)
    skv.kv_gather(B.problem, ind, ko, vo, stream=s)
    s.synchronize()
    assert same(ko, decode(encode(k, "e4m3", K_SCALE), "e4m3", K_SCALE, "bf16"))
    assert same(vo, decode(encode(v, "e4m3", V_SCALE), "e4m3", V_SCALE, "bf16"))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    # an E4M3 pool of 4.3 GB (8 heads, 64 x 128 pages): the request's pages lie at its two ends
    heads, page, dim = 8, 64, 128
    pages = 2 ** 32 // (heads * page * dim) + 600
    pool = torch.zeros(pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    T = 150
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    prob = skv.AttentionProblem(
        q=torch.empty(T, heads, dim, dtype=torch.bfloat16, device="cuda"), k_cache=pool, v_cache=pool.clone(), page_table=table,
        seq_lens=i32([T]), qo_indptr=i32([0, T]), num_q_heads=heads, num_kv_heads=heads, head_dim_qk=dim, head_dim_v=dim,
        page_size=page, scale=0.1, k_scale=K_SCALE, v_scale=V_SCALE)
    k, v = (torch.randn(T, heads, dim).bfloat16() for _ in range(2))
    skv.kv_append(prob, k.cuda(), v.cuda())
    want = encode(k[:64], "e4m3", K_SCALE).transpose(0, 1)
    assert same_codes(pool[pages - 1], want)
    ko, vo = torch.empty(T, heads, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(T, heads, dim, dtype=torch.bfloat16, device="cuda")
    skv.kv_gather(prob, i32([0, T]), ko, vo)
    torch.cuda.synchronize()
    assert same(ko, decode(encode(k, "e4m3", K_SCALE), "e4m3", K_SCALE, "bf16"))
    assert same(vo, decode(encode(v, "e4m3", V_SCALE), "e4m3", V_SCALE, "bf16"))


# ------------------------------------------------------------------ refusals (no GPU needed)
def _cpu(**kw):
    return Batch([20, 20], [2, 1], dev="cpu", **kw)


def _refused(status, call, *args, **kw):
    with pytest.raises(skv.SplitKVError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value
    return str(e.value)


def test_row_shapes_and_types_are_checked():
    B = _cpu()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    ind = torch.zeros(3, dtype=torch.int32)
    for bad in (k[:2], k[:, :1], torch.zeros(3, 2, 63, dtype=torch.bfloat16), k.view(3, 128)):
        with pytest.raises(TypeError):
            skv.kv_append(B.problem, bad, bad)
    with pytest.raises(TypeError):
        skv.kv_append(B.problem, k, None)
    with pytest.raises(TypeError):
        skv.kv_append(B.problem, k, k.float())
    with pytest.raises(TypeError):
        skv.kv_append(B.problem, k.half(), k.half())
    with pytest.raises(TypeError):
        skv.kv_append(B.problem, torch.zeros(3, 2, 128, dtype=torch.bfloat16)[..., ::2], k)
    with pytest.raises(TypeError):
        skv.kv_gather(B.problem, ind[:2], k, k)
    with pytest.raises(TypeError):
        skv.kv_gather(B.problem, ind.long(), k, k)
    with pytest.raises(TypeError):
        skv.kv_gather(B.problem, ind, k, k, ind)


def test_host_memory_is_refused():
    B = _cpu()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    _refused(skv.ERR_INVALID_ARG, skv.kv_append, B.problem, k, k)
    _refused(skv.ERR_INVALID_ARG, skv.kv_gather, B.problem, torch.zeros(3, dtype=torch.int32), k, k)


def test_overlapping_output_rows_are_refused():
    B = _cpu()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    ind = torch.zeros(3, dtype=torch.int32)
    one = torch.zeros(1, 2, 64, dtype=torch.bfloat16).expand(3, 2, 64)
    assert "overlap" in _refused(skv.ERR_INVALID_ARG, skv.kv_gather, B.problem, ind, one, k)
    heads = torch.zeros(3, 1, 64, dtype=torch.bfloat16).expand(3, 2, 64)
    assert "overlap" in _refused(skv.ERR_INVALID_ARG, skv.kv_gather, B.problem, ind, k, heads)


def test_lengths_and_the_problem_are_checked_first():
    B = _cpu()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    bad = B.make_problem(seq_lens_host=[1, 20])          # q_len 2 > seq_len 1
    assert "q_len" in _refused(skv.ERR_INVALID_ARG, skv.kv_append, bad, k, k)
    f = Batch([20], [1], dev="cpu", cache="e4m3")
    f32 = f.make_problem(q=torch.zeros(1, 2, 64))
    _refused(skv.ERR_UNSUPPORTED, skv.kv_append, f32, k[:1], k[:1])


def test_no_rows_is_no_work():
    B = Batch([20, 20], [0, 0], dev="cpu")
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16)
    skv.kv_append(B.problem, k, k)
    skv.kv_gather(B.problem, torch.zeros(3, dtype=torch.int32), k, k)
