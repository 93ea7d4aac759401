"""kv_append and kv_gather where test_gpu_cache_rows does not look: scales whose quotients come closest to a border
between two codes, and float32 rows (or caches) on 16-byte but not 32-byte boundaries.  Exact, as there."""
import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv
from tests.test_gpu_cache_rows import _ALL, K_SCALE, ROW, V_SCALE, Batch, awkward, decode, encode, same, same_codes


@pytest.mark.gpu
def test_scales_near_the_borders_own_multiples():
    B = Batch([64], [64], cache="e4m3", heads=8, dim=128, page=64, seed=40)
    page, slot = B.slots(0, 0, 64)
    borders = (_ALL[1:] + _ALL[:-1]) / 2
    for k in range(8, 16):
        for d in (-3, -2, -1, 1, 2, 3):
            mantissa = (k << 20) + d
            if mantissa < 1 << 23:
                continue
            scale = np.float32(mantissa * 2.0 ** (-23 - (k % 5)))
            at = torch.from_numpy(borders * np.float64(scale)).float()
            up, down = [at], [at]
            for _ in range(4):
                up.append(torch.nextafter(up[-1], torch.full((), 3e38)))
                down.append(torch.nextafter(down[-1], torch.zeros(())))
            near = torch.cat(up + down)
            f = torch.zeros(64 * 8 * 128)
            f[:len(near)], f[4000:4000 + len(near)] = near, -near
            f = f.view(64, 8, 128)
            skv.kv_append(B.make_problem(k_scale=float(scale), v_scale=float(scale)), f.cuda(), f.cuda())
            torch.cuda.synchronize()
            want = B.k.clone()
            want[page, :, slot] = encode(f, "e4m3", scale)
            assert same_codes(B.k_dev, want), f"scale {scale!r}"


def _rows_on_16_bytes(shape, dtype, gen):
    """A slice of a wider tensor whose rows start 16 bytes past a 32-byte boundary, every second one on it."""
    x = awkward(torch.randn(shape, generator=gen).to(dtype))
    step = 16 // x.element_size()
    wide = torch.zeros(shape[0], shape[1] * shape[2] + 3 * step, dtype=dtype, device="cuda")
    d = wide[:, step:step + shape[1] * shape[2]].view(shape)
    d.copy_(x)
    assert d.data_ptr() % 32 == 16 and d.stride(0) * d.element_size() % 16 == 0
    return d, x


@pytest.mark.gpu
@pytest.mark.parametrize("heads,dim,page", [(2, 64, 16), (3, 8, 5), (1, 128, 64)])
@pytest.mark.parametrize("cache,rows", [("f32", "f32"), ("bf16", "f32"), ("e4m3", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_rows_on_16_byte_boundaries(cache, rows, heads, dim, page):
    B = Batch([1, 40, 17, 200, 64], [1, 37, 0, 70, 64], cache=cache, heads=heads, dim=dim, page=page, seed=50)
    T, g = int(B.qo[-1]), torch.Generator().manual_seed(51)
    kd, k = _rows_on_16_bytes((T, heads, dim), ROW[rows], g)
    vd, v = _rows_on_16_bytes((T, heads, dim), ROW[rows], g)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.kv_append(B.problem, kd, vd, err)
    assert skv.read_device_error(err) == (skv.OK, 0)
    after = B.write(k, v)
    B.check(*after)
    # the same tokens back, into other rows of that layout, one of them behind the last request
    ko, kx = _rows_on_16_bytes((T + 1, heads, dim), ROW[rows], g)
    vo, vx = _rows_on_16_bytes((T + 1, heads, dim), ROW[rows], g)
    begin = [n - t for n, t in zip(B.seq, B.new)]
    for b in range(len(B.seq)):
        lo, hi = B.qo[b], B.qo[b + 1]
        at = B.slots(b, begin[b], B.seq[b])
        kx[lo:hi], vx[lo:hi] = (decode(c[at[0], :, at[1]], cache, s, rows) for c, s in zip(after, (K_SCALE, V_SCALE)))
    skv.kv_gather(B.problem, torch.from_numpy(B.qo).cuda(), ko, vo, torch.tensor(begin, dtype=torch.int32, device="cuda"), err)
    assert skv.read_device_error(err) == (skv.OK, 0)
    assert same(ko, kx) and same(vo, vx)


@pytest.mark.gpu
def test_a_float32_cache_on_16_byte_boundaries():
    B = Batch([40, 9], [33, 9], cache="f32", heads=2, dim=64, page=16, seed=52)
    for name in ("k_dev", "v_dev"):
        t = getattr(B, name)
        flat = torch.zeros(t.numel() + 4, device="cuda")
        view = flat[4:].view(t.shape)
        view.copy_(t)
        assert view.data_ptr() % 32 == 16
        setattr(B, name, view)
    g = torch.Generator().manual_seed(53)
    k, v = torch.randn(42, 2, 64, generator=g), torch.randn(42, 2, 64, generator=g)
    skv.kv_append(B.make_problem(), k.cuda(), v.cuda())
    torch.cuda.synchronize()
    B.check(*B.write(k, v))
