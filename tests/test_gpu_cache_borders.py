"""kv_append where test_gpu_cache_rows does not look: scales whose quotients come closest to a border between two
codes.  Exact, as there."""
import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv
from tests.test_gpu_cache_rows import _ALL, Batch, encode, same_codes


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
