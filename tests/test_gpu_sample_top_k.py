"""top_k around the largest k whose candidates come from the lanes' maxima (280 with one CTA a row, 440, 510, 560, 600 and
640 with more), at every number of CTAs."""
import pytest
import torch

from tests.test_gpu_sample import check, logits_of, uniform

pytestmark = pytest.mark.gpu
K = [200, 201, 256, 280, 281, 440, 441, 510, 511, 560, 561, 600, 601, 640, 641, 1100, 2500]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("slope", [0.0, 1.5])
@pytest.mark.parametrize("V", [3000, 8000, 12000, 16000, 20000, 24000, 28000, 32768])     # 1 to 8 CTAs
def test_top_k_of_some_hundreds(V, slope, dtype):
    n = len(K)
    x = logits_of(n, V, seed=V + n, slope=slope, dtype=dtype)
    check(x, uniform(n, V + 1), k=K)
    check(x, uniform(n, V + 2), k=K, p=[0.9] * n, t=[0.8] * n)


@pytest.mark.parametrize("V", [3000, 32768])
def test_candidates_in_one_segment(V):
    """The largest logits side by side, so that few lanes hold them all, and equal logits at the cut."""
    x = logits_of(len(K), V, seed=5, dtype=torch.float32)
    x[:, 100:900] += 8.0
    check(x, uniform(len(K), 6), k=K)
    x[:, 1000:] = -3.0
    check(x, uniform(len(K), 7), k=K, mp=[1e-6] * len(K))
