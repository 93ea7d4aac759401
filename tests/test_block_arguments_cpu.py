"""Arguments that the calls over block scales and pages take and refuse, without a GPU."""
import pytest
import torch

import long_context_split_gb300 as skv
from tests.test_more_operators_cpu import i32, pages, problem


@pytest.mark.parametrize("shape", [(), (1,), (1, 1), (1, 1, 1), (1, 1, 1, 1)])
def test_scales_of_one_entry_are_numbers(shape):
    """Whatever their dimensions: the cache has more than one block."""
    p = problem(k_scale=torch.full(shape, 0.5), v_scale=torch.full(shape, 0.25))
    assert (p.k_scale, p.v_scale, p.scale_block, p._s.kv_fp8) == (0.5, 0.25, 0, 1)
    p = problem(k_scale=torch.full(shape, 0.5), v_scale=0.25)
    assert (p.k_scale, p.v_scale, p.scale_block) == (0.5, 0.25, 0)
    p = problem(kind="mla", heads=1, v_cache=None, k_scale=torch.full(shape, 0.5), v_scale=torch.full(shape, 0.25))
    assert (p.k_scale, p.scale_block) == (0.5, 0)


def test_the_one_block_of_a_cache_of_one_page_and_head_has_a_block_scale():
    s = torch.ones(1, 1, 1)
    p = problem(pages=1, heads=1, block=64, k_scale=s, v_scale=s.clone())
    assert p.scale_block == 64 and p._s.kv_fp8 == 2
    with pytest.raises(TypeError, match="both"):
        problem(pages=1, heads=1, block=64, k_scale=s, v_scale=0.5)
    assert problem(pages=1, heads=1, block=64, k_scale=torch.ones(1, 1), v_scale=0.5).scale_block == 0


def test_no_slots_come_with_row_bounds():
    """A step without new tokens: an empty slots tensor has no address, and is not refused for it."""
    for over in (dict(), dict(qo_indptr=i32(3), slots=i32(0).long())):
        with pytest.raises(skv.SplitKVError) as e:          # (host memory: refused behind the checks of the arguments)
            pages(**over)
        assert "come together" not in str(e.value) and "page_table" in str(e.value)
