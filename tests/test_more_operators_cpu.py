"""Arguments that the block-scaled cache, assign_pages and sample_tokens refuse, before anything reaches a
device (no GPU needed), and the binding's packed structures against the header's."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import long_context_split_gb300 as skv
from long_context_split_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def problem(page=64, block=16, heads=2, dim=128, pages=4, kind="gqa", **over):
    kw = dict(q=torch.zeros(1, heads, dim, dtype=torch.bfloat16), k_cache=torch.zeros(pages, heads, page, dim, dtype=torch.uint8),
              v_cache=torch.zeros(pages, heads, page, dim, dtype=torch.uint8), page_table=i32(1, 4),
              seq_lens=torch.tensor([100], dtype=torch.int32), qo_indptr=torch.tensor([0, 1], dtype=torch.int32), num_q_heads=heads,
              num_kv_heads=heads, head_dim_qk=dim, head_dim_v=dim, page_size=page, scale=0.1, kind=kind,
              k_scale=torch.ones(pages, heads, page // block), v_scale=torch.ones(pages, heads, page // block))
    kw.update(over)
    return skv.AttentionProblem(**kw)


def test_structures_match_the_header():
    """Field offsets and sizes as a C compiler lays them out."""
    code = r"""
#include <stdio.h>
#include "splitkv.h"
int main(void) {
    printf("%zu %zu %zu %zu %zu %zu %zu\n", sizeof(splitkv_problem), offsetof(splitkv_problem, k_block_scales),
           offsetof(splitkv_problem, scale_block), sizeof(splitkv_pages), offsetof(splitkv_pages, num_slots),
           sizeof(splitkv_sample), offsetof(splitkv_sample, probs_stride));
    return 0;
}
"""
    exe = os.path.join(ROOT, "long_context_split_gb300", "_build", "layout_test")
    os.makedirs(os.path.dirname(exe), exist_ok=True)
    subprocess.run(["gcc", "-x", "c", "-", "-I", os.path.join(ROOT, "include"), "-o", exe], input=code, text=True, check=True)
    got = list(map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()))
    P = _lib.Problem
    assert got == [ctypes.sizeof(P), P.k_block_scales.offset, P.scale_block.offset, _lib._PAGES.size, _lib._PAGES.size - 8,
                   _lib._SAMPLE.size, _lib._SAMPLE.size - 8]


def test_block_scales_of_wrong_shapes_and_types():
    ok = torch.ones(4, 2, 4)
    problem()
    for k, v in ((ok, 0.5), (0.5, ok), (ok, torch.ones(4, 2, 2)), (ok.double(), ok.double()), (ok[:, :1], ok[:, :1]),
                 (torch.ones(4, 2, 3), torch.ones(4, 2, 3)), (ok.transpose(1, 2).contiguous().transpose(1, 2), ok), (ok[0], ok[0])):
        with pytest.raises(TypeError):
            problem(k_scale=k, v_scale=v)
    with pytest.raises(TypeError, match="come with"):
        problem(k_cache=torch.zeros(4, 2, 64, 128, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="GQA"):
        problem(kind="mla", heads=1)
    # numbers, also as tensors of one entry, stay one scale per tensor
    assert problem(k_scale=torch.tensor(0.5), v_scale=0.25).scale_block == 0
    assert problem(k_scale=torch.tensor([0.5]), v_scale=torch.tensor([0.25])).k_scale == 0.5


@pytest.mark.parametrize("page,block", [(64, 8), (256, 256), (64, 1), (96, 48)])
def test_block_sizes_without_a_kernel(page, block):
    p = problem(page=page, block=block)
    with pytest.raises(skv.SplitKVError, match="scale_block") as e:
        skv.splitkv_plan(p)
    assert e.value.status == skv.ERR_INVALID_ARG
    with pytest.raises(skv.SplitKVError, match="scale_block"):
        skv.kv_append(p, torch.zeros(1, 2, 128), torch.zeros(1, 2, 128))


def test_block_scaled_problems_that_no_kernel_takes():
    with pytest.raises(skv.SplitKVError) as e:
        skv.splitkv_plan(problem(dim=72))
    assert e.value.status == skv.ERR_UNSUPPORTED
    p = problem(q=torch.zeros(1, 2, 128))
    with pytest.raises(skv.SplitKVError) as e:
        skv.splitkv_plan(p)
    assert e.value.status == skv.ERR_UNSUPPORTED
    with pytest.raises(skv.SplitKVError, match="BF16"):
        skv.kv_append(p, torch.zeros(1, 2, 128), torch.zeros(1, 2, 128))
    p = problem()
    p._s.kv_fp8 = 3
    with pytest.raises(skv.SplitKVError, match="kv_fp8"):
        skv.splitkv_plan(p)
    p._s.kv_fp8, p._s.reserved1 = 2, 1
    with pytest.raises(skv.SplitKVError, match="reserved1"):
        skv.splitkv_plan(p)


def test_problems_without_block_scales_do_not_read_the_new_fields():
    """A caller compiled before those fields existed passes a shorter structure."""
    p = problem(k_scale=0.5, v_scale=0.5)
    p._s.k_block_scales, p._s.scale_block, p._s.reserved1 = 0x1234, 77, 99
    assert skv.splitkv_plan(p).kernel_path == 1


def test_plans_of_both_kinds_of_scale_do_not_mix():
    blocks, one = problem(), problem(k_scale=0.5, v_scale=0.5)
    plan = skv.splitkv_plan(blocks)
    ws, out = torch.zeros(256, dtype=torch.uint8), torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(skv.SplitKVError, match="plan"):
        skv.splitkv_decode(one, plan, ws, out)


def test_host_memory_is_refused():
    p = problem()
    with pytest.raises(skv.SplitKVError):
        skv.kv_append(p, torch.zeros(1, 2, 128), torch.zeros(1, 2, 128))
    with pytest.raises(skv.SplitKVError):
        skv.assign_pages(i32(2, 4), i32(2), i32(2), i32(8), i32(1), page_size=16)
    with pytest.raises(skv.SplitKVError):
        skv.sample_tokens(torch.zeros(2, 10), torch.zeros(2))


def pages(**over):
    kw = dict(page_table=i32(2, 4), held=i32(2), seq_lens=i32(2), free_pages=i32(8), free_count=i32(1), page_size=16)
    kw.update(over)
    skv.assign_pages(kw.pop("page_table"), kw.pop("held"), kw.pop("seq_lens"), kw.pop("free_pages"), kw.pop("free_count"), **kw)


def test_pages_refusals():
    for over in (dict(page_table=i32(3, 4)), dict(page_table=i32(4, 4)[::2]), dict(held=i32(2).long()), dict(seq_lens=i32(3)),
                 dict(free_count=i32(2)), dict(free_pages=i32(8, 2)[:, 0]), dict(held_out=i32(1)), dict(free_count_out=i32(0)),
                 dict(qo_indptr=i32(3)), dict(slots=i32(4).long()), dict(qo_indptr=i32(2), slots=i32(4).long()),
                 dict(qo_indptr=i32(3), slots=i32(4))):
        with pytest.raises(TypeError):
            pages(**over)
    for over, text in ((dict(page_size=0), "page_size"), (dict(free_pages=i32(0)), "capacity"),
                       (dict(page_table=i32(2, 0)), "max_pages")):
        with pytest.raises(skv.SplitKVError, match=text) as e:
            pages(**over)
        assert e.value.status == skv.ERR_INVALID_ARG
    n = 8193
    with pytest.raises(skv.SplitKVError) as e:
        pages(page_table=i32(n, 1), held=i32(n), seq_lens=i32(n))
    assert e.value.status == skv.ERR_UNSUPPORTED


def test_sample_refusals():
    x, u, f = torch.zeros(2, 10), torch.zeros(2), torch.zeros
    for args, over in (((x.half(), u), {}), ((f(10, 2).T, u), {}), ((x, f(3)), {}), ((x, u.double()), {}), ((x, None), {}),
                       ((x, None), dict(out_tokens=i32(2))), ((x, u), dict(out_tokens=i32(2).long())),
                       ((x, u), dict(temperature=f(1))), ((x, u), dict(top_k=f(2))), ((x, u), dict(top_p=i32(2))),
                       ((x, u), dict(min_p=f(2).double())), ((x, u), dict(probs_out=f(2, 9))), ((x, u), dict(probs_out=f(2, 10).double())),
                       ((x, u), dict(probs_out=f(10, 2).T))):
        with pytest.raises(TypeError):
            skv.sample_tokens(*args, **over)
    for shape, text in (((2, 0), "vocab"), ((1, (1 << 19) + 1), "vocab")):
        with pytest.raises(skv.SplitKVError, match=text):
            skv.sample_tokens(torch.zeros(shape), f(shape[0]))
    with pytest.raises(skv.SplitKVError, match="overlap"):
        skv.sample_tokens(x, None, probs_out=x)
    # no rows: nothing to do
    assert skv.sample_tokens(f(0, 10), f(0)).numel() == 0


def test_exported_names():
    text = open(os.path.join(ROOT, "include", "splitkv.h")).read()
    n = int(re.search(r"SPLITKV_KERNEL_COUNT = (\d+)", text).group(1))
    assert len(skv.KERNEL_NAMES) == n
    assert skv.KERNEL_NAMES[-2:] == ["assign_pages_kernel", "sample_tokens_kernel"]
    assert callable(skv.assign_pages) and callable(skv.sample_tokens) and sys.modules["long_context_split_gb300"]
