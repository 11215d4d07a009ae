"""Listed keys of heads of every width where a warp gathers one unit of a list right behind another: clusters of two
CTAs, and single CTAs, that take a list of 2048 each."""

import pytest
import torch

from fp4_case import Case, choose

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [45, 100])
@pytest.mark.parametrize("hq,dim", [(4, 16), (12, 32), (8, 48), (4, 64), (4, 80), (16, 80), (24, 96), (8, 112), (4, 128)])
def test_units_gathered_one_behind_the_other(cuda_lib, hq, dim, rows):
    assert 2048 // 64 > 12 * 2 and 8 * 45 > 152 >= rows          # more units than warps, fewer items than CTAs
    c = Case([2500], [rows], hq=hq, hkv=1, dim=dim, dtype="fp16", seed=dim)
    topk = choose(c, 2048, seed=rows)
    got = c.selected(cuda_lib, topk)
    c.check(got, topk)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(got, c.selected(cuda_lib, topk)))
