"""Attention over finite scores so large that a step of FP32 is a factor of two and more between weights.

All columns of a query are one number and all columns of a key another, few bits each.  One key's score (or that of
some equal keys) stands far above all others, so the output is that key's value, or their values' mean, whatever the
scores' own rounding does.  Tolerances: the weight is rounded to the cache's type and so is the output, eps / 2 of
|v| each, and FP32 sums of a few terms stay below 2^-20.  The log-sum-exp is scale times a sum of dim products, each
addition off by 2^-24 of it at most (2^-23 for a truncating one), and five more roundings of it.
"""

import numpy as np
import pytest
import torch

from attend_case import DT, Case

pytestmark = pytest.mark.gpu


def large_case(dtype, sign, tops, **kw):
    """Every row's scores: its keys' numbers are 1 to 900 (times 2^up), the keys at `tops` 1000 to 1023."""
    c = Case(dtype=dtype, seed=5, **kw)
    up = 2 ** 5 if dtype == "fp16" else 2 ** 24
    g = torch.Generator().manual_seed(11)
    pages = c.k.shape[0]
    hkv, dim = c.k.shape[2:]
    num = torch.randint(1, 900, (pages, 64, hkv), generator=g)
    if dtype == "bf16":
        num = num // 8 * 8               # eight bits
    tables = c.block_table.tolist()
    for j, t in tops:
        page = c.prefix_pages[t // 64] if j < 0 else tables[j][t // 64]
        num[int(page), t % 64] = 1016
    live = ~torch.isnan(c.k.float()).cpu()
    c.k.copy_(torch.where(live, (num[..., None] * up).float(), float("nan")).to(c.k.dtype))
    q = torch.randint(129, 255, c.q.shape[:2], generator=g).float() * sign
    c.q = (q[..., None] * (4 if dtype == "fp16" else 2 ** 20)).expand(c.q.shape).to(c.q.device, c.q.dtype).contiguous()
    return c


def check(c, got, keys_of):
    out, lse = (t.double().cpu() for t in got)
    k, v, q = (t.double().cpu() for t in (c.k, c.v, c.q))
    group = q.shape[1] // k.shape[2]
    eps = torch.finfo(DT[c.dtype]).eps
    for r in range(q.shape[0]):
        keys = keys_of(r)
        if not keys:
            continue
        for h in range(q.shape[1]):
            vs = torch.stack([v[p, t, h // group] for p, t in keys])
            want, size = vs.mean(0), vs.abs().mean(0)
            err = (out[r, h] - want).abs()
            assert (err <= (eps + 2.0 ** -20) * size).all(), (r, h, float(err.max()))
            p, t = keys[0]
            score = float((q[r, h] * k[p, t, h // group]).sum()) * c.scale
            assert abs(float(lse[r, h]) - score - np.log(len(keys))) <= 2.0 ** -23 * (q.shape[2] + 5) * abs(score), (r, h)


FORMS = [dict(hq=8, hkv=2, dim=64), dict(hq=16, hkv=1, dim=128), dict(hq=40, hkv=2, dim=64), dict(hq=64, hkv=1, dim=128)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f['hq']}x{f['dim']}")
def test_one_key_far_above_the_others(cuda_lib, form, dtype):
    tops = [(0, 3), (1, 250), (2, 1337)]
    c = large_case(dtype, 1, tops, lens=[60, 300, 4000], qlens=[1, 1, 1], **form)
    tables = c.block_table.tolist()
    at = {j: [(tables[j][t // 64], t % 64)] for j, t in tops}
    check(c, c.paged(cuda_lib), lambda r: at[r])
    topk = torch.tensor([[t if i == 77 else (i * 7) % 60 for i in range(300)] for _, t in tops], dtype=torch.int32).cuda()
    check(c, c.selected(cuda_lib, topk), lambda r: at[r] if r else [])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f['hq']}x{f['dim']}")
def test_equal_keys_share_the_weight_across_tiles_and_pieces(cuda_lib, form, dtype):
    tops = [(0, t) for t in (5, 6, 40, 130, 700, 2999, 3000, 9999)]
    c = large_case(dtype, 1, tops, lens=[10000], qlens=[1], **form)
    table = c.block_table.tolist()[0]
    check(c, c.paged(cuda_lib), lambda r: [(table[t // 64], t % 64) for _, t in tops])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f['hq']}x{f['dim']}")
def test_behind_a_prefix(cuda_lib, form, dtype):
    """The largest score among the prefix's keys, own keys far below it, and the other way round."""
    for tops in ([(-1, 400)], [(0, 100), (1, 20), (2, 0)]):
        c = large_case(dtype, 1, tops, lens=[150, 21, 1], qlens=[1, 1, 1], prefix=1000, **form)
        tables, shared = c.block_table.tolist(), c.prefix_pages.tolist()
        at = {j: [(shared[t // 64] if j < 0 else tables[j][t // 64], t % 64)] for j, t in tops}
        check(c, c.paged(cuda_lib), lambda r: at[-1] if -1 in at else at[r])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_scores_far_below_zero(cuda_lib, dtype):
    """One key: its weight is one however far below zero its score is."""
    c = large_case(dtype, -1, [(0, 0)], lens=[1], qlens=[1], hq=8, hkv=2, dim=64)
    page = c.block_table.tolist()[0][0]
    check(c, c.paged(cuda_lib), lambda r: [(page, 0)])
