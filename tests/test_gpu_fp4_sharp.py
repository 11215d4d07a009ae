"""Scores of any size over the 4-bit cache: a key that is ahead of all others by more than scores are rounded takes
all the weight, and no weight passes FP16, however far FP32 rounds the scores."""

import math

import numpy as np
import pytest
import torch

from fp4_case import DT, Case
from oracle import attention as A
from oracle import fp4_cache as F

pytestmark = pytest.mark.gpu

FORMS = [(4, 1), (16, 1), (32, 1)]      # tiles of 8, 16 and 32 rows


@pytest.mark.parametrize("heat", [1e3, 1e6, 1e7, 1e8, 1e9])
@pytest.mark.parametrize("lens", [[300, 65], [20000, 64]], ids=str)
@pytest.mark.parametrize("hq,hkv,dim", [(hq, hkv, dim) for hq, hkv in FORMS for dim in (64, 128)])
def test_one_key_takes_all_the_weight(cuda_lib, hq, hkv, dim, lens, heat):
    c = Case(lens, [1, 1], hq=hq, hkv=hkv, dim=dim, heat=heat)
    k, v = F.decode(c.host, dim)
    out, lse = c.paged(cuda_lib)
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    out, q, sure = out.double().cpu().numpy(), c.q.double().cpu().numpy(), 0
    for r, n in enumerate(lens):
        pages, t = c.block_table[r].cpu().numpy(), np.arange(n)
        keys, values = k[pages[t // 64], t % 64, 0], v[pages[t // 64], t % 64, 0]
        score = q[r] @ keys.T * c.scale
        size = np.abs(q[r]) @ np.abs(keys).T * c.scale
        first, second = np.argsort(score, axis=1)[:, -1], np.sort(score, axis=1)[:, -2]
        # two scores, each off by its sum's roundings, and as many again where pieces are joined; the rest of the
        # keys together below 2^-20
        off = 4 * 2.0 ** -24 * (dim + 4) * size.max(axis=1)
        alone = score.max(axis=1) - second > off + math.log(n) + 20 * math.log(2.0)
        want = values[first]
        tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -19) * np.abs(want) + 2.0 ** -19 * np.abs(values).max()
        assert (np.abs(out[r] - want) <= tol)[alone].all(), (r, np.abs(out[r] - want)[alone].max())
        sure += int(alone.sum())
    assert sure >= hq                    # of 2 hq


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv", FORMS)
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_a_score_a_step_of_fp32_ahead(cuda_lib, hq, hkv, dim, dtype):
    """Ten requests under eight key heads: a CTA each, whose first warp has keys 0 and 24 * 64 + 5 whatever the warps.
    The queries' first column is 1 (2^14 inside) and meets 2688 in both keys, so their scores are near 21 * 2^21, where
    a step of FP32 is 4; the second key is ahead by that step, 11.2 powers of two under the scale taken.  Products and
    sums are exact in FP32.  The other keys score 0."""
    c = Case([25 * 64] * 10, [1] * 10, hq=8 * hq, hkv=8 * hkv, dim=dim, dtype=dtype)
    kc, vc, ks, vs = F.views(c.host, dim)
    kc[:], ks[:], vs[:] = 0, 0x38, 0x38
    for table in c.block_table.cpu().numpy():
        for key in (0, 24 * 64 + 5):
            page, t = table[key // 64], key % 64
            kc[page, t, :, 0], ks[page, t, :, 0] = 0x7, 0x7E              # 6 * 448
            kc[page, t, :, 8] = 0x2 if key else 0                         # column 16: 1
    c.cache.copy_(torch.from_numpy(c.host))
    c.q.zero_()
    c.q[:, :, 0], c.q[:, :, 16] = 1.0, 2.0 ** -12
    gap = 4 * 2.8                                                         # powers of two
    scale = 2.8 * 2.0 ** 14 * math.log(2.0)
    out, _ = c.paged(cuda_lib, scale=scale)
    _, v = F.decode(c.host, dim)
    for r, table in enumerate(c.block_table.cpu().numpy()):
        a, b = v[table[0], 0], v[table[24], 5]                            # [key heads, dim]
        w = 2.0 ** -gap / (1 + 2.0 ** -gap)
        want = np.repeat(b * (1 - w) + a * w, hq, axis=0)
        # the scale's own roundings move the gap by at most 2^-22 of it; weights to FP16, the output
        eps = torch.finfo(DT[dtype]).eps
        tol = eps / 2 * np.abs(want) + (2.0 ** -11 + 2.0 ** -19) * np.repeat(np.abs(b) + np.abs(a) * w, hq, axis=0)
        tol += 2.0 ** -25
        got = out[r].double().cpu().numpy()
        assert (np.abs(got - want) <= tol).all(), (r, np.abs(got - want).max())
