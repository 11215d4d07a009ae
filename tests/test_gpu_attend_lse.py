"""The log-sum-exp where it is small: a key of score zero and one far below it, log(1 + exp(s)).

The sum of the weights is one rounding of FP32 (2^-24) off, the small weight 2^-22 of itself and, by its exponent's
rounding, 2^-22 |s|; the logarithm and its product with ln 2 are 2^-22 of themselves off.  FP16 weights are kept 2^7
larger, and the logarithm of such a sum is rounded to 2^-22."""

import numpy as np
import pytest
import torch

from attend_case import DT, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 1), (40, 1)])      # narrow tiles of 8 and 16 rows, wide ones
def test_a_small_log_sum_exp(cuda_lib, hq, hkv, dtype):
    n = 500
    c = Case([2] * n, [1] * n, hq=hq, hkv=hkv, dim=64, dtype=dtype)
    c.q.fill_(1.0)
    k1 = (-torch.linspace(0.01, 1.9, n, device="cuda")).to(DT[dtype])   # scores 64 k1 / 8
    pages = c.block_table[:, 0].long()
    c.k[pages, 0] = 0.0
    c.k[pages, 1] = k1[:, None, None]
    lse = c.paged(cuda_lib)[1].double().cpu().numpy()
    s = 8.0 * k1.double().cpu().numpy()
    w = np.exp(s)
    want = np.log1p(w)
    tol = 2.0 ** -24 + w * 2.0 ** -22 * (1 + np.abs(s)) + 2.0 ** -22 * want + (2.0 ** -22 if dtype == "fp16" else 0.0)
    assert (np.abs(lse - want[:, None]) <= tol[:, None]).all(), (np.abs(lse - want[:, None]) / tol[:, None]).max()
