"""FP16 attention over many keys, to a tolerance in which a lost tile of values shows.

Stored weights are 2^7 larger than relative to the running reference, which is some key's score of the same tiles or
at most 2^8 below the largest: the largest stored weight is 2^7 or more.  A stored weight below 2^-14 is off by at
most 2^-25, so by 2^-32 of the largest, and all of them move an output by at most 2^-32 max |v| a key.  Larger weights
and the output are off by eps / 2 of themselves, outputs below 2^-14 by 2^-25, and FP32 adds what attend_case counts.
"""

import numpy as np
import pytest
import torch

from attend_case import Case, choose
from oracle import attention as A

EPS = torch.finfo(torch.float16).eps


def row(c, r, topk=None, lost=()):
    """The row's output in 64 bits and its tolerance; `lost`: keys whose values count as zeros."""
    k, v, q = c.host
    keys = A.visible(r, c.starts.tolist(), c.row_ends.tolist(), c.block_table.tolist(), c.prefix_pages.tolist(),
                     0 if topk is not None else c.prefix_len, None if topk is None else topk.tolist())
    if len(lost):
        v = v.copy()
        for i in lost:
            v[keys[i]] = 0.0
    o, _, mean_abs, size = A.attend(q[r], k, v, keys, c.scale)
    vmax = np.abs(v[tuple(np.array(keys).T)]).max()
    moved = 2.0 ** -24 * (q.shape[2] + 4) * size
    tol = EPS / 2 * np.abs(o) + (EPS / 2 + 2.0 ** -20 + 4 * moved[:, None]) * mean_abs
    return o, tol + len(keys) * 2.0 ** -32 * vmax + 2.0 ** -25, len(keys)


def on_host(c):
    c.host = [t.double().cpu().numpy() for t in (c.k, c.v, c.q)]
    return c


@pytest.mark.parametrize("hq,hkv,prefix,dim,places", [(7, 7, 33793, 16, 27), (64, 2, 12001, 128, 4),
                                                      (128, 1, 7301, 64, 4)])
def test_a_lost_tile_of_values_is_outside_the_tolerance(hq, hkv, prefix, dim, places):
    """128 keys' values taken out of the 64-bit form, at some places along the prefix."""
    c = on_host(Case([40], [1], prefix=prefix, hq=hq, hkv=hkv, dim=dim, dtype="fp16", seed=6, device="cpu"))
    o, tol, n = row(c, 0)
    for tile in np.linspace(0, prefix // 128 - 1, places).astype(int):
        without, _, _ = row(c, 0, lost=range(128 * tile, 128 * tile + 128))
        assert (np.abs(without - o) > tol).any(), tile


def check(c, got, rows, topk=None):
    out = got[0].double().cpu().numpy()
    for r in rows:
        o, tol, n = row(c, r, topk)
        assert (np.abs(out[r] - o) <= tol).all(), (r, n, (np.abs(out[r] - o) / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,rows,prefix,dim,layout", [
    (7, 7, 129, 33793, 16, "odd"), (64, 2, 81, 12001, 128, "hnd"), (128, 1, 65, 7301, 64, "nhd"),   # pairs of row tiles
    (8, 2, 3, 33793, 64, "nhd"), (40, 2, 5, 20000, 128, "pair")])                                  # prefixes on the axis
def test_long_prefixes(cuda_lib, hq, hkv, rows, prefix, dim, layout):
    lens = [(37 * j) % 150 for j in range(rows)]
    c = on_host(Case(lens, [1] * rows, prefix=prefix, hq=hq, hkv=hkv, dim=dim, dtype="fp16", layout=layout, seed=6))
    check(c, c.paged(cuda_lib), [1, rows // 2, rows - 2, rows - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (16, 1, 64), (40, 2, 80)])
def test_long_rows_and_lists(cuda_lib, hq, hkv, dim):
    c = on_host(Case([40011, 9000], [1, 3], hq=hq, hkv=hkv, dim=dim, dtype="fp16"))
    check(c, c.paged(cuda_lib), range(4))
    topk = choose(c, 6000)
    check(c, c.selected(cuda_lib, topk), range(4), topk)
