"""The 4-bit attention under block tables wider than the requests need, over lists that are sparse in long contexts,
and the cache read back into a paged 16-bit one that the 16-bit attention then reads."""

import numpy as np
import pytest
import torch

from fp4_case import DT, Case, choose
from oracle import attention as A
from oracle import fp4_cache as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [385, 2048, 20000])
@pytest.mark.parametrize("lens,qlens,hq,hkv,dim", [([1000], [1], 32, 8, 128), ([130 + 90 * j for j in range(9)], [2] * 9, 8, 2, 64),
                                                   ([40 * j for j in range(70)], [1] * 70, 6, 2, 80)])
def test_short_requests_under_a_wide_table(cuda_lib, lens, qlens, hq, hkv, dim, pages):
    c = Case(lens, qlens, hq=hq, hkv=hkv, dim=dim, pad_rows=1)
    wide = torch.full((len(lens), pages), 10 ** 9, dtype=torch.int32, device="cuda")     # (no page)
    wide[:, :c.block_table.shape[1]] = c.block_table
    topk = choose(c, 90)
    c.block_table = wide
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(c.paged(cuda_lib, status=status))
    c.check(c.selected(cuda_lib, topk, status=status), topk)
    assert int(status) == 0


def test_sparse_lists_put_in_order(cuda_lib):
    """Two positions a page; each row a list of its own over the same request."""
    rows, k = 70, 2048
    c = Case([70000], [rows], hq=8, hkv=4, dim=64, dtype="fp16")
    assert rows * 4 * (k // 64) * F.section_bytes(64) >= 32 << 20
    topk = choose(c, k, holes=False)
    got = c.selected(cuda_lib, topk)
    c.check(got, topk, rows=range(0, rows, 7))
    again = c.selected(cuda_lib, topk.flip(1).contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_lists_over_more_positions_than_are_put_in_order(cuda_lib):
    rows, k, n = 700, 2048, (1 << 20) + 4000
    c = Case([n], [rows], hq=4, hkv=1, dim=16)
    assert rows * (k // 64) * F.section_bytes(16) >= 32 << 20
    rng = np.random.default_rng(4)
    topk = torch.from_numpy(rng.integers(0, n - rows, (rows, k))).to(torch.int32).cuda()
    topk[:, 5] = torch.arange(n - rows, n, dtype=torch.int32)              # each row's last key
    c.check(c.selected(cuda_lib, topk), topk, rows=range(0, rows, 60))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,dim", [(32, 8, 128), (10, 2, 80), (4, 1, 64)])
def test_read_back_into_a_paged_cache(cuda_lib, hq, hkv, dim, dtype):
    """A prompt's later rows: the context read back once, then 16-bit attention over the same pages.  Codes by scales
    by powers of two are exact in both types, so both attentions have the same values."""
    lens, qlens = [700, 90, 333], [300, 90, 1]
    c = Case(lens, qlens, hq=hq, hkv=hkv, dim=dim, dtype=dtype, k_scale=0.5, v_scale=2.0)
    pages = c.cache.shape[0]
    k = torch.zeros((pages, 64, hkv, dim), dtype=DT[dtype], device="cuda")
    v = torch.zeros_like(k)
    need = [-(-n // 64) for n in lens]
    table = c.block_table.cpu().numpy()
    for j, n in enumerate(lens):             # a request's whole pages at a time, past its end too (unseen)
        for p in table[j, :need[j]]:
            slots = torch.arange(64, device="cuda") + int(p) * 64
            cuda_lib.kv_read_fp4(slots, c.cache, dim, DT[dtype], k_out=k[p], v_out=v[p], **c.scales)
    held_k, held_v = F.decode(c.host, dim, **c.scales)
    for j, n in enumerate(lens):
        at = np.arange(n)
        place = (table[j][at // 64], at % 64)
        for got, held in ((k, held_k), (v, held_v)):
            assert np.array_equal(got.double().cpu().numpy()[place], held[place])
    out, lse = cuda_lib.attend_paged(c.q, k, v, c.block_table, c.starts, c.row_ends, c.qlen, want_lse=True)
    q, starts, ends = c.q.double().cpu().numpy(), c.starts.tolist(), c.row_ends.tolist()
    eps, small = torch.finfo(DT[dtype]).eps, 2.0 ** -25 if dtype == "fp16" else 0.0
    out = out.double().cpu().numpy()
    for r in range(0, q.shape[0], 13):
        keys = A.visible(r, starts, ends, table.tolist())
        o, _, mean_abs, size = A.attend(q[r], held_k, held_v, keys, c.scale)
        tol = eps / 2 * np.abs(o) + (eps / 2 + 2.0 ** -20 + 4 * 2.0 ** -24 * (dim + 4) * size[:, None]) * mean_abs
        tol += small + len(keys) * small * 2.0 ** -7 * np.abs(held_v[tuple(np.array(keys).T)]).max()
        assert (np.abs(out[r] - o) <= tol).all(), (r, np.abs(out[r] - o).max())
    c.check(c.paged(cuda_lib), rows=range(0, q.shape[0], 13))
