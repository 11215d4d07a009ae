"""Attention over the 4-bit cache on the GPU against the 64-bit formula."""

import numpy as np
import pytest
import torch

from fp4_case import Case, choose, pool
from oracle import fp4_cache as F

pytestmark = pytest.mark.gpu

LENS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 256, 300]
HEADS = [(8, 2, 64), (4, 4, 128), (16, 1, 128), (6, 2, 80), (3, 1, 16), (40, 2, 96), (100, 1, 128), (9, 3, 48),
         (24, 1, 64), (14, 2, 112), (48, 2, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layers", [1, 2])
@pytest.mark.parametrize("hq,hkv,dim", HEADS)
def test_paged_lengths(cuda_lib, hq, hkv, dim, layers, dtype):
    c = Case(LENS, [1] * len(LENS), hq=hq, hkv=hkv, dim=dim, layers=layers, dtype=dtype, pad_rows=2)
    c.check(c.paged(cuda_lib))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("qlens", [[1, 1, 1], [4, 2, 3], [1, 40, 0], [0, 0, 130]])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 64), (16, 2, 128), (5, 1, 96)])
def test_rows_of_a_request(cuda_lib, hq, hkv, dim, qlens, dtype):
    c = Case([70, 200, 333], qlens, hq=hq, hkv=hkv, dim=dim, dtype=dtype, pad_rows=1)
    for hint in (c.qlen, 1, 1000):                       # a hint: the results do not depend on it
        c.check(c.paged(cuda_lib, max_query_len=hint))


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("k", [1, 63, 64, 65, 200])
def test_selected(cuda_lib, hq, hkv, dim, k):
    c = Case(LENS, [1 + j % 3 for j in range(len(LENS))], hq=hq, hkv=hkv, dim=dim, dtype="fp16" if k % 2 else "bf16",
             layers=1 + k % 2, pad_rows=1, ends=None)
    topk = choose(c, k, seed=k)
    c.check(c.selected(cuda_lib, topk), topk)


@pytest.mark.parametrize("k_scale,v_scale", [(0.25, 3.0), (1e-12, 1e10), (1.3e15, 2.0 ** -60)])
def test_scales(cuda_lib, k_scale, v_scale):
    c = Case([100, 500, 3], [2, 1, 1], hq=8, hkv=2, dim=128, k_scale=k_scale, v_scale=v_scale)
    c.check(c.paged(cuda_lib))
    topk = choose(c, 80)
    c.check(c.selected(cuda_lib, topk), topk)
    c.check(c.paged(cuda_lib, scale=0.01), scale=0.01)


@pytest.mark.parametrize("requests", [255, 256, 257, 511, 512, 513, 700])
def test_many_requests(cuda_lib, requests):
    c = Case([(53 * j) % 301 for j in range(requests)], [j % 3 for j in range(requests)], hq=4, hkv=2, dim=64)
    c.check(c.paged(cuda_lib), rows=range(0, c.q.shape[0], 7))
    topk = choose(c, 50)
    c.check(c.selected(cuda_lib, topk), topk, rows=range(0, c.q.shape[0], 7))


def test_many_rows(cuda_lib):
    """More rows than every CTA lays out by itself, in one request and in many."""
    c = Case([4200], [4200], hq=2, hkv=1, dim=64)
    c.check(c.paged(cuda_lib), rows=range(0, 4200, 311))
    c = Case([40] * 300, [16] * 300, hq=2, hkv=1, dim=32)
    c.check(c.paged(cuda_lib), rows=range(0, 4800, 401))


@pytest.mark.parametrize("qlen", [33, 64, 257, 700])
@pytest.mark.parametrize("hq,hkv,dim", [(24, 2, 128), (5, 1, 64)])
def test_rows_of_a_prompt(cuda_lib, hq, hkv, dim, qlen):
    """Even and odd numbers of row tiles, whose bounds rise from the first key to the last, beside short requests."""
    c = Case([qlen, 90, 0, qlen + 300], [qlen, 1, 2, 40], hq=hq, hkv=hkv, dim=dim, pad_rows=3)
    rows = sorted({*range(0, c.q.shape[0], 29), 0, qlen - 1, qlen, c.q.shape[0] - 1})
    c.check(c.paged(cuda_lib), rows=rows)
    topk = choose(c, 100)
    c.check(c.selected(cuda_lib, topk), topk, rows=rows)


@pytest.mark.parametrize("hq,hkv,lens", [(16, 1, [20000] * 2), (32, 8, [9001]), (64, 8, [5000, 10, 7000]),
                                         (12, 4, [30001])])
def test_long(cuda_lib, hq, hkv, lens):
    """Items that many warps share."""
    c = Case(lens, [1] * len(lens), hq=hq, hkv=hkv, dim=128)
    c.check(c.paged(cuda_lib))
    topk = choose(c, 2048)
    c.check(c.selected(cuda_lib, topk), topk)


def test_sharp_scores(cuda_lib):
    """Scores of any size: one key takes all the weight, or a few share it."""
    for heat in (30.0, 1000.0, 1e6):
        c = Case([300, 65], [1, 2], hq=4, hkv=2, dim=64, heat=heat)
        out, lse = c.paged(cuda_lib)
        k, v = F.decode(c.host, 64)
        assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
        # every output is a mean of visible values
        for r, j in ((0, 0), (1, 1), (2, 1)):
            pages = c.block_table[j].cpu().numpy()
            t = np.arange(int(c.row_ends[r]))
            seen = v[pages[t // 64], t % 64]                  # [n, hkv, dim]
            o = out[r].double().cpu().numpy()
            for h in range(4):
                lo, hi = seen[:, h // 2].min(0), seen[:, h // 2].max(0)
                slack = 2.0 ** -7 * np.maximum(np.abs(lo), np.abs(hi)) + 1e-6
                assert (o[h] >= lo - slack).all() and (o[h] <= hi + slack).all()


def test_queries_of_any_size(cuda_lib):
    c = Case([300, 65], [1, 2], hq=4, hkv=2, dim=64)
    c.q[0] *= 2.0 ** -100                                 # (BF16) near even weights
    c.q[1, 0] = 0
    c.q[2, 1, :32] *= 2.0 ** -30
    c.check(c.paged(cuda_lib))
    c.q[:] = (c.q.float() * 2.0 ** 60).to(c.q.dtype)
    c.check(c.paged(cuda_lib, scale=2.0 ** -63), scale=2.0 ** -63, rows=[1, 2])


def test_a_nan_scale_reaches_the_rows_that_see_it(cuda_lib):
    c = Case([130, 70], [3, 2], hq=8, hkv=2, dim=128)
    clean = c.paged(cuda_lib)[0]
    kc, vc, ks, vs = F.views(c.host, 128)
    page = int(c.block_table[0, 2])                       # keys 128 and 129 of request 0: row 0 sees 128 keys
    vs[page, 0, 1, 3] = 0x7F
    ks[int(c.block_table[1, 1]), 5, 0, 5] = 0xFF          # key 69 of request 1: row 4 alone sees it
    c.cache.copy_(torch.from_numpy(c.host))
    got = c.paged(cuda_lib)[0]
    want = torch.zeros_like(clean, dtype=torch.bool)
    want[1:3, 4:8, 48:64] = True                          # rows 1 and 2, the heads of key head 1, block 3
    want[4, 0:4] = True                                   # a key's: the whole row of its head
    assert torch.equal(torch.isnan(got), want)
    assert torch.equal(got[~want], clean[~want])
    topk = torch.full((5, 70), -1, dtype=torch.int32, device="cuda")
    topk[1, 3], topk[1, 66], topk[2, 0] = 128, 5, 7
    got = c.selected(cuda_lib, topk)[0]
    want = torch.zeros_like(want)
    want[1, 4:8, 48:64] = True
    assert torch.equal(torch.isnan(got), want)


def test_bad_pages_are_skipped(cuda_lib):
    for bad in (-1, 10 ** 6):
        c = Case([200, 500], [1, 1], hq=8, hkv=2, dim=64)
        c.block_table[1, 3] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.paged(cuda_lib, status=status)
        assert int(status) == 2
        c.check(got, rows=[0])
        status.zero_()
        lists = torch.stack([torch.arange(200), torch.arange(192, 392)]).to(torch.int32).cuda()
        sel = c.selected(cuda_lib, lists, status=status)
        assert int(status) == 2
        c.check(sel, lists, rows=[0])
        # without the page's keys
        keep = torch.where((lists >= 192) & (lists < 256), -1, lists)
        keep[0] = lists[0]
        assert all(torch.equal(a, b) for a, b in zip(sel, c.selected(cuda_lib, keep)))


def test_bad_geometry_is_flagged(cuda_lib):
    c = Case([200, 500], [2, 1], hq=8, hkv=2, dim=64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.paged(cuda_lib, status=status)
    assert int(status) == 0
    for change in (lambda: c.starts.copy_(torch.tensor([0, 3, 2])), lambda: c.starts.copy_(torch.tensor([-2, 2, 3])),
                   lambda: c.starts.copy_(torch.tensor([0, 2, 9]))):
        change()
        for call in (lambda: c.paged(cuda_lib, status=status), lambda: c.selected(cuda_lib, choose(c, 5), status=status)):
            status.zero_()
            call()
            assert int(status) & 4
    c = Case([200, 500], [2, 1], hq=8, hkv=2, dim=64)
    c.row_ends[1] = 10 ** 6                               # past the table: cut to it (its last entry is no page)
    status.zero_()
    got = c.paged(cuda_lib, status=status)
    assert int(status) == 4 | 2
    c.check(got, rows=[0, 2])
    c.row_ends[1] = -4
    status.zero_()
    got = c.paged(cuda_lib, status=status)
    assert int(status) == 4 and not got[0][1].any()
    c.check(got, rows=[0, 2])


def test_list_entries_past_the_bound(cuda_lib):
    c = Case([200, 500], [2, 1], hq=8, hkv=2, dim=64)
    topk = choose(c, 40)
    clean = c.selected(cuda_lib, topk)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    more = torch.cat([topk, torch.tensor([[199, 5000], [-5, -2 ** 31], [2 ** 31 - 1, 500]], dtype=torch.int32,
                                         device="cuda")], dim=1)
    got = c.selected(cuda_lib, more, status=status)
    assert int(status) == 4
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    twice = topk[:, :4].repeat(1, 2)                      # listed twice counts twice
    a, b = c.selected(cuda_lib, twice), c.selected(cuda_lib, topk[:, :4].contiguous())
    c.check((a[0], a[1] - np.log(2.0)), topk[:, :4])
    c.check(b, topk[:, :4])


def test_nothing_to_see(cuda_lib):
    c = Case([0, 0], [1, 2], hq=8, hkv=2, dim=64, pad_rows=1)
    c.check(c.paged(cuda_lib))
    empty = torch.empty((4, 0), dtype=torch.int32, device="cuda")
    c.check(c.selected(cuda_lib, empty), empty)
    c = Case([100], [2], hq=8, hkv=2, dim=64)
    empty = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    c.check(c.selected(cuda_lib, empty), empty)
    none = torch.full((2, 100), -1, dtype=torch.int32, device="cuda")
    c.check(c.selected(cuda_lib, none), none)
    q = c.q[:0]
    out, lse = cuda_lib.attend_paged_fp4(q, c.cache, c.block_table[:0], c.starts[:1], c.row_ends[:0], 1, want_lse=True)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    out, lse = cuda_lib.attend_paged_fp4(c.q, pool(0, 2, 64), c.block_table[:, :0], c.starts,
                                         torch.zeros_like(c.row_ends), 1, want_lse=True)
    assert not out.any() and bool(torch.isneginf(lse).all())
    out, lse = cuda_lib.attend_selected_fp4(c.q, c.cache, c.block_table[:0], torch.zeros(1, dtype=torch.int32,
                                            device="cuda"), c.row_ends, none, want_lse=True)
    assert not out.any() and bool(torch.isneginf(lse).all())


def test_strided_queries_and_outputs(cuda_lib):
    c = Case([90, 300], [2, 1], hq=8, hkv=2, dim=96)
    want = c.paged(cuda_lib)
    wide = torch.zeros((3, 10, 2, 104), dtype=c.q.dtype, device="cuda")
    q = wide[:, 1:9, 1, :96]
    q.copy_(c.q)
    out = torch.full((3, 8, 104), 9.0, dtype=c.q.dtype, device="cuda")
    got = cuda_lib.attend_paged_fp4(q, c.cache, c.block_table, c.starts, c.row_ends, 2, out=out[:, :, :96])
    assert torch.equal(got[0], want[0]) and bool((out[..., 96:] == 9).all()) and got[1] is None
    topk = choose(c, 30)
    lists = torch.full((3, 64), 10 ** 6, dtype=torch.int32, device="cuda")
    lists[:, :30] = topk
    a = cuda_lib.attend_selected_fp4(q, c.cache, c.block_table, c.starts, c.row_ends, lists[:, :30], want_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(a, c.selected(cuda_lib, topk)))
    # every row the same query: a stride of 0
    same = c.q[:1].expand(3, 8, 96)
    a = cuda_lib.attend_paged_fp4(same, c.cache, c.block_table, c.starts, c.row_ends, 2)
    b = cuda_lib.attend_paged_fp4(same.contiguous(), c.cache, c.block_table, c.starts, c.row_ends, 2)
    assert torch.equal(a[0], b[0])


def test_any_bytes_may_be_in_a_workspace(cuda_lib):
    for c in (Case([3000, 100, 777], [2, 1, 1], hq=16, hkv=2, dim=128),
              Case([(53 * j) % 301 for j in range(600)], [1 + j % 2 for j in range(600)], hq=4, hkv=2, dim=64)):
        topk = choose(c, 100)
        rows, hq, dim = c.q.shape
        args = (rows, c.block_table.shape[0], hq, c.hkv, dim)
        n = max(cuda_lib.attend_workspace_size_fp4(*args, c.qlen), cuda_lib.attend_workspace_size_fp4(*args, 1, 100))
        results = []
        for byte in (0, 0x7F, 0xFF):
            ws = torch.full((n,), byte, dtype=torch.uint8, device="cuda")
            results.append(c.paged(cuda_lib, workspace=ws) + c.selected(cuda_lib, topk, workspace=ws.fill_(byte)))
        for r in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], r))


def test_far_pages(cuda_lib):
    """Sections past 2^32 bytes of the pool read as those at its start."""
    c = Case([300], [2], hq=16, hkv=8, dim=128)
    pages = 60000
    big = torch.zeros((pages,) + tuple(c.cache.shape[1:]), dtype=torch.uint8, device="cuda")
    far = torch.tensor([[59999, 58999, 58300, 59500, 58257, -7]], dtype=torch.int32, device="cuda")
    for j in range(5):
        big[int(far[0, j])] = c.cache[int(c.block_table[0, j])]
    want = c.paged(cuda_lib)
    topk = choose(c, 150)
    want_s = c.selected(cuda_lib, topk)
    c.cache, c.block_table = big, far
    assert all(torch.equal(a, b) for a, b in zip(c.paged(cuda_lib), want))
    assert all(torch.equal(a, b) for a, b in zip(c.selected(cuda_lib, topk), want_s))


def test_captured_and_on_another_stream(cuda_lib):
    c = Case([700, 90, 20], [2, 1, 3], hq=16, hkv=2, dim=128)
    topk = choose(c, 100)
    want = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    c.q.neg_()                                            # new inputs in the captured call's tensors
    graph.replay()
    torch.cuda.synchronize()
    c.check(got[:2])
    c.check(got[2:], topk)


@pytest.mark.parametrize("lens,qlens,hq,hkv,dim", [
    ([1000], [1], 32, 8, 128), ([64 * 90], [4], 16, 4, 128), ([64 * 100 + 1], [2], 8, 2, 64), ([0, 5, 130], [1, 2, 1], 8, 2, 96),
    ([20000], [1], 4, 1, 128), ([24576], [2], 30, 1, 80), ([700, 0], [3, 0], 24, 2, 128), ([300, 300], [1, 1], 128, 2, 48),
    ([100 + 170 * j for j in range(5)], [1, 4, 2, 1, 3], 24, 6, 128), ([130 + 40 * j for j in range(9)], [1] * 9, 32, 8, 128),
    ([64 * (j % 9) for j in range(19)], [1 + j % 2 for j in range(19)], 16, 8, 64), ([777] * 37, [2] * 37, 16, 1, 112),
    ([40 + j % 7 for j in range(120)], [31] * 120, 1, 1, 16)])
def test_few_items(cuda_lib, lens, qlens, hq, hkv, dim):
    """Batches small enough for a cluster an item (and, by a hint that is too small, their row tiles in turn)."""
    c = Case(lens, qlens, hq=hq, hkv=hkv, dim=dim, pad_rows=2)
    rows = range(0, c.q.shape[0], 1 + c.q.shape[0] // 400)
    for hint in (c.qlen, 1):
        c.check(c.paged(cuda_lib, max_query_len=hint), rows=rows)
    for k in (3, 2048):
        topk = choose(c, k, seed=k)
        c.check(c.selected(cuda_lib, topk), topk, rows=rows)


def test_few_items_and_many_agree(cuda_lib):
    """The same request alone and among others: the parts of its keys are joined in another order."""
    one = Case([1500], [2], hq=8, hkv=2, dim=128, seed=3)
    alone = one.paged(cuda_lib)
    one.check(alone)
    table = one.block_table.repeat(40, 1)
    q = one.q.repeat(40, 1, 1)
    starts = torch.arange(0, 82, 2, dtype=torch.int32, device="cuda")
    out, lse = cuda_lib.attend_paged_fp4(q, one.cache, table, starts, one.row_ends.repeat(40), 2, want_lse=True)
    for j in (0, 17, 39):
        one.check((out[2 * j: 2 * j + 2], lse[2 * j: 2 * j + 2]))


def test_lists_in_order_of_their_positions(cuda_lib):
    """A batch large enough that lists are put in order first: random orders, holes, positions listed twice, past the
    bound, and pages outside the pool."""
    lens = [200 + 37 * j for j in range(130)]
    c = Case(lens, [1] * 130, hq=8, hkv=8, dim=128)
    topk = choose(c, 700)
    assert 130 * 8 * 11 * F.section_bytes(128) >= 64 << 20
    got = c.selected(cuda_lib, topk)
    c.check(got, topk, rows=range(0, 130, 9))
    shuffled = topk.clone()
    for r in (3, 77):
        shuffled[r] = topk[r][torch.randperm(700, device="cuda")]
    again = c.selected(cuda_lib, shuffled)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    twice = topk.clone()
    twice[5, :60], twice[5, 60:] = torch.arange(60), -1
    twice[5, 60:120] = torch.arange(60)
    twice[6, 5] = 10 ** 6
    out, lse = c.selected(cuda_lib, twice, status=status)
    assert int(status) == 4
    c.check((out, lse - np.log(2.0)), topk=twice[:, :60].contiguous(), rows=[5])
    assert torch.equal(out[7:], got[0][7:])
    c.block_table[9, 1] = 10 ** 7
    status.zero_()
    out, lse = c.selected(cuda_lib, topk, status=status)
    assert int(status) == 2 and torch.equal(out[10:], got[0][10:])
    keep = topk.clone()                                   # (the same keys, in units of their own)
    keep[9] = torch.where((topk[9] >= 64) & (topk[9] < 128), -1, topk[9])
    c.check((out, lse), keep, rows=[9])


def test_two_streams_at_once(cuda_lib):
    """Calls of both kinds side by side, each stream with a workspace of its own, give what they give alone."""
    cases = [Case([900 + 61 * j for j in range(24)], [4] * 24, hq=64, hkv=8, dim=128, seed=5),
             Case([1300], [2], hq=16, hkv=2, dim=128, dtype="fp16", seed=6)]
    lists = [choose(c, 300, seed=9) for c in cases]
    spaces = [torch.empty(max(cuda_lib.attend_workspace_size_fp4(c.q.shape[0], c.starts.numel() - 1, c.q.shape[1], c.hkv,
                                                                 c.dim, c.qlen, k) for k in (0, 300)),
                          dtype=torch.uint8, device="cuda") for c in cases]

    def run(i):
        c = cases[i]
        args = (c.q, c.cache, c.block_table, c.starts, c.row_ends)
        return (cuda_lib.attend_paged_fp4(*args, c.qlen, workspace=spaces[i])[0],
                cuda_lib.attend_selected_fp4(*args, lists[i], workspace=spaces[i])[0])

    alone = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(4):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got.append((i, run(i)))
    torch.cuda.synchronize()
    for i, outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, alone[i]))


@pytest.mark.parametrize("requests", [1, 90])
def test_rows_before_the_first_request(cuda_lib, requests):
    c = Case([150 + j for j in range(requests)], [2] * requests, hq=8, hkv=2, dim=96)
    topk = choose(c, 70)
    q = torch.cat([c.q[:1].expand(3, -1, -1), c.q])
    ends = torch.cat([torch.full((3,), 40, dtype=torch.int32, device="cuda"), c.row_ends])
    args = (q, c.cache, c.block_table, c.starts + 3, ends)
    for got, lists in ((cuda_lib.attend_paged_fp4(*args, 2, want_lse=True), None),
                       (cuda_lib.attend_selected_fp4(*args, torch.cat([topk[:1].expand(3, -1), topk]), want_lse=True), topk)):
        assert not got[0][:3].any() and bool(torch.isneginf(got[1][:3]).all())
        c.check(tuple(t[3:] for t in got), lists, rows=range(0, 2 * requests, 7))


def test_output_in_the_place_of_the_queries(cuda_lib):
    c = Case([500 + 9 * j for j in range(40)], [3] * 40, hq=24, hkv=2, dim=64)
    want = c.paged(cuda_lib)[0]
    q = c.q.clone()
    out, _ = cuda_lib.attend_paged_fp4(q, c.cache, c.block_table, c.starts, c.row_ends, c.qlen, out=q)
    assert out is q and torch.equal(q, want)
