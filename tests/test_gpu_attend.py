"""The append and attention calls on the GPU against the 64-bit oracle."""

import numpy as np
import pytest
import torch

from attend_case import DT, Case, choose, empty_cache
from oracle import attention as A

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append
def append_case(n, hq, hkv, dim, rot, dtype, layout, seed=0, packed=True):
    g = torch.Generator().manual_seed(seed)
    pages = n // 64 + 2
    x = torch.randn((n, (hq + 2 * hkv) * dim), generator=g).to(DT[dtype]).cuda()
    q, k, v = x.split([hq * dim, hkv * dim, hkv * dim], dim=1)     # views of one projection, as a layer has them
    q, k, v = q.unflatten(1, (hq, dim)), k.unflatten(1, (hkv, dim)), v.unflatten(1, (hkv, dim))
    if not packed:
        q, k, v = q.transpose(0, 1).contiguous().transpose(0, 1), k.contiguous(), v.contiguous()
    kc, vc = empty_cache(pages, hkv, dim, dtype, layout, fill=0.5)
    slots = torch.randperm(pages * 64, generator=g)[:n].cuda()
    pos = torch.randint(0, 500, (n,), generator=g).cuda()
    ang = torch.rand((500, max(rot // 2, 1)), generator=g) * 6.28
    cs = torch.cat([ang.cos(), ang.sin()], 1).cuda() if rot else None
    return q, k, v, slots, kc, vc, pos, cs


def check_append(dsa, q, k, v, slots, kc, vc, pos, cs, inter, want_status=0, **kw):
    ref_k, ref_v = kc.double().cpu().numpy(), vc.double().cpu().numpy()
    before_k = ref_k.copy()
    host = [None if t is None else t.double().cpu().numpy() for t in (k, v, q, cs)]
    ref_q = A.append(host[0], host[1], slots.tolist(), ref_k, ref_v, None if pos is None else pos.tolist(), host[3],
                     host[2], inter)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = dsa.kv_append(k, v, slots, kc, vc, pos, cs, q=q, interleaved=inter, status=status, **kw)
    assert int(status) == want_status
    eps = torch.finfo(kc.dtype).eps
    # two FP32 products and a sum, each off by 2^-24 of the larger of |a| + |b| (at most 2 max |x|), and one rounding
    worst = 2.0 ** -23 * 2 * float(max(np.abs(host[0]).max(initial=0), 0 if q is None else np.abs(host[2]).max(initial=0)))
    tiny = 2.0 ** -25 if kc.dtype == torch.float16 else 0.0

    def near(x, y):
        assert (np.abs(x - y) <= eps / 2 * np.abs(y) + worst + tiny).all(), np.abs(x - y).max()

    near(kc.double().cpu().numpy(), ref_k)
    np.testing.assert_array_equal(vc.double().cpu().numpy(), ref_v)
    untouched = np.ones(before_k.shape[:2], dtype=bool)
    for s in slots.tolist():
        if 0 <= s < untouched.size:
            untouched[s // 64, s % 64] = False
    np.testing.assert_array_equal(kc.double().cpu().numpy()[untouched], before_k[untouched])
    if q is not None:
        near(got.double().cpu().numpy(), ref_q)
    else:
        assert got is None


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hkv,dim,rot,layout", [
    (1, 8, 2, 128, 128, "nhd"), (3, 32, 8, 128, 64, "hnd"), (77, 5, 5, 80, 32, "pair"), (130, 6, 1, 96, 96, "nhd"),
    (9, 7, 1, 256, 16, "hnd"), (40, 4, 2, 64, 64, "odd"), (2, 3, 3, 512, 512, "nhd"), (5, 2, 1, 16, 16, "nhd"), (700, 4, 4, 64, 64, "hnd")])
def test_append(cuda_lib, n, hq, hkv, dim, rot, layout, inter, dtype):
    check_append(cuda_lib, *append_case(n, hq, hkv, dim, rot, dtype, layout, packed=n != 9), inter)


def test_append_without_rotation_or_queries(cuda_lib):
    q, k, v, slots, kc, vc, pos, _ = append_case(50, 4, 2, 64, 0, "bf16", "nhd")
    check_append(cuda_lib, None, k, v, slots, kc, vc, None, None, False)
    check_append(cuda_lib, q, k, v, slots, kc, vc, None, None, False)
    q, k, v, slots, kc, vc, pos, cs = append_case(50, 4, 2, 64, 64, "fp16", "nhd")
    check_append(cuda_lib, None, k, v, slots, kc, vc, pos, cs, True)


def test_append_padding_bad_slots_and_positions(cuda_lib):
    q, k, v, slots, kc, vc, pos, cs = append_case(8, 4, 2, 64, 32, "bf16", "hnd")
    slots[2] = -1
    pos[2] = 10 ** 12                                    # a padding token's position is clamped and not flagged
    check_append(cuda_lib, q, k, v, slots, kc, vc, pos, cs, False)
    slots[3] = kc.shape[0] * 64                          # past the pool
    check_append(cuda_lib, q, k, v, slots, kc, vc, pos, cs, False, want_status=1)
    slots[3] = 2 ** 62
    pos[4], pos[5] = -3, 500
    check_append(cuda_lib, q, k, v, slots, kc, vc, pos, cs, False, want_status=5)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    check_append(cuda_lib, q[:0], k[:0], v[:0], none, kc, vc, none, cs, False)


def test_append_in_place_equals_out_of_place(cuda_lib):
    q, k, v, slots, kc, vc, pos, cs = append_case(300, 8, 2, 128, 128, "bf16", "nhd")
    a = cuda_lib.kv_append(k, v, slots, kc, vc, pos, cs, q=q)
    b = cuda_lib.kv_append(k, v, slots, kc, vc, pos, cs, q=q, q_out=q)
    assert b is q and torch.equal(a, b)


# ------------------------------------------------------------------ attention
LENS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 256, 300]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "pair", "odd"])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 64), (4, 4, 128), (16, 1, 128), (6, 2, 80), (3, 1, 16), (40, 2, 96),
                                        (100, 1, 128)])
def test_paged_lengths(cuda_lib, hq, hkv, dim, layout, dtype):
    c = Case(LENS, [1] * len(LENS), hq=hq, hkv=hkv, dim=dim, layout=layout, dtype=dtype, pad_rows=2)
    c.check(c.paged(cuda_lib))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("prefix", [1, 64, 127, 500])
@pytest.mark.parametrize("qlens", [[1, 1, 1], [4, 2, 3], [1, 40, 0]])
def test_paged_prefix(cuda_lib, qlens, prefix, dtype):
    c = Case([0, 200, 70], qlens, prefix=prefix, hq=8, hkv=2, dim=96, dtype=dtype, pad_rows=1)
    c.check(c.paged(cuda_lib))


@pytest.mark.parametrize("hq,hkv,rows,prefix", [(64, 8, 17, 129), (16, 2, 50, 1000), (128, 1, 3, 300), (7, 7, 300, 65),
                                                (12, 4, 100, 640), (4, 4, 129, 128), (32, 2, 33, 4001)])
def test_many_rows_behind_a_prefix(cuda_lib, hq, hkv, rows, prefix):
    """More rows of one key head than a tile has: several row tiles read the prefix."""
    lens = [(37 * j) % 150 for j in range(rows)]
    c = Case(lens, [1] * rows, prefix=prefix, hq=hq, hkv=hkv, dim=64, pad_rows=1, seed=3)
    c.check(c.paged(cuda_lib), rows=list(range(0, rows + 1, 7)) + [rows])
    wide = Case(lens, [1] * rows, prefix=prefix, hq=hq, hkv=hkv, dim=128, dtype="fp16", layout="hnd", seed=4)
    wide.check(wide.paged(cuda_lib), rows=range(0, rows, 11))


# (the last row tile without a partner, tiles that are not full, prefixes that end inside a page or with a tile)
PAIRED = [(128, 1, 65, 7301, 64, "bf16", "nhd"), (64, 2, 81, 12001, 128, "fp16", "hnd"),
          (48, 16, 100, 7680, 96, "bf16", "pair"), (7, 7, 129, 33793, 16, "fp16", "odd"),
          (64, 8, 320, 8200, 128, "bf16", "odd")]


@pytest.mark.parametrize("hq,hkv,rows,prefix,dim,dtype,layout", PAIRED)
def test_long_prefix_behind_many_rows(cuda_lib, hq, hkv, rows, prefix, dim, dtype, layout):
    """So many tiles that the prefix has a launch of its own, in pairs of row tiles."""
    tiles = -(-rows // (128 // (hq // hkv)))
    assert (tiles + 1) // 2 * hkv * -(-prefix // 128) > 12 * torch.cuda.get_device_properties(0).multi_processor_count
    lens = [(37 * j) % 150 for j in range(rows)]
    c = Case(lens, [1] * rows, prefix=prefix, hq=hq, hkv=hkv, dim=dim, dtype=dtype, layout=layout, pad_rows=2, seed=6)
    got = c.paged(cuda_lib)
    c.check(got, rows=[0, 1, rows // 2, rows - 2, rows - 1, rows, rows + 1])
    again = c.paged(cuda_lib)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_paged_long_rows(cuda_lib, dtype):
    """Few rows over long contexts: the keys are split over the GPU and joined."""
    c = Case([20011, 9000], [1, 3], hq=8, hkv=2, dim=128, dtype=dtype)
    c.check(c.paged(cuda_lib))
    c = Case([1, 40], [1, 1], prefix=12345, hq=4, hkv=1, dim=64, dtype=dtype)
    c.check(c.paged(cuda_lib))


def test_max_query_len_is_only_a_hint(cuda_lib):
    c = Case([100, 300], [9, 3], prefix=70, hq=8, hkv=2, dim=64)
    for hint in (0, 1, 2, 100):
        c.qlen = hint
        c.check(c.paged(cuda_lib))


def test_bounds_of_rows_need_not_rise(cuda_lib):
    """Row bounds of one request in any order, one of them zero."""
    c = Case([400], [5], hq=4, hkv=2, dim=64, ends=[400, 0, 7, 130, 64])
    c.check(c.paged(cuda_lib))


def test_one_score_far_above_the_others(cuda_lib):
    """The running maximum jumps late: what was summed before is scaled away, exactly to zero or nearly."""
    c = Case([700], [1], hq=4, hkv=2, dim=64)
    c.q.fill_(1.0)
    table = c.block_table[0].tolist()
    c.k[table[9], 50] = 30.0
    c.check(c.paged(cuda_lib))
    c.k[table[2], 3] = 12.0
    c.check(c.paged(cuda_lib))
    c.q.fill_(-1.0)
    c.check(c.paged(cuda_lib))


def test_keys_of_other_rows_do_not_leak(cuda_lib):
    """A later verify row's key and value hold NaN and infinities: the earlier rows do not see them."""
    c = Case([200, 90], [4, 1], prefix=100, hq=8, hkv=2, dim=64)
    t = c.block_table[0].tolist()
    c.check(c.paged(cuda_lib))
    c.k[t[3], 7], c.v[t[3], 7] = float("nan"), float("inf")      # position 199: the last row's alone
    c.v[t[3], 6, 0] = float("-inf")                              # position 198: the last two rows', one head
    out, lse = c.paged(cuda_lib)
    c.check((out, lse), rows=[0, 1, 4])
    assert torch.isnan(out[3]).all()
    assert torch.isfinite(out[2, 4:]).all() and not torch.isfinite(out[2, :4]).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("k", [1, 7, 128, 129, 300])
@pytest.mark.parametrize("hq,hkv,dim,layout", [(8, 2, 64, "nhd"), (16, 1, 128, "hnd"), (6, 3, 80, "pair"), (4, 4, 16, "nhd"),
                                               (6, 2, 96, "odd"), (40, 2, 64, "nhd"), (128, 1, 128, "hnd")])
def test_selected(cuda_lib, hq, hkv, dim, layout, k, dtype):
    c = Case([0, 1, 64, 200, 999], [1, 1, 2, 3, 1], hq=hq, hkv=hkv, dim=dim, layout=layout, dtype=dtype, pad_rows=1)
    for holes in (False, True):
        topk = choose(c, k, holes=holes)
        c.check(c.selected(cuda_lib, topk), topk)


def test_selected_long_lists(cuda_lib):
    c = Case([5000, 2048, 100], [1, 2, 1], hq=32, hkv=8, dim=128)
    topk = choose(c, 2048)
    c.check(c.selected(cuda_lib, topk), topk)
    one = Case([8192], [1], hq=32, hkv=8, dim=128, dtype="fp16")
    topk = choose(one, 2048, holes=False)
    one.check(one.selected(cuda_lib, topk), topk)


def test_selected_duplicates_strides_and_empty_lists(cuda_lib):
    c = Case([150, 300], [2, 1], hq=4, hkv=2, dim=64)
    wide = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    wide[0, :6] = torch.tensor([3, 3, 3, 77, 148, 3])
    wide[2, 30:33] = torch.tensor([299, 0, 64])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(c.selected(cuda_lib, wide[:, :33], status=status), wide[:, :33])
    assert int(status) == 0
    none = wide[:, :0]
    c.check(c.selected(cuda_lib, none), none)


def test_selected_positions_past_the_bound_are_skipped_and_flagged(cuda_lib):
    c = Case([150, 300], [2, 1], hq=4, hkv=2, dim=64)
    topk = choose(c, 20)
    topk[0, 4], topk[2, 0] = 149, 2 ** 31 - 1            # row 0 sees 149 keys, row 2 300
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(c.selected(cuda_lib, topk, status=status), topk)
    assert int(status) == 4


def test_bad_pages_are_not_read_and_flagged(cuda_lib):
    c = Case([300, 200], [1, 1], prefix=130, hq=4, hkv=2, dim=64)
    c.block_table[0, 1], c.block_table[0, 2] = 10 ** 6, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.paged(cuda_lib, status=status)
    assert int(status) == 2
    c.check(got, rows=[1])
    status.zero_()
    topk = choose(c, 200)
    c.check(c.selected(cuda_lib, topk, status=status), topk, rows=[1])
    assert int(status) == 2


def test_bad_geometry_is_clamped_and_flagged(cuda_lib):
    c = Case([100, 64], [1, 1], hq=4, hkv=2, dim=64)
    good = c.row_ends.clone()
    width = c.block_table.shape[1] * 64
    for bad in (-5, width + 1, 2 ** 31 - 1):
        c.row_ends[0] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.paged(cuda_lib, status=status)
        assert int(status) & 4
        c.check(got, rows=[1])
    c.row_ends.copy_(good)
    for starts in ([0, 1, 5], [0, -3, 2], [0, 2, 1]):
        c.starts.copy_(torch.tensor(starts, dtype=torch.int32))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.paged(cuda_lib, status=status)
        assert int(status) & 4
    torch.cuda.synchronize()


def test_empty_calls(cuda_lib):
    c = Case([10], [1], hq=4, hkv=2, dim=64)
    out, lse = cuda_lib.attend_paged(c.q[:0], c.k, c.v, c.block_table, c.starts, c.row_ends[:0], 1, want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # no requests: every row is padding, even behind a prefix
    out, lse = cuda_lib.attend_paged(c.q, c.k, c.v, c.block_table[:0], c.starts[:1], c.row_ends, 1, want_lse=True,
                                     prefix_pages=c.block_table[0, :1], prefix_len=10)
    assert not out.any() and torch.isneginf(lse).all()
    # requests without a block-table column see the prefix alone
    bare = Case([0, 0], [1, 1], prefix=100, hq=4, hkv=2, dim=64)
    bare.block_table = bare.block_table[:, :0]
    bare.check(bare.paged(cuda_lib))


def test_strided_queries_and_outputs(cuda_lib):
    c = Case([130, 70], [2, 1], prefix=66, hq=8, hkv=2, dim=64)
    plain = c.paged(cuda_lib)
    wide = torch.zeros((3, 8, 200), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 64:128] = c.q
    c.q = wide[:, :, 64:128]
    out = torch.full((8, 3, 72), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got = c.paged(cuda_lib, out=out[:, :, :64])
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    assert (out[:, :, 64:] == 7.0).all()


def test_workspace_is_reusable_across_sizes_and_results_repeat(cuda_lib):
    big = Case([3000, 100, 777], [2, 1, 1], prefix=1500, hq=16, hkv=2, dim=128)
    small = Case([90], [1], hq=16, hkv=2, dim=128)
    n = max(cuda_lib.attend_workspace_size(4, 3, 16, 2, 128, 2), cuda_lib.attend_workspace_size(4, 3, 16, 2, 128, 2, 500))
    ws = cuda_lib.new_workspace(n, "cuda")
    topk = choose(big, 500)
    first = [t.clone() for t in big.paged(cuda_lib, workspace=ws) + big.selected(cuda_lib, topk, workspace=ws)]
    for _ in range(3):
        small.check(small.paged(cuda_lib, workspace=ws))
        again = big.paged(cuda_lib, workspace=ws) + big.selected(cuda_lib, topk, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_repeated_calls_agree_on_every_bit(cuda_lib):
    """Nothing depends on the order in which CTAs finish."""
    c = Case([9000, 5000, 1], [2, 4, 1], prefix=2000, hq=32, hkv=4, dim=128, dtype="fp16")
    topk = choose(c, 900)
    first = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, c.paged(cuda_lib) + c.selected(cuda_lib, topk)))


def test_a_workspace_too_small_is_refused(cuda_lib):
    c = Case([90], [1], hq=4, hkv=2, dim=64)
    n = cuda_lib.attend_workspace_size(1, 1, 4, 2, 64, 1)
    with pytest.raises(RuntimeError, match="invalid"):
        c.paged(cuda_lib, workspace=torch.zeros(n - 1, dtype=torch.uint8, device="cuda"))


def test_many_requests(cuda_lib):
    """More segments than a CTA lays out itself, empty ones among them."""
    lens = [(53 * j) % 301 for j in range(300)]
    c = Case(lens, [1 + j % 3 if j % 7 else 0 for j in range(300)], hq=4, hkv=2, dim=64, pad_rows=3)
    rows = range(0, c.q.shape[0], 17)
    c.check(c.paged(cuda_lib), rows=rows)
    topk = choose(c, 150)
    c.check(c.selected(cuda_lib, topk), topk, rows=rows)
    behind = Case(lens, [1] * 300, prefix=300, hq=4, hkv=2, dim=64, dtype="fp16")
    behind.check(behind.paged(cuda_lib), rows=rows[:10])


def test_a_row_of_many_heads_and_long_queries(cuda_lib):
    """Requests with more rows than a tile has, bounds that end inside a tile of rows."""
    c = Case([700, 90, 1500], [130, 3, 260], prefix=33, hq=6, hkv=2, dim=64)
    c.check(c.paged(cuda_lib), rows=[0, 41, 42, 43, 129, 130, 132, 133, 174, 175, 392])
    c.qlen = 4
    c.check(c.paged(cuda_lib), rows=[0, 42, 129, 130, 175, 392])


def test_calls_follow_the_current_stream(cuda_lib):
    c = Case([500, 300], [1, 2], prefix=64, hq=8, hkv=2, dim=64)
    q = c.q.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        c.q = torch.empty_like(q)
        c.q.copy_(q)
        got = c.paged(cuda_lib)
    side.synchronize()
    c.check(got)


def test_a_captured_step_repeats_on_new_inputs(cuda_lib):
    """append, dense and selected attention in one CUDA graph."""
    c = Case([500, 300], [1, 1], prefix=64, hq=8, hkv=2, dim=64)
    ws = cuda_lib.new_workspace(max(cuda_lib.attend_workspace_size(2, 2, 8, 2, 64, 1),
                                    cuda_lib.attend_workspace_size(2, 2, 8, 2, 64, 1, 40)), "cuda")
    topk = choose(c, 40)
    table = c.block_table.tolist()
    slots = torch.tensor([table[0][7] * 64 + 51, table[1][4] * 64 + 43], device="cuda")   # positions 499 and 299
    k, v = (torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))

    def step():
        cuda_lib.kv_append(k, v, slots, c.k, c.v)
        return c.paged(cuda_lib, workspace=ws) + c.selected(cuda_lib, topk, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        k.normal_()
        v.normal_()
        c.q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.k[table[0][7], 51], k[0]) and torch.equal(c.v[table[1][4], 43], v[1])
        c.check(got[:2])
        c.check(got[2:], topk)


def test_offsets_past_32_bits(cuda_lib):
    """A pool of more than 2^32 elements: the pages used lie at its two ends."""
    hkv, dim = 8, 128
    pages = 2 ** 32 // (64 * hkv * dim) + 3
    c = Case([200, 150], [1, 2], prefix=70, hq=16, hkv=hkv, dim=dim)
    k, v = (torch.empty((pages, 64, hkv, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = c.k.shape[0]
    far = torch.arange(n, device="cuda") + pages - n
    k[pages - n:], v[pages - n:] = c.k, c.v
    c.block_table = torch.where(c.block_table >= 0, far[c.block_table.clamp(min=0).long()].int(), -7).contiguous()
    c.prefix_pages = far[c.prefix_pages.long()].int()
    small = c.k, c.v
    c.k, c.v = k, v
    topk = choose(c, 100)
    got, sel = c.paged(cuda_lib), c.selected(cuda_lib, topk)
    slot = torch.tensor([(pages - 1) * 64 + 63], device="cuda")
    new = torch.randn((1, hkv, dim), device="cuda").to(torch.bfloat16)
    cuda_lib.kv_append(new, new, slot, k, v)
    assert torch.equal(k[-1, -1], new[0]) and torch.equal(v[-1, -1], new[0])
    c.k, c.v = small
    back = pages - n
    c.block_table = torch.where(c.block_table >= 0, c.block_table - back, -7)
    c.prefix_pages = c.prefix_pages - back
    c.check(got)
    c.check(sel, topk)
