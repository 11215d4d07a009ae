"""Tensors whose dimensions of one element come with odd strides, as transposes and slices leave them: they hold what
their contiguous copies hold.  On the CPU such a call gets as far as the check that the caches are CUDA tensors."""

import pytest
import torch

from attend_case import Case, choose, empty_cache

BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


def odd(t, d, step):
    """t with the stride of its one-element dimension d replaced."""
    assert t.shape[d] == 1
    strides = list(t.stride())
    strides[d] = step
    return t.as_strided(t.shape, strides, t.storage_offset())


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_indexer_score_gb300 import build
    try:
        build.build()
    except RuntimeError as e:   # no nvcc on this machine
        pytest.skip(str(e))
    from sparse_attention_indexer_score_gb300 import dsa as d
    return d


def test_rows_of_one_column_are_dense(dsa):
    """[3, 1] and [2, 1] tensors whose column stride is not one."""
    z = torch.zeros
    args = dict(q=z(2, 8, 64, dtype=BF), k_cache=z(3, 64, 2, 64, dtype=BF), v_cache=z(3, 64, 2, 64, dtype=BF),
                block_table=odd(z(3, 1, dtype=I32), 1, 7), starts=z(4, dtype=I32), row_ends=z(2, dtype=I32))
    with pytest.raises(ValueError, match="CUDA"):
        dsa.attend_paged(**args, max_query_len=1)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.attend_selected(**args, topk=odd(z(2, 1, dtype=I32), 1, 5))


@pytest.mark.gpu
@pytest.mark.parametrize("step", [0, 1, 3, 4096])
def test_one_row_one_request_one_key_head(cuda_lib, step):
    """Block table, lists, queries, outputs and caches of one row, request, head or page with any stride there."""
    c = Case([300], [1], hq=16, hkv=1, dim=64)
    topk = choose(c, 90)
    want, listed = c.paged(cuda_lib), c.selected(cuda_lib, topk)
    c.check(want)
    c.block_table, c.q = odd(c.block_table, 0, step), odd(c.q, 0, step)
    c.k, c.v = odd(c.k, 2, step), odd(c.v, 2, step)
    out = odd(torch.zeros_like(c.q), 0, step)
    got = c.paged(cuda_lib, out=out)
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(got[1], want[1])
    got = c.selected(cuda_lib, odd(topk, 0, step), out=out)
    assert got[0] is out and torch.equal(out, listed[0]) and torch.equal(got[1], listed[1])
    head = Case([60, 50], [1, 1], hq=1, hkv=1, dim=64, dtype="fp16", layout="hnd")
    want = head.paged(cuda_lib)
    head.q, head.k, head.v = odd(head.q, 1, step), odd(head.k, 2, step), odd(head.v, 2, step)
    assert torch.equal(head.paged(cuda_lib)[0], want[0])
    short = Case([40], [1], hq=4, hkv=2, dim=64)
    topk = torch.arange(40, device="cuda", dtype=I32)[None]
    want, listed = short.paged(cuda_lib), short.selected(cuda_lib, topk)
    pages = short.block_table[0, :1].tolist()
    short.k, short.v = (odd(t[pages], 0, step) for t in (short.k, short.v))      # a pool of one page
    short.block_table = torch.zeros((1, 1), dtype=I32, device="cuda")
    assert torch.equal(short.paged(cuda_lib)[0], want[0])
    assert torch.equal(short.selected(cuda_lib, topk)[0], listed[0])


@pytest.mark.gpu
@pytest.mark.parametrize("step", [0, 1, 3, 4096])
def test_append_of_one_token(cuda_lib, step):
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((1, h, 64), generator=g).to(BF).cuda() for h in (4, 1, 1))
    cs = torch.rand((1, 64), generator=g).cuda()
    slot, pos = torch.tensor([5], device="cuda"), torch.zeros(1, dtype=I64, device="cuda")
    kc, vc = empty_cache(1, 1, 64, "bf16", "nhd", fill=0.0)
    want = cuda_lib.kv_append(k, v, slot, kc, vc, pos, cs, q=q)
    kd, vd = empty_cache(1, 1, 64, "bf16", "nhd", fill=0.0)
    out = odd(torch.zeros_like(q), 0, step)
    got = cuda_lib.kv_append(odd(odd(k, 0, step), 1, step), odd(odd(v, 0, step), 1, step), slot,
                             odd(odd(kd, 0, step), 2, step), odd(odd(vd, 0, step), 2, step), pos, odd(cs, 0, step),
                             q=odd(q, 0, step), q_out=out)
    assert got is out and torch.equal(out, want) and torch.equal(kc, kd) and torch.equal(vc, vd)


@pytest.mark.gpu
def test_a_broadcast_query_is_refused(cuda_lib):
    c = Case([70, 50], [1, 1], hq=8, hkv=2, dim=64)
    for q in (c.q[:1].expand(2, 8, 64), c.q[:, :1].expand(2, 8, 64)):
        c.q = q
        with pytest.raises(RuntimeError, match="unsupported"):
            c.paged(cuda_lib)
