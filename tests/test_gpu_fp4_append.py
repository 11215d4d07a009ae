"""The 4-bit cache's append and reading back on the GPU against the oracle, byte for byte."""

import numpy as np
import pytest
import torch

from fp4_case import DT, pool
from oracle import fp4_cache as F

pytestmark = pytest.mark.gpu


def case(n, hq, hkv, dim, rot, dtype, layers=1, seed=0, pages=None, fill=0x35):
    g = torch.Generator().manual_seed(seed)
    pages = n // 64 + 2 if pages is None else pages
    x = torch.randn((n, (hq + 2 * hkv) * dim), generator=g) * 3
    x[:, hq * dim] *= 20                                            # a column that is larger than the others
    q, k, v = x.to(DT[dtype]).cuda().split([hq * dim, hkv * dim, hkv * dim], dim=1)   # views of one projection
    q, k, v = q.unflatten(1, (hq, dim)), k.unflatten(1, (hkv, dim)), v.unflatten(1, (hkv, dim))
    slots = torch.randperm(pages * 64, generator=g)[:n].cuda()
    pos = torch.randint(0, 500, (n,), generator=g).cuda()
    ang = torch.rand((500, max(rot // 2, 1)), generator=g) * 6.28
    cs = torch.cat([ang.cos(), ang.sin()], 1).cuda() if rot else None
    return q, k, v, slots, pool(pages, hkv, dim, layers, fill=fill), pos, cs


def check(dsa, q, k, v, slots, cache, pos, cs, inter=False, want_status=0, k_scale=1.0, v_scale=1.0, **kw):
    dim = k.shape[2]
    want = cache.cpu().numpy().copy()
    host = [None if t is None else t.float().cpu().numpy() for t in (k, v, cs)]
    F.append(host[0], host[1], slots.cpu().numpy(), want, dim, None if pos is None else pos.cpu().numpy(), host[2],
             inter, k_scale, v_scale)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = dsa.kv_append_fp4(k, v, slots, cache, pos, cs, q=q, interleaved=inter, status=status, k_scale=k_scale,
                            v_scale=v_scale, **kw)
    assert int(status) == want_status
    for a, b, what in zip(F.views(cache.cpu().numpy(), dim), F.views(want, dim), ("k", "v", "k scale", "v scale")):
        np.testing.assert_array_equal(a, b, err_msg=what)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)        # ... and the padding is as it was
    if q is None:
        assert got is None
    else:
        pages = k.shape[0] // 64 + 2
        kc, vc = (torch.zeros((pages, 64) + tuple(k.shape[1:]), dtype=k.dtype, device="cuda") for _ in range(2))
        assert torch.equal(got, dsa.kv_append(k, v, torch.full_like(slots, -1), kc, vc, pos, cs, q=q,
                                              interleaved=inter))
    # what the slots hold, read back
    real = ((slots >= 0) & (slots < cache.shape[0] * 64)).cpu()
    at = slots.cpu()[real].numpy()
    for dtype in ("bf16", "fp16"):
        back = dsa.kv_read_fp4(torch.where(real.cuda(), slots, -1), cache, dim, DT[dtype], k_scale=k_scale,
                               v_scale=v_scale)
        for x, all_values in zip(back, F.decode(want, dim, k_scale, v_scale)):
            ref = torch.zeros(k.shape, dtype=DT[dtype])
            ref[real] = torch.from_numpy(all_values[at // 64, at % 64]).float().to(DT[dtype])   # FP32's (c s) g, rounded
            torch.testing.assert_close(x.cpu(), ref, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hkv,dim,rot,layers", [
    (1, 8, 2, 128, 128, 1), (3, 32, 8, 128, 64, 2), (77, 5, 5, 80, 32, 1), (130, 6, 1, 96, 96, 3), (40, 4, 2, 64, 64, 1),
    (5, 2, 1, 16, 16, 1), (7, 3, 3, 112, 48, 1), (9, 1, 1, 128, 16, 1), (20, 2, 2, 80, 80, 1), (11, 2, 7, 32, 32, 2),
    (700, 4, 4, 64, 48, 1), (650, 33, 3, 128, 112, 1), (5, 1, 2, 48, 48, 1)])
def test_append(cuda_lib, n, hq, hkv, dim, rot, layers, inter, dtype):
    check(cuda_lib, *case(n, hq, hkv, dim, rot, dtype, layers), inter)


@pytest.mark.parametrize("k_scale,v_scale", [(0.25, 2.0), (0.37, 1.9e-5), (2.0 ** 64, 2.0 ** -64), (3.3e7, 7.1)])
def test_scales(cuda_lib, k_scale, v_scale):
    for dtype in ("bf16", "fp16"):
        check(cuda_lib, *case(90, 4, 2, 96, 64, dtype), k_scale=k_scale, v_scale=v_scale)


def test_append_without_rotation_or_queries(cuda_lib):
    q, k, v, slots, cache, pos, _ = case(50, 4, 2, 64, 0, "bf16")
    check(cuda_lib, None, k, v, slots, cache, None, None)
    check(cuda_lib, q, k, v, slots, cache, None, None)
    q, k, v, slots, cache, pos, cs = case(50, 4, 2, 80, 48, "fp16")
    check(cuda_lib, None, k, v, slots, cache, pos, cs, True)
    check(cuda_lib, None, k, v, slots, cache, pos, cs, False)


def test_padding_bad_slots_and_positions(cuda_lib):
    q, k, v, slots, cache, pos, cs = case(8, 4, 2, 64, 32, "bf16")
    slots[2] = -1
    pos[2] = 10 ** 12                                    # a padding token's position is clamped and not flagged
    check(cuda_lib, q, k, v, slots, cache, pos, cs)
    slots[3] = cache.shape[0] * 64                       # past the pool
    check(cuda_lib, q, k, v, slots, cache, pos, cs, want_status=1)
    slots[3] = 2 ** 62
    pos[4], pos[5] = -3, 500
    check(cuda_lib, q, k, v, slots, cache, pos, cs, want_status=5)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    check(cuda_lib, q[:0], k[:0], v[:0], none, cache, none, cs)
    check(cuda_lib, q, k, v, torch.full_like(slots, -1), pool(0, 2, 64), pos, cs)


def test_every_bf16_value(cuda_lib):
    """All BF16 patterns, NaN and infinities among them, as blocks of neighbours and as blocks next to ones."""
    bits = np.arange(65536, dtype=np.uint16).reshape(-1, 1, 16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    ones = x.clone()
    ones[:, :, 1:] = torch.tensor([1.0, -0.75, 2.5, 5.0, -3.5, 1.25, 0.0, -0.0, 1.75, 6.0, 0.25, -0.5, 3.0, 4.0, 0.7],
                                  dtype=torch.bfloat16).cuda()
    slots = torch.arange(4096, device="cuda")
    for g in (1.0, 0.3, 2.0 ** -60, 1e12):
        check(cuda_lib, None, x, ones, slots, pool(64, 1, 16), None, None, k_scale=g, v_scale=g)


def test_every_tie(cuda_lib):
    """Values on the borders between codes, and beside them, for every scale that a block can get."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    scales = np.array([float(F.e4m3_decode(i)) for i in range(1, 0x7F)])
    rows = []
    for near in (0, -1, 1):
        b = np.concatenate([borders, -borders])
        b = np.nextafter(b.astype(np.float16), np.float16(near * 1000)).astype(np.float64) if near else b
        b[7] = 6.0                                        # the block's scale is the one wanted
        rows.append(scales[:, None] * b)
    x = torch.from_numpy(np.concatenate(rows)).float().to(torch.float16)[:, None, :].cuda()
    slots = torch.arange(x.shape[0], device="cuda")
    check(cuda_lib, None, x, x * 0.5, slots, pool(6, 1, 16), None, None, k_scale=1.0, v_scale=0.5)


def test_in_place_equals_out_of_place(cuda_lib):
    q, k, v, slots, cache, pos, cs = case(300, 8, 2, 128, 128, "bf16")
    a = cuda_lib.kv_append_fp4(k, v, slots, cache, pos, cs, q=q)
    b = cuda_lib.kv_append_fp4(k, v, slots, cache, pos, cs, q=q, q_out=q)
    assert b is q and torch.equal(a, b)


def test_read_into_views_and_past_the_pool(cuda_lib):
    q, k, v, slots, cache, pos, cs = case(70, 1, 3, 96, 96, "bf16", layers=2)
    cuda_lib.kv_append_fp4(k, v, slots, cache, pos, cs)
    want = cuda_lib.kv_read_fp4(slots, cache, 96)
    both = torch.full((70, 2, 3, 104), 7.0, dtype=torch.bfloat16, device="cuda")
    got = cuda_lib.kv_read_fp4(slots, cache, 96, k_out=both[:, 0, :, :96], v_out=both[:, 1, :, :96])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((both[..., 96:] == 7).all())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots[3], slots[5] = cache.shape[0] * 64, -9
    got = cuda_lib.kv_read_fp4(slots, cache, 96, status=status)
    assert int(status) == 1
    for a, b in zip(got, want):
        assert not a[3].any() and not a[5].any() and torch.equal(a[6:], b[6:])
    assert cuda_lib.kv_read_fp4(slots[:0], cache, 96)[0].shape == (0, 3, 96)


@pytest.mark.parametrize("at,width", [(0, 96), (0, 104), (8, 112), (16, 112), (8, 104)])
def test_read_into_any_alignment(cuda_lib, at, width):
    """Rows that begin on 32 bytes, and on 16 only."""
    q, k, v, slots, cache, pos, cs = case(67, 1, 3, 80, 80, "fp16")
    cuda_lib.kv_append_fp4(k, v, slots, cache, pos, cs)
    want = cuda_lib.kv_read_fp4(slots, cache, 80, torch.float16)
    room = torch.full((2, 67, 3, width), 7.0, dtype=torch.float16, device="cuda")
    got = cuda_lib.kv_read_fp4(slots, cache, 80, torch.float16, k_out=room[0][..., at:at + 80], v_out=room[1][..., at:at + 80])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((room[..., :at] == 7).all()) and bool((room[..., at + 80:] == 7).all())


def test_far_pages(cuda_lib):
    """Sections past 2^32 bytes of the pool."""
    pages, heads, dim = 60000, 8, 128                     # 4.4 GB
    q, k, v, slots, _, pos, cs = case(5, 2, heads, dim, 128, "bf16")
    cache = torch.zeros((pages, heads, F.section_bytes(dim)), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([pages * 64 - 1, pages * 64 - 64, 59000 * 64 + 3, 58255 * 64, 7], device="cuda")
    cuda_lib.kv_append_fp4(k, v, slots, cache, pos, cs)
    near = torch.arange(5, device="cuda")
    small = torch.zeros((1, heads, F.section_bytes(dim)), dtype=torch.uint8, device="cuda")
    cuda_lib.kv_append_fp4(k, v, near, small, pos, cs)
    for a, b in zip(cuda_lib.kv_read_fp4(slots, cache, dim), cuda_lib.kv_read_fp4(near, small, dim)):
        assert torch.equal(a, b) and bool(a.any())
