"""The 4-bit calls over caches whose heads lie outside their pages, over block tables that are a part of a wider one's
columns and rows, in inference mode, and captured before they ever ran."""

import os
import subprocess
import sys

import pytest
import torch

from fp4_case import Case, choose

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 64), (16, 4, 128), (6, 2, 80)])
def test_heads_outside_pages(cuda_lib, hq, hkv, dim):
    c = Case([70, 300, 1], [2, 1, 1], hq=hq, hkv=hkv, dim=dim)
    topk = choose(c, 50)
    want = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    slots = torch.tensor([3, 64, -1, 130], device="cuda")
    kv = torch.randn((2, 4, hkv, dim), device="cuda").bfloat16()
    pages = c.cache.shape[0]
    other = torch.full((hkv, pages, c.cache.shape[2] + 48), 0xFF, dtype=torch.uint8, device="cuda")
    view = other[:, :, :c.cache.shape[2]].transpose(0, 1)
    assert view.stride(0) < view.stride(1)
    view.copy_(c.cache)
    plain, c.cache = c.cache, view
    got = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for cache in (plain, view):
        cuda_lib.kv_append_fp4(kv[0], kv[1], slots, cache)
    assert torch.equal(plain, view)
    assert bool((other[:, :, c.cache.shape[2]:] == 0xFF).all())
    for a, b in zip(cuda_lib.kv_read_fp4(slots, plain, dim), cuda_lib.kv_read_fp4(slots, view, dim)):
        assert torch.equal(a, b) and bool(a[2].eq(0).all())


def test_a_part_of_a_table(cuda_lib):
    c = Case([70, 300, 1000], [2, 1, 1], hq=8, hkv=2, dim=128)
    topk = choose(c, 50)
    want = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    n, m = c.block_table.shape
    wide = torch.full((n + 4, m + 9), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[2:2 + n, 5:5 + m] = c.block_table
    c.block_table = wide[2:2 + n, 5:5 + m]
    got = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_in_inference_mode(cuda_lib):
    c = Case([70, 300], [2, 1], hq=8, hkv=2, dim=64)
    topk = choose(c, 50)
    want = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
    with torch.inference_mode():
        got = c.paged(cuda_lib) + c.selected(cuda_lib, topk)
        assert all(t.is_inference() for t in got)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def captured_first():
    """In a process of its own: every call's first run is its capture."""
    from sparse_attention_indexer_score_gb300 import dsa

    small = Case([70, 300], [2, 1], hq=8, hkv=2, dim=64)
    large = Case([300 + j for j in range(200)], [1] * 200, hq=32, hkv=4, dim=128)
    lists = [choose(c, 700) for c in (small, large)]
    slots, kv = torch.tensor([3, 64, -1], device="cuda"), torch.randn((2, 3, 2, 64), device="cuda").bfloat16()
    cache = dsa.new_kv_cache_fp4(2, 2, 64, "cuda")

    def run():
        dsa.kv_append_fp4(kv[0], kv[1], slots, cache)
        out = dsa.kv_read_fp4(slots, cache, 64)
        for c, topk in zip((small, large), lists):
            out += c.paged(dsa) + c.selected(dsa, topk)
        return out

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, run()))
    large.check(got[6:8], rows=range(0, 200, 40))
    print("captured first")


def test_captured_before_it_ever_ran(cuda_lib):
    here = os.path.dirname(os.path.abspath(__file__))
    code = "import sys; sys.path[:0] = [%r, %r]\nimport test_gpu_fp4_layouts as t\nt.captured_first()" % (os.path.dirname(here), here)
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "captured first" in got.stdout, got.stderr[-2000:]
