"""Which way a batch takes through the 4-bit attention, and its results: requests of very different row counts go by
the axis (an attention kernel and a join), alike ones to a cluster an item (one kernel)."""

import ctypes

import pytest
import torch

from fp4_case import Case

pytestmark = pytest.mark.gpu


def launches(call):
    """Kernels of a call, from its capture."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = ctypes.c_size_t(0)
    rc = ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n))
    assert rc == 0
    return n.value


def paged(dsa, c, hint=None):
    """The call with a workspace and an output of its own, as a captured step makes it."""
    rows, hq, dim = c.q.shape
    hint = c.qlen if hint is None else hint
    size = dsa.attend_workspace_size_fp4(rows, c.starts.numel() - 1, hq, c.hkv, dim, hint)
    ws, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty_like(c.q)
    return lambda: c.paged(dsa, max_query_len=hint, workspace=ws, out=out, want_lse=False)


@pytest.mark.parametrize("lens,qlens,hq,hkv,dim", [
    ([600 + j for j in range(64)], [1] * 63 + [67], 16, 1, 128),          # 34 tiles in one request
    ([500] * 64, [0] * 63 + [64], 16, 1, 64),                             # the others idle
    ([40 + 30 * j for j in range(9)], [1] * 4 + [32] + [1] * 4, 32, 8, 128),
    ([300] * 120, [150] + [1] * 119, 1, 1, 80)])
def test_one_long_request_among_short_ones(cuda_lib, lens, qlens, hq, hkv, dim):
    c = Case(lens, qlens, hq=hq, hkv=hkv, dim=dim)
    c.check(c.paged(cuda_lib), rows=range(0, c.q.shape[0], 3))
    assert launches(paged(cuda_lib, c)) == 2


@pytest.mark.parametrize("lens,qlens,hq,hkv,dim", [
    ([600 + j for j in range(64)], [2] * 64, 16, 1, 128), ([500] * 30, [1] * 29 + [4], 16, 1, 64),
    ([1000], [1], 32, 8, 128), ([40 + 30 * j for j in range(9)], [1] * 8 + [16], 32, 8, 128)])
def test_requests_of_one_or_two_tiles(cuda_lib, lens, qlens, hq, hkv, dim):
    c = Case(lens, qlens, hq=hq, hkv=hkv, dim=dim)
    c.check(c.paged(cuda_lib), rows=range(0, c.q.shape[0], 3))
    assert launches(paged(cuda_lib, c)) == 1
