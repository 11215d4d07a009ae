"""What the attention calls ask of their workspace: nothing but its size."""

import pytest
import torch

from attend_case import Case, choose

pytestmark = pytest.mark.gpu


def cases():
    """Plans made in the CTAs and by their kernel, prefixes on the axis and in pairs of row tiles."""
    yield Case([3000, 100, 777], [2, 1, 1], prefix=1500, hq=16, hkv=2, dim=128)
    yield Case([(53 * j) % 301 for j in range(300)], [1 + j % 2 for j in range(300)], hq=4, hkv=2, dim=64)
    yield Case([(37 * j) % 150 for j in range(65)], [1] * 65, prefix=7301, hq=128, hkv=1, dim=64, pad_rows=1)


def sizes(dsa, c, k):
    rows, hq, dim = c.q.shape
    args = (rows, c.block_table.shape[0], hq, c.k.shape[2], dim)
    return dsa.attend_workspace_size(*args, c.qlen), dsa.attend_workspace_size(*args, 1, k)


def test_any_bytes_may_be_in_a_workspace(cuda_lib):
    for c in cases():
        topk = choose(c, 100)
        n = max(sizes(cuda_lib, c, 100))
        results = []
        for byte in (0, 0x7F, 0xFF):
            ws = torch.full((n,), byte, dtype=torch.uint8, device="cuda")
            results.append(c.paged(cuda_lib, workspace=ws) + c.selected(cuda_lib, topk, workspace=ws.fill_(byte)))
        for r in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], r))


def test_a_call_does_not_clear_its_own_workspace(cuda_lib):
    """The bytes of a buffer that the allocator gives to the call next are still there afterwards, but for what the
    call wrote (pieces' results, which fill a small part)."""
    c = Case([90, 70], [1, 1], hq=64, hkv=8, dim=128)
    topk = choose(c, 40)
    for call, n in zip((lambda: c.paged(cuda_lib), lambda: c.selected(cuda_lib, topk)), sizes(cuda_lib, c, 40)):
        assert n > 1 << 20                       # a block of its own, not one of the small ones
        kept = call()                            # (library loaded, small blocks there)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
        got = call()
        left = torch.empty((n,), dtype=torch.uint8, device="cuda")
        assert int((left == 0xAB).sum()) > n // 2
        assert all(torch.equal(a, b) for a, b in zip(kept, got))


def test_scoring_after_attention_in_the_layer(cuda_lib):
    """A layer's indexer has a workspace of its own, which attention does not touch."""
    from test_gpu_attention_step import build
    from synth import make_workload

    layer, a = build(make_workload("tiny_fp8", R=3, seq=(70, 300)))
    chosen = layer.step(**a)[1]
    first = chosen.topk.sort(dim=1).values           # (a set of positions, in any order)
    for _ in range(2):
        layer.dense_step(a["q"], a["k"], a["v"], a["slots"], a["positions"], chosen.starts, chosen.row_ends)
        assert torch.equal(layer.step(**a)[1].topk.sort(dim=1).values, first)
