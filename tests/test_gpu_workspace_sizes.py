"""Steps of different row counts on one workspace, as a serving loop makes them: each finds the top-k that it finds on
a workspace of its own."""

import pytest
import torch

from dsa_case import bf16_tensor
from synth import make_workload

pytestmark = pytest.mark.gpu


def indexer(wl):
    from sparse_attention_indexer_score_gb300.step import DecodeIndexer

    dev = torch.device("cuda")
    ix = DecodeIndexer(wl.fmt, wl.num_pages, torch.from_numpy(wl.block_table), torch.from_numpy(wl.gamma),
                       torch.from_numpy(wl.beta), wl.eps, wl.num_rows, wl.topk, dev)
    for r in range(wl.R):
        bits, slots = wl.prefill(r)
        if len(slots):
            ix.insert(bf16_tensor(bits, dev), torch.from_numpy(slots).to(dev))
    return ix


def step(ix, wl, requests):
    """The step of the first `requests` requests; the rows' top-k as sets."""
    n = int(wl.query_lens[:requests].sum())
    t = lambda a: torch.from_numpy(a).cuda()   # noqa: E731
    out = ix.step(bf16_tensor(wl.q_bits[:n], "cuda"), bf16_tensor(wl.wv_bits[:n], "cuda"),
                  bf16_tensor(wl.step_key_bits[:n], "cuda"), t(wl.step_slots[:n]), t(wl.seq_lens[:requests]),
                  t(wl.query_lens[:requests]), int(wl.query_lens.max()))
    return [set(r) for r in out.topk.tolist()]


@pytest.mark.parametrize("name,over", [("spec_verify", dict(R=40, seq=(3000, 6000), topk=256)),
                                       ("mxfp4_decode", dict(R=60, seq=(600, 2500), topk=130)),
                                       ("tiny_fp8", dict(R=3, seq=(40000, 60000), topk=64))])
def test_rows_of_a_step_may_vary(cuda_lib, name, over):
    wl = make_workload(name, **over)
    ix = indexer(wl)
    fresh = ix.workspace
    order = [wl.R, 1, wl.R, 2, max(1, wl.R // 3), wl.R // 2 + 1, 1, wl.R]
    alone = {}
    for r in order:
        ix.workspace = torch.zeros_like(fresh)
        alone[r] = step(ix, wl, r)
    ix.workspace = fresh
    for r in order:
        got = step(ix, wl, r)
        assert got == alone[r], r
    assert ix.status_bits() == 0


def test_topk_calls_of_different_rows_share_a_workspace(cuda_lib):
    g = torch.Generator().manual_seed(2)
    ws = cuda_lib.new_workspace(cuda_lib.topk_workspace_size(90, 300), "cuda")
    for rows in (90, 3, 90, 1, 44, 90):
        x = torch.randn((rows, 20000), generator=g).cuda()
        ends = torch.full((rows,), 20000, dtype=torch.int32, device="cuda")
        got = cuda_lib.topk(x, ends, 300, workspace=ws)
        assert torch.equal(got.long().sort(dim=1).values, x.topk(300, dim=1).indices.sort(dim=1).values)
