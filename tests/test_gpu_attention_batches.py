"""The layer's decode step for batches that change from step to step."""

import pytest
import torch

from synth import make_workload
from test_gpu_attention_step import build, check

pytestmark = pytest.mark.gpu


def first(a, wl, requests):
    """The arguments of a step of the first requests."""
    n = int(wl.query_lens[:requests].sum())
    return {k: v[:requests] if k in ("seq_lens", "query_lens") else v[:n] for k, v in a.items()}


@pytest.mark.parametrize("name,over", [("tiny_fp8", dict(R=5, seq=(70, 300))),
                                       ("spec_verify", dict(R=12, seq=(100, 900), topk=64))])
def test_a_step_of_fewer_requests_than_the_block_table(cuda_lib, name, over):
    wl = make_workload(name, **over)
    layer, a = build(wl)
    for requests in (wl.R, 1, wl.R // 2, wl.R, 2):
        s = first(a, wl, requests)
        out, chosen = layer.step(**s)
        assert out.shape[0] == s["q"].shape[0] and chosen.starts.numel() == requests + 1
        q = cuda_lib.kv_append(s["k"], s["v"], s["slots"], layer.k_cache, layer.v_cache, s["positions"], layer.cos_sin,
                               q=s["q"])
        check(layer, q, out, chosen.starts, chosen.row_ends, chosen.topk)
        dense = layer.dense_step(s["q"], s["k"], s["v"], s["slots"], s["positions"], chosen.starts, chosen.row_ends)
        check(layer, q, dense, chosen.starts, chosen.row_ends)


def test_a_step_without_requests(cuda_lib):
    wl = make_workload("tiny_fp8", R=3, seq=(70, 300))
    layer, a = build(wl)
    s = {k: v[:0] for k, v in a.items()}
    out, chosen = layer.step(**s)
    assert out.shape[0] == 0 and chosen.topk.shape[0] == 0
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    dense = layer.dense_step(s["q"], s["k"], s["v"], s["slots"], s["positions"], starts, chosen.row_ends)
    assert dense.shape[0] == 0 and layer.indexer.status_bits() == 0
