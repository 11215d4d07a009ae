"""The layer's decode step (indexer, append, attention) on seeded workloads."""

import numpy as np
import pytest
import torch

from dsa_case import bf16_tensor
from oracle import attention as A
from synth import make_workload

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, DIM = 8, 2, 64


def build(wl):
    from sparse_attention_indexer_score_gb300.attention import DecodeAttention, angle_table
    from sparse_attention_indexer_score_gb300.step import DecodeIndexer

    dev = torch.device("cuda")
    ix = DecodeIndexer(wl.fmt, wl.num_pages, torch.from_numpy(wl.block_table), torch.from_numpy(wl.gamma),
                       torch.from_numpy(wl.beta), wl.eps, wl.num_rows, wl.topk, dev)
    most = int(wl.query_lens.max())
    layer = DecodeAttention(ix, HEADS, KV_HEADS, DIM, angle_table(int(wl.seq_lens.max()) + 1, DIM), wl.num_rows, most)
    g = torch.Generator().manual_seed(wl.seed)
    for r in range(wl.R):
        bits, slots = wl.prefill(r)
        n = len(slots)
        if n:
            ix.insert(bf16_tensor(bits, dev), torch.from_numpy(slots).to(dev))
            kv = torch.randn((2, n, KV_HEADS, DIM), generator=g).to(torch.bfloat16).to(dev)
            layer.append(kv[0], kv[1], torch.from_numpy(slots).to(dev), torch.arange(n, device=dev))
    n = wl.num_rows
    t = lambda a: torch.from_numpy(a).to(dev)   # noqa: E731
    args = dict(iq=bf16_tensor(wl.q_bits, dev), wv=bf16_tensor(wl.wv_bits, dev), ikeys=bf16_tensor(wl.step_key_bits, dev),
                q=torch.randn((n, HEADS, DIM), generator=g).to(torch.bfloat16).to(dev),
                k=torch.randn((n, KV_HEADS, DIM), generator=g).to(torch.bfloat16).to(dev),
                v=torch.randn((n, KV_HEADS, DIM), generator=g).to(torch.bfloat16).to(dev), slots=t(wl.step_slots),
                positions=t(np.maximum(wl.row_position, 0)), seq_lens=t(wl.seq_lens), query_lens=t(wl.query_lens))
    return layer, args


def check(layer, q, out, starts, ends, topk=None):
    """Against the 64-bit formula on the cache and the rotated queries that the append produced (the append has
    its own tests); roundings as in attend_case."""
    k, v = layer.k_cache.double().cpu().numpy(), layer.v_cache.double().cpu().numpy()
    q, out, table = q.double().cpu().numpy(), out.double().cpu().numpy(), layer.indexer.block_table.tolist()
    starts, ends = starts.tolist(), ends.tolist()
    topk = None if topk is None else topk.tolist()
    eps = torch.finfo(torch.bfloat16).eps
    for r in range(q.shape[0]):
        keys = A.visible(r, starts, ends, table, topk=topk)
        o, _, mean_abs, size = A.attend(q[r], k, v, keys, DIM ** -0.5)
        tol = eps / 2 * np.abs(o) + (eps / 2 + 2.0 ** -20 + 4 * 2.0 ** -24 * (DIM + 4) * size[:, None]) * mean_abs
        assert (np.abs(out[r] - o) <= tol).all(), (r, len(keys), np.abs(out[r] - o).max())
    assert layer.indexer.status_bits() == 0


@pytest.mark.parametrize("name,over", [("tiny_fp8", {}), ("spec_verify", dict(R=6, seq=(100, 700), topk=64)),
                                       ("mxfp4_decode", dict(R=3, seq=(40, 900), topk=130))])
def test_layer_step(cuda_lib, name, over):
    wl = make_workload(name, **over)
    layer, a = build(wl)
    out, chosen = layer.step(**a)
    q = cuda_lib.kv_append(a["k"], a["v"], a["slots"], layer.k_cache, layer.v_cache, a["positions"], layer.cos_sin,
                           q=a["q"])
    check(layer, q, out, chosen.starts, chosen.row_ends, chosen.topk)
    dense = layer.dense_step(a["q"], a["k"], a["v"], a["slots"], a["positions"], chosen.starts, chosen.row_ends)
    check(layer, q, dense, chosen.starts, chosen.row_ends)


def test_rows_with_few_keys_attend_to_all_of_them(cuda_lib):
    """Up to top-k keys the selection is every key: both steps see the same."""
    wl = make_workload("tiny_fp8", seq=(30, 64), topk=64, R=5)
    layer, a = build(wl)
    out, chosen = layer.step(**a)
    dense = layer.dense_step(a["q"], a["k"], a["v"], a["slots"], a["positions"], chosen.starts, chosen.row_ends)
    # the same tile of keys in the same order, in one kernel or the other
    assert torch.equal(out, dense)


def test_layer_step_in_a_graph(cuda_lib):
    wl = make_workload("tiny_fp8", R=3, seq=(70, 300))
    layer, a = build(wl)
    eager, _ = layer.step(**a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, chosen = layer.step(**a)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    q = cuda_lib.kv_append(a["k"], a["v"], a["slots"], layer.k_cache, layer.v_cache, a["positions"], layer.cos_sin,
                           q=a["q"])
    check(layer, q, out, chosen.starts, chosen.row_ends, chosen.topk)
