"""The layer's decode step over a 4-bit cache: indexer, quantising append, attention, reading back."""

import numpy as np
import pytest
import torch

from dsa_case import bf16_tensor
from fp4_case import DT
from oracle import attention as A
from oracle import fp4_cache as F
from synth import make_workload

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, DIM = 8, 2, 64
SCALES = dict(k_scale=0.5, v_scale=2.0)


def build(wl, dtype="bf16"):
    from sparse_attention_indexer_score_gb300.attention import DecodeAttention, angle_table
    from sparse_attention_indexer_score_gb300.step import DecodeIndexer

    dev = torch.device("cuda")
    ix = DecodeIndexer(wl.fmt, wl.num_pages, torch.from_numpy(wl.block_table), torch.from_numpy(wl.gamma),
                       torch.from_numpy(wl.beta), wl.eps, wl.num_rows, wl.topk, dev)
    layer = DecodeAttention(ix, HEADS, KV_HEADS, DIM, angle_table(int(wl.seq_lens.max()) + 1, DIM), wl.num_rows,
                            int(wl.query_lens.max()), dtype=DT[dtype], kv_format="nvfp4", **SCALES)
    g = torch.Generator().manual_seed(wl.seed)
    for r in range(wl.R):
        bits, slots = wl.prefill(r)
        n = len(slots)
        if n:
            ix.insert(bf16_tensor(bits, dev), torch.from_numpy(slots).to(dev))
            kv = torch.randn((2, n, KV_HEADS, DIM), generator=g).to(DT[dtype]).to(dev)
            layer.append(kv[0], kv[1], torch.from_numpy(slots).to(dev), torch.arange(n, device=dev))
    n = wl.num_rows
    t = lambda a: torch.from_numpy(a).to(dev)   # noqa: E731
    r = lambda h: torch.randn((n, h, DIM), generator=g).to(DT[dtype]).to(dev)   # noqa: E731
    args = dict(iq=bf16_tensor(wl.q_bits, dev), wv=bf16_tensor(wl.wv_bits, dev), ikeys=bf16_tensor(wl.step_key_bits, dev),
                q=r(HEADS), k=r(KV_HEADS), v=r(KV_HEADS), slots=t(wl.step_slots),
                positions=t(np.maximum(wl.row_position, 0)), seq_lens=t(wl.seq_lens), query_lens=t(wl.query_lens))
    return layer, args


def check(layer, q, out, starts, ends, topk=None):
    """Against the 64-bit formula on what the cache holds (the append has its own tests); roundings as in fp4_case."""
    k, v = F.decode(layer.kv_cache.cpu().numpy(), DIM, **SCALES)
    eps = torch.finfo(out.dtype).eps
    q, out, table = q.double().cpu().numpy(), out.double().cpu().numpy(), layer.indexer.block_table.tolist()
    starts, ends = starts.tolist(), ends.tolist()
    topk = None if topk is None else topk.tolist()
    for r in range(q.shape[0]):
        keys = A.visible(r, starts, ends, table, topk=topk)
        o, _, mean_abs, size = A.attend(q[r], k, v, keys, DIM ** -0.5)
        tol = eps / 2 * np.abs(o) + (2.0 ** -11 + 2.0 ** -20 + 4 * 2.0 ** -24 * (DIM + 4) * size[:, None] +
                                     2.0 ** -23 * (len(keys) / 16 + 64)) * mean_abs
        if keys:
            tol += len(keys) * 2.0 ** -31 * np.abs(v[tuple(np.array(keys).T)]).max() + 2.0 ** -25
        assert (np.abs(out[r] - o) <= tol).all(), (r, len(keys), np.abs(out[r] - o).max())
    assert layer.indexer.status_bits() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name,over", [("tiny_fp8", {}), ("spec_verify", dict(R=6, seq=(100, 700), topk=64)),
                                       ("mxfp4_decode", dict(R=30, seq=(40, 900), topk=130))])
def test_layer_step(cuda_lib, name, over, dtype):
    layer, a = build(make_workload(name, **over), dtype)
    out, chosen = layer.step(**a)
    q = layer.append(a["k"], a["v"], a["slots"], a["positions"], a["q"])
    check(layer, q, out, chosen.starts, chosen.row_ends, chosen.topk)
    dense = layer.dense_step(a["q"], a["k"], a["v"], a["slots"], a["positions"], chosen.starts, chosen.row_ends)
    check(layer, q, dense, chosen.starts, chosen.row_ends)
    slots = a["slots"].cpu().numpy()
    for got, held in zip(layer.read(a["slots"]), F.decode(layer.kv_cache.cpu().numpy(), DIM, **SCALES)):
        want = np.where((slots >= 0)[:, None, None], held[slots // 64, slots % 64], 0)
        assert torch.equal(got.cpu(), torch.from_numpy(want).float().to(DT[dtype]))


def test_layer_step_in_a_graph(cuda_lib):
    layer, a = build(make_workload("tiny_fp8", R=3, seq=(70, 300)))
    layer.step(**a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, chosen = layer.step(**a)
        dense = layer.dense_step(a["q"], a["k"], a["v"], a["slots"], a["positions"], chosen.starts, chosen.row_ends)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    q = layer.append(a["k"], a["v"], a["slots"], a["positions"], a["q"])
    check(layer, q, out, chosen.starts, chosen.row_ends, chosen.topk)
    check(layer, q, dense, chosen.starts, chosen.row_ends)


def _rows(layer, a):
    chosen = layer.indexer.step(a["iq"], a["wv"], a["ikeys"], a["slots"], a["seq_lens"], a["query_lens"],
                                layer.max_query_len)
    return chosen.starts, chosen.row_ends


def test_what_a_four_bit_layer_refuses(cuda_lib):
    layer, a = build(make_workload("tiny_fp8"))
    starts, ends = _rows(layer, a)
    with pytest.raises(ValueError, match="prefix"):
        layer.dense_step(a["q"], a["k"], a["v"], a["slots"], a["positions"], starts, ends,
                         prefix_pages=torch.zeros(1, dtype=torch.int32, device="cuda"), prefix_len=10)
    from test_gpu_attention_step import build as build16

    with pytest.raises(ValueError, match="16-bit"):
        build16(make_workload("tiny_fp8"))[0].read(a["slots"])
