"""The layer's step in its other forms: FP16 caches, adjacent pairs, partial rotation, a scale of its own, and a prefix
that the batch shares."""

import numpy as np
import pytest
import torch

from dsa_case import bf16_tensor
from oracle import attention as A
from synth import make_workload

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, DIM, PREFIX = 12, 2, 96, 150
FORMS = [dict(dtype=torch.float16), dict(interleaved=True), dict(scale=0.05), dict(rot=32),
         dict(dtype=torch.float16, interleaved=True, scale=0.2, rot=64)]


def build(wl, rot=DIM, dtype=torch.bfloat16, **kw):
    """The layer over a pool with room for the prefix behind the workload's pages, its prompts appended."""
    from sparse_attention_indexer_score_gb300.attention import DecodeAttention, angle_table
    from sparse_attention_indexer_score_gb300.step import DecodeIndexer

    dev, more = torch.device("cuda"), -(-PREFIX // 64)
    ix = DecodeIndexer(wl.fmt, wl.num_pages + more, torch.from_numpy(wl.block_table), torch.from_numpy(wl.gamma),
                       torch.from_numpy(wl.beta), wl.eps, wl.num_rows, wl.topk, dev)
    layer = DecodeAttention(ix, HEADS, KV_HEADS, DIM, angle_table(int(wl.seq_lens.max()) + PREFIX + 1, rot), wl.num_rows,
                            int(wl.query_lens.max()), dtype=dtype, **kw)
    g = torch.Generator().manual_seed(wl.seed)
    rand = lambda *n: torch.randn(n, generator=g).to(dtype).to(dev)   # noqa: E731
    for r in range(wl.R):
        bits, slots = wl.prefill(r)
        n = len(slots)
        if n:
            ix.insert(bf16_tensor(bits, dev), torch.from_numpy(slots).to(dev))
            layer.append(rand(n, KV_HEADS, DIM), rand(n, KV_HEADS, DIM), torch.from_numpy(slots).to(dev),
                         torch.arange(n, device=dev))
    pages = torch.arange(wl.num_pages, wl.num_pages + more, dtype=torch.int32, device=dev).flip(0)
    at = torch.arange(PREFIX, device=dev)
    layer.append(rand(PREFIX, KV_HEADS, DIM), rand(PREFIX, KV_HEADS, DIM), pages.long()[at // 64] * 64 + at % 64, at)
    t = lambda a: torch.from_numpy(a).to(dev)   # noqa: E731
    n = wl.num_rows
    args = dict(iq=bf16_tensor(wl.q_bits, dev), wv=bf16_tensor(wl.wv_bits, dev), ikeys=bf16_tensor(wl.step_key_bits, dev),
                q=rand(n, HEADS, DIM), k=rand(n, KV_HEADS, DIM), v=rand(n, KV_HEADS, DIM), slots=t(wl.step_slots),
                positions=t(np.maximum(wl.row_position, 0)), seq_lens=t(wl.seq_lens), query_lens=t(wl.query_lens))
    return layer, args, pages


def append_reference(layer, a):
    """Rotated queries and the step's rows of the cache against the 64-bit form; returns the rotated queries."""
    k, v, q, cs = (t.double().cpu().numpy() for t in (a["k"], a["v"], a["q"], layer.cos_sin))
    kc, vc = (np.zeros(tuple(t.shape)) for t in (layer.k_cache, layer.v_cache))
    slots = a["slots"].tolist()
    want = A.append(k, v, slots, kc, vc, a["positions"].tolist(), cs, q, layer.interleaved)
    got = layer.append(a["k"], a["v"], a["slots"], a["positions"], a["q"]).double().cpu().numpy()
    eps = torch.finfo(layer.k_cache.dtype).eps
    worst = 2.0 ** -22 * float(max(np.abs(k).max(), np.abs(q).max())) + 2.0 ** -25
    assert (np.abs(got - want) <= eps / 2 * np.abs(want) + worst).all()
    have = layer.k_cache.double().cpu().numpy()
    for s in slots:
        if s >= 0:
            assert (np.abs(have[s // 64, s % 64] - kc[s // 64, s % 64]) <= eps / 2 * np.abs(kc[s // 64, s % 64]) + worst).all()
    return got


def check(layer, q, out, starts, ends, topk=None, pages=(), prefix=0):
    k, v = layer.k_cache.double().cpu().numpy(), layer.v_cache.double().cpu().numpy()
    out, table = out.double().cpu().numpy(), layer.indexer.block_table.tolist()
    starts, ends = starts.tolist(), ends.tolist()
    scale = DIM ** -0.5 if layer.scale is None else layer.scale
    eps = torch.finfo(layer.k_cache.dtype).eps
    small = 2.0 ** -25 if layer.k_cache.dtype == torch.float16 else 0.0
    for r in range(out.shape[0]):
        keys = A.visible(r, starts, ends, table, pages, prefix, topk)
        o, _, mean_abs, size = A.attend(q[r], k, v, keys, scale)
        tol = eps / 2 * np.abs(o) + (eps / 2 + 2.0 ** -20 + 4 * 2.0 ** -24 * (DIM + 4) * size[:, None]) * mean_abs
        if keys:   # (FP16 weights below 2^-14: 2^-32 of the largest each)
            tol += small + len(keys) * small * 2.0 ** -7 * np.abs(v[tuple(np.array(keys).T)]).max()
        assert (np.abs(out[r] - o) <= tol).all(), (r, len(keys), np.abs(out[r] - o).max())
    assert layer.indexer.status_bits() == 0


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(f))
def test_forms_of_the_layer(cuda_lib, form):
    wl = make_workload("spec_verify", R=5, seq=(100, 500), topk=64)
    layer, a, pages = build(wl, **form)
    out, chosen = layer.step(**a)
    q = append_reference(layer, a)
    check(layer, q, out, chosen.starts, chosen.row_ends, chosen.topk.tolist())
    dense = layer.dense_step(a["q"], a["k"], a["v"], a["slots"], a["positions"], chosen.starts, chosen.row_ends)
    check(layer, q, dense, chosen.starts, chosen.row_ends)
    for n in (PREFIX, 64, 1):
        dense = layer.dense_step(a["q"], a["k"], a["v"], a["slots"], a["positions"], chosen.starts, chosen.row_ends,
                                 prefix_pages=pages, prefix_len=n)
        check(layer, q, dense, chosen.starts, chosen.row_ends, pages=pages.tolist(), prefix=n)
