"""Seeded cases of the 4-bit cache's attention tests, and their tolerances.

Codes times scales are exact, so the formula runs on what the cache's bytes stand
for.  An output is rounded once (eps / 2 of it), every softmax weight once to FP16
(2^-11 of the weighted mean of |v|), and a weight below 2^-20 of the largest keeps an
absolute half step of 2^-31 of the largest (weights are kept times 2^6, FP16 has
2^-25 there), times the largest |v|, for each key; outputs below 2^-14 in FP16
likewise 2^-25.  A score is a sum of dim products, off by at most
2^-24 (dim + 4) of scale * sum |q||k|, and a query column under 2^-28 of its head's
largest is off by 2^-39 of that one; both move every weight and their sum by that
much of themselves.  An exponential is good to 2^-20 of itself.  Outputs are sums of
one product of 16 keys after the other, each addition off by at most 2^-23.
"""

import numpy as np
import torch

from oracle import attention as A
from oracle import fp4_cache as F

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def pool(pages, heads, dim, layers=1, device="cuda", fill=0xFF):
    """A cache [pages, heads, section] full of `fill` (0xFF: NaN scales); with several layers, a view of their pool."""
    t = torch.full((pages, layers, heads, F.section_bytes(dim)), fill, dtype=torch.uint8, device=device)
    return t[:, layers - 1]


class Case:
    """Requests with `lens` keys and `qlens` rows; the scales are NaN wherever no row may look (and in the padding
    of the scale rows), and the block table -7 where a request has no page."""

    def __init__(self, lens, qlens, hq=8, hkv=2, dim=64, dtype="bf16", layers=1, pad_rows=0, seed=0, ends=None,
                 k_scale=1.0, v_scale=1.0, device="cuda", extra_pages=1, heat=None):
        rng = np.random.default_rng(seed)
        need = [-(-n // 64) for n in lens]
        pages = sum(need) + extra_pages
        perm = rng.permutation(pages)
        self.dim, self.hkv, self.scales = dim, hkv, dict(k_scale=k_scale, v_scale=v_scale)
        host = np.full((pages, hkv, F.section_bytes(dim)), 0xFF, dtype=np.uint8)
        parts = F.views(host, dim)
        table = np.full((len(lens), max(need + [0]) + 1), -7, dtype=np.int32)
        at = 0
        for j, n in enumerate(lens):
            p = perm[at:at + need[j]]
            table[j, :need[j]] = p
            at += need[j]
            for i in range(0, n, 64):
                m = min(64, n - i)
                for x in parts[:2]:
                    x[p[i // 64], :m] = rng.integers(0, 256, (m, hkv, dim // 2))
                for x in parts[2:]:      # normal scales, some subnormal, zero and negative ones
                    s = rng.integers(0x20, 0x38, (m, hkv, dim // 16))
                    odd = rng.random(s.shape)
                    s = np.where(odd < 0.02, rng.integers(0, 8, s.shape), s)
                    x[p[i // 64], :m] = np.where(odd > 0.98, s | 0x80, s)
        self.host = host
        self.cache = pool(pages, hkv, dim, layers, device)
        self.cache.copy_(torch.from_numpy(host))
        starts, bounds = [0], []
        for n, m in zip(lens, qlens):
            bounds += [max(0, n - m + i + 1) for i in range(m)]
            starts.append(starts[-1] + m)
        bounds += [5] * pad_rows                 # rows outside every request: no keys, whatever their bound
        if ends is not None:
            bounds = ends
        rows = len(bounds)
        h = np.linspace(0.2, 2.0, hq)[:, None] if heat is None else heat
        self.q = torch.from_numpy(rng.standard_normal((rows, hq, dim)) * h / k_scale).to(DT[dtype]).to(device)
        self.block_table = torch.from_numpy(table).to(device)
        self.starts = torch.tensor(starts, dtype=torch.int32, device=device)
        self.row_ends = torch.tensor(bounds, dtype=torch.int32, device=device)
        self.qlen, self.dtype, self.scale = max(qlens + [0]), dtype, dim ** -0.5

    def paged(self, dsa, **kw):
        return dsa.attend_paged_fp4(self.q, self.cache, self.block_table, self.starts, self.row_ends,
                                    **{**dict(max_query_len=self.qlen, want_lse=True), **self.scales, **kw})

    def selected(self, dsa, topk, **kw):
        return dsa.attend_selected_fp4(self.q, self.cache, self.block_table, self.starts, self.row_ends, topk,
                                       **{**dict(want_lse=True), **self.scales, **kw})

    def check(self, got, topk=None, rows=None, scale=None, heads=None):
        """Every output and log-sum-exp of `got` against the 64-bit formula."""
        out, lse = (t.double().cpu().numpy() for t in got)
        k, v = F.decode(self.host, self.dim, **self.scales)
        q = self.q.double().cpu().numpy()
        scale = self.scale if scale is None else scale
        starts, ends, table = self.starts.tolist(), self.row_ends.tolist(), self.block_table.tolist()
        lists = None if topk is None else topk.tolist()
        eps = torch.finfo(DT[self.dtype]).eps
        for r in range(q.shape[0]) if rows is None else rows:
            keys = A.visible(r, starts, ends, table, topk=lists)
            o, l, mean_abs, size = A.attend(q[r], k, v, keys, scale)
            if not keys:
                assert not out[r].any() and np.isneginf(lse[r]).all(), r
                continue
            at = tuple(np.array(keys).T)
            vmax, kmax = np.abs(v[at]).max(), np.abs(k[at]).max()
            moved = 2.0 ** -24 * (self.dim + 4) * size + \
                2.0 ** -39 * np.abs(q[r]).max(axis=1) * kmax * self.dim * scale
            tol = eps / 2 * np.abs(o) + (2.0 ** -11 + 2.0 ** -20 + 4 * moved[:, None] +
                                         2.0 ** -23 * (len(keys) / 16 + 64)) * mean_abs
            tol += len(keys) * 2.0 ** -31 * vmax + (2.0 ** -25 if self.dtype == "fp16" else 0)
            bad = np.abs(out[r] - o) > tol
            assert not bad.any(), (r, len(keys), float(np.abs(out[r] - o).max()), np.argwhere(bad)[:3])
            tol_l = 2 * moved + 2.0 ** -24 * (len(keys) + 64) + 2.0 ** -20 * np.maximum(1, np.abs(l))
            assert (np.abs(lse[r] - l) <= tol_l).all(), (r, np.abs(lse[r] - l).max(), tol_l.min())


def choose(case, k, seed=0, holes=True):
    """k distinct positions below each row's bound in random order; the rest -1, scattered if `holes`."""
    rng = np.random.default_rng(seed)
    rows = []
    for e in case.row_ends.tolist():
        n = min(k, max(e, 0))
        t = np.full(k, -1)
        t[:n] = rng.permutation(max(e, 0))[:n]
        if holes:
            t = rng.permutation(t)
        rows.append(t)
    return torch.tensor(np.array(rows).reshape(len(rows), k), dtype=torch.int32, device=case.q.device)
