"""Seeded cases of the append and attention tests, and their tolerances.

A rounding to a type is off by at most half a step, eps / 2 of the value.  An
attention output is rounded once (eps / 2 of it) and every softmax weight once
before it meets the values (eps / 2 of the weighted mean of |v|).  FP32 leaves:
a score is a sum of dim products, off by at most 2^-24 (dim + 4) of
scale * sum |q||k|, which moves every weight and the sum of the weights by that
much of themselves; an exponential is good to 2^-20 of itself.  FP16 weights
below 2^-14 keep an absolute half step of 2^-25, at most 2^-25 of the largest
weight and |v| for each key; outputs below 2^-14 likewise 2^-25.
"""

import numpy as np
import torch

from oracle import attention as A

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def empty_cache(pages, heads, dim, dtype, layout, device="cuda", fill=float("nan")):
    """Pools [pages, 64, heads, dim] in one of four memory orders, full of `fill`."""
    if layout == "odd":    # padded tokens and pages: strides whose common divisor is less than a row
        tok, extra = heads * dim + 8, 24
        both = [torch.full((pages * (64 * tok + extra),), fill, dtype=DT[dtype], device=device) for _ in range(2)]
        return [b.as_strided((pages, 64, heads, dim), (64 * tok + extra, tok, dim, 1)) for b in both]
    n = dict(nhd=(pages, 64, heads, dim), hnd=(pages, heads, 64, dim), pair=(pages, 2, 64, heads, dim))[layout]
    if layout == "pair":   # both pools in one tensor, page by page, as merged caches are
        both = torch.full(n, fill, dtype=DT[dtype], device=device)
        return both[:, 0], both[:, 1]
    k, v = (torch.full(n, fill, dtype=DT[dtype], device=device) for _ in range(2))
    return (k, v) if layout == "nhd" else (k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3))


class Case:
    """Requests with `lens` keys and `qlens` rows behind `prefix` shared keys; the caches hold NaN
    wherever no row may look, and the block table -7 where a request has no page."""

    def __init__(self, lens, qlens, prefix=0, hq=8, hkv=2, dim=64, dtype="bf16", layout="nhd", pad_rows=0, seed=0,
                 device="cuda", ends=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // 64) for n in lens]
        np_pages = -(-prefix // 64)
        pages = sum(need) + np_pages + 1
        perm = torch.randperm(pages, generator=g)
        self.k, self.v = empty_cache(pages, hkv, dim, dtype, layout, device)
        table = torch.full((len(lens), max(need + [0]) + 1), -7, dtype=torch.int32)
        at = 0
        for j, n in enumerate(lens):
            p = perm[at:at + need[j]]
            table[j, :need[j]] = p.to(torch.int32)
            at += need[j]
            self._fill(p, n, g)
        shared = perm[at:at + np_pages]
        self._fill(shared, prefix, g)
        self.prefix_pages, self.prefix_len = shared.to(torch.int32).to(device), prefix
        starts, bounds = [0], []
        for n, m in zip(lens, qlens):
            bounds += [max(0, n - m + i + 1) for i in range(m)]
            starts.append(starts[-1] + m)
        bounds += [5] * pad_rows                 # rows outside every request: no keys, whatever their bound
        if ends is not None:
            bounds = ends
        rows = len(bounds)
        heat = torch.linspace(0.3, 4.0, hq)[:, None]
        self.q = (torch.randn((rows, hq, dim), generator=g) * heat).to(DT[dtype]).to(device)
        self.block_table, self.starts = table.to(device), torch.tensor(starts, dtype=torch.int32, device=device)
        self.row_ends = torch.tensor(bounds, dtype=torch.int32, device=device)
        self.qlen, self.dtype, self.scale = max(qlens + [0]), dtype, dim ** -0.5

    def _fill(self, pages, n, g):
        for i in range(0, n, 64):
            m = min(64, n - i)
            for c in (self.k, self.v):
                x = torch.randn((m,) + tuple(c.shape[2:]), generator=g)
                c[int(pages[i // 64]), :m] = x.to(c.dtype).to(c.device)

    def paged(self, dsa, **kw):
        return dsa.attend_paged(self.q, self.k, self.v, self.block_table, self.starts, self.row_ends, self.qlen,
                                prefix_pages=self.prefix_pages, prefix_len=self.prefix_len, want_lse=True, **kw)

    def selected(self, dsa, topk, **kw):
        return dsa.attend_selected(self.q, self.k, self.v, self.block_table, self.starts, self.row_ends, topk,
                                   want_lse=True, **kw)

    def check(self, got, topk=None, rows=None):
        """Every output and log-sum-exp of `got` against the 64-bit formula."""
        out, lse = (t.double().cpu().numpy() for t in got)
        k, v, q = (t.double().cpu().numpy() for t in (self.k, self.v, self.q))
        starts, ends, table = self.starts.tolist(), self.row_ends.tolist(), self.block_table.tolist()
        pp = self.prefix_pages.tolist()
        lists = None if topk is None else topk.tolist()
        eps = torch.finfo(DT[self.dtype]).eps
        for r in range(q.shape[0]) if rows is None else rows:
            prefix = 0 if lists is not None else self.prefix_len
            keys = A.visible(r, starts, ends, table, pp, prefix, lists)
            o, l, mean_abs, size = A.attend(q[r], k, v, keys, self.scale)
            if not keys:
                assert not out[r].any() and np.isneginf(lse[r]).all(), r
                continue
            vmax = np.abs(v[tuple(np.array(keys).T)]).max()
            moved = 2.0 ** -24 * (q.shape[2] + 4) * size
            tol = eps / 2 * np.abs(o) + (eps / 2 + 2.0 ** -20 + 4 * moved[:, None]) * mean_abs
            if self.dtype == "fp16":
                tol += len(keys) * 2.0 ** -25 * vmax + 2.0 ** -25
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
