"""Workloads of the attention beside the indexer: the paged key/value append with its rotation, paged
attention with a prefix that the batch shares, and attention over the indexer's selected keys.

``run`` computes a case in plain torch operations, or through the library's calls where ``own`` is set.
"""

import math

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One new token of one request: the smallest append, where the call's latency is all.
        dict(name="append one token", op="append", tokens=1, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", layout="nhd", max_pos=131072),
        # The rows of a speculative-verify step (128 requests, up to 4 rows and 4 padding rows), partial rotation.
        dict(name="append verify rows", op="append", tokens=333, hq=64, hkv=8, d=128, rot=64, interleaved=True,
             dtype="fp16", layout="hnd", max_pos=65536),
        # A prompt's chunk of tokens going into the cache.
        dict(name="append prompt chunk", op="append", tokens=16384, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", layout="nhd", max_pos=131072),
        # One request, one row, a short context: latency.
        dict(name="paged one request", op="paged", requests=1, qlen=1, prefix=0, lo=1000, hi=1000, hq=32, hkv=8, d=128,
             dtype="bf16", layout="nhd"),
        # A decode batch without anything shared: the cache is read once.
        dict(name="paged decode", op="paged", requests=64, qlen=1, prefix=0, lo=4096, hi=8192, hq=32, hkv=8, d=128,
             dtype="bf16", layout="nhd"),
        # A few long contexts under one key head (all query heads share it).
        dict(name="paged long one head", op="paged", requests=8, qlen=1, prefix=0, lo=131071, hi=131071, hq=16, hkv=1,
             d=128, dtype="fp16", layout="hnd"),
        # A small batch behind one system prompt, odd lengths, some requests with nothing of their own yet.
        dict(name="shared small batch", op="paged", requests=17, qlen=1, prefix=4001, lo=0, hi=517, hq=32, hkv=4, d=64,
             dtype="fp16", layout="nhd"),
        # A verify step of a large batch behind one long document.
        dict(name="shared verify batch", op="paged", requests=128, qlen=4, prefix=32768, lo=64, hi=4096, hq=64, hkv=8,
             d=128, dtype="bf16", layout="hnd"),
        # One row's selected keys: latency.
        dict(name="selected one row", op="selected", requests=1, qlen=1, k=2048, lo=8192, hi=8192, hq=32, hkv=8, d=128,
             dtype="bf16", layout="nhd"),
        # The indexer's decode batch: 2048 keys a row out of 4096 to 8192.
        dict(name="selected decode", op="selected", requests=64, qlen=1, k=2048, lo=4096, hi=8192, hq=32, hkv=8, d=128,
             dtype="bf16", layout="nhd"),
        # Verify rows, some with fewer keys than k; rows of a request share half of their keys.
        dict(name="selected verify rows", op="selected", requests=40, qlen=4, k=1000, lo=500, hi=32768, hq=48, hkv=4,
             d=64, dtype="fp16", layout="hnd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "selected"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, hq=hkv * rng.choice([1, 2, 3, 4, 6, 8, 16]), hkv=hkv, d=rng.choice([64, 80, 96, 128]),
             dtype=rng.choice(["bf16", "fp16"]), layout=rng.choice(["nhd", "hnd"]))
    if op == "append":
        c |= dict(tokens=_log(rng, 1, 8192), rot=rng.choice([c["d"], 32, 64]), interleaved=rng.choice([False, True]),
                  max_pos=_log(rng, 4096, 131072))
        return c
    c |= dict(requests=_log(rng, 1, 128), qlen=rng.choice([1, 1, 2, 3, 4]))
    # at most 256 K keys of one request each in all, so that no case costs more than the largest listed one
    most = min(65536, max(512, 262144 // c["requests"]))
    hi = _log(rng, 64, most)
    if op == "paged":
        c |= dict(prefix=rng.choice([0, _log(rng, 1, 16384)]), lo=rng.randint(0, hi // 2), hi=hi)
    else:
        c |= dict(k=_log(rng, 16, 2048), lo=rng.randint(1, hi), hi=hi)
    return c


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], both ends among them where there is room."""
    return [hi] if n == 1 else [lo + (hi - lo) * j // (n - 1) for j in range(n)]


def _sizes(c):
    """Key counts and row counts of the requests, before they are shuffled together (the sums are the case's)."""
    lens = _spread(c["requests"], c["lo"], c["hi"])
    rows = [1 + j % c["qlen"] for j in range(c["requests"])]
    return [max(n, q) if c["lo"] > 0 else n for n, q in zip(lens, rows)], rows


def _cache(c, pages, g):
    """A page pool [pages, 64, heads, d], in memory token by token or head by head."""
    shape = (pages, PAGE, c["hkv"], c["d"]) if c["layout"] == "nhd" else (pages, c["hkv"], PAGE, c["d"])
    t = torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[c["dtype"]])
    return t if c["layout"] == "nhd" else t.permute(0, 2, 1, 3)


def _pages(lens, g, extra=0):
    """Block table over a shuffled pool (unused entries -1), the pages of `extra` shared keys, and the pool's size."""
    need = [-(-n // PAGE) for n in lens]
    shared = -(-extra // PAGE)
    total = sum(need) + shared
    perm = torch.randperm(max(total, 1), generator=g, device="cuda").to(torch.int32)
    counts = torch.tensor(need, device="cuda")
    first = torch.cumsum(counts, 0) - counts
    col = torch.arange(max(max(need), 1), device="cuda")
    at = (first[:, None] + col).clamp(max=max(total - 1, 0))
    table = torch.where(col < counts[:, None], perm[at].to(torch.int64), -1).to(torch.int32)
    return table.contiguous(), perm[total - shared: total].contiguous() if shared else perm[:0], max(total, 1)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] == "append":
        n, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
        pages = -(-n // PAGE) + 2
        packed = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device="cuda", dtype=dt)   # one projection's output
        q, k, v = packed.split([hq * d, hkv * d, hkv * d], dim=1)
        st |= dict(q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hkv, d)), v=v.unflatten(1, (hkv, d)))
        start = int(torch.randint(0, max(1, c["max_pos"] - n), (1,), generator=g, device="cuda"))
        st["positions"] = torch.arange(n, device="cuda") % (c["max_pos"] - start) + start
        slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:n]
        if n > 4:
            slots[-4:] = -1                                            # padding rows of the step
        st["slots"] = slots.contiguous()
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        ang = torch.arange(c["max_pos"], device="cuda", dtype=torch.float64)[:, None] * freq
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32)
        st |= dict(k_cache=_cache(c, pages, g), v_cache=_cache(c, pages, g))
        return st
    lens, rows = _sizes(c)
    order = torch.randperm(c["requests"], generator=g, device="cuda").tolist()
    lens, rows = [lens[j] for j in order], [rows[j] for j in order]
    extra = c.get("prefix", 0)
    table, prefix_pages, total = _pages(lens, g, extra)
    n = sum(rows)
    ends, starts = [], [0]
    for m, r in zip(lens, rows):
        ends += [max(0, m - r + i + 1) for i in range(r)]
        starts.append(starts[-1] + r)
    # heads from diffuse to sharp, as the heads of a layer are
    heat = torch.linspace(0.5, 4.0, c["hq"], device="cuda")[:, None]
    st["q"] = (torch.randn((n, c["hq"], c["d"]), generator=g, device="cuda") * heat).to(dt)
    st |= dict(k_cache=_cache(c, total, g), v_cache=_cache(c, total, g), block_table=table, prefix_pages=prefix_pages,
               starts=torch.tensor(starts, device="cuda", dtype=torch.int32),
               row_ends=torch.tensor(ends, device="cuda", dtype=torch.int32), qlen=max(rows))
    if c["op"] == "selected":
        st["topk"] = _choose(starts, st["row_ends"], c, g)
    return st


def _choose(starts, row_ends, c, g):
    """k distinct positions of each row below its bound, in any order and then -1.  The rows of a request take every
    second key from its common ranking and the others from their own, as successive rows of one text do."""
    n, k = row_ends.numel(), c["k"]
    width = max(int(row_ends.max()), k)
    req = (torch.arange(n, device="cuda")[:, None] >= torch.tensor(starts[1:], device="cuda")).sum(1)
    common = torch.rand((len(starts) - 1, width), generator=g, device="cuda")[req]
    alone = torch.rand((n, width), generator=g, device="cuda")
    even = torch.arange(width, device="cuda") % 2 == 0
    score = torch.where(even, common, alone)
    score = torch.where(torch.arange(width, device="cuda") < row_ends[:, None], score, -1.0)
    top, at = score.topk(k, dim=1)
    return torch.where(top >= 0, at, -1).to(torch.int32)


def _rotate(x, cos, sin, interleaved):
    """x [n, heads, d] in FP32 with its first columns turned by the angles [n, rot / 2]."""
    half = cos.shape[1]
    c, s = cos[:, None, :], sin[:, None, :]
    r = x[..., : 2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, w = a * c - b * s, b * c + a * s
    turned = torch.stack([u, w], dim=-1).flatten(-2) if interleaved else torch.cat([u, w], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _append_plain(st):
    c = st["case"]
    dt, half = st["q"].dtype, c["rot"] // 2
    table = st["cos_sin"][st["positions"]]
    cos, sin = table[:, :half], table[:, half:]
    q = _rotate(st["q"].float(), cos, sin, c["interleaved"]).to(dt)
    k = _rotate(st["k"].float(), cos, sin, c["interleaved"]).to(dt)
    real = st["slots"] >= 0
    slots = st["slots"][real]
    st["k_cache"][slots // PAGE, slots % PAGE] = k[real]
    st["v_cache"][slots // PAGE, slots % PAGE] = st["v"][real]
    return q, st["k_cache"], st["v_cache"]


def _requests(st):
    """The request of every row and its place there."""
    at = torch.arange(st["row_ends"].numel(), device="cuda")
    req = (at[:, None] >= st["starts"][1:]).sum(1)
    return req, at - st["starts"][req]


def _join(parts, dt):
    """The softmax over several key ranges: parts of (scores with -inf where masked, values)."""
    top = torch.stack([s.amax(-1) for s, _ in parts if s.shape[-1]]).amax(0)
    base = torch.where(top == float("-inf"), 0.0, top)[..., None]
    weights = [(s - base).exp() for s, _ in parts]
    total = sum(w.sum(-1) for w in weights)
    out = sum(torch.matmul(w, v) for w, (_, v) in zip(weights, parts))
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    return out.to(dt), torch.where(total > 0, base[..., 0] + total.log(), float("-inf"))


def _paged_plain(st):
    c = st["case"]
    hq, hkv, d, dt = c["hq"], c["hkv"], c["d"], st["q"].dtype
    group, scale = hq // hkv, d ** -0.5
    req, place = _requests(st)
    n, reqs, most = st["q"].shape[0], c["requests"], st["qlen"]
    pages = st["block_table"].clamp(min=0).long()
    keys = st["k_cache"][pages].flatten(1, 2).float().transpose(1, 2)                  # [requests, hkv, keys, d]
    values = st["v_cache"][pages].flatten(1, 2).float().transpose(1, 2)
    width = keys.shape[2]
    q = torch.zeros((reqs, most, hq, d), device="cuda")
    q[req, place] = st["q"].float()
    ends = torch.zeros((reqs, most), device="cuda", dtype=torch.int64)
    ends[req, place] = st["row_ends"].long()
    q = q.unflatten(2, (hkv, group)).transpose(1, 2).flatten(2, 3)                     # [requests, hkv, most * group, d]
    s = torch.matmul(q, keys.transpose(2, 3)) * scale
    seen = torch.arange(width, device="cuda") < ends.repeat_interleave(group, 1)[:, None, :, None]
    parts = [(torch.where(seen, s, float("-inf")), values)]
    if c["prefix"]:
        shared = st["prefix_pages"].long()
        pk = st["k_cache"][shared].flatten(0, 1)[: c["prefix"]].float().transpose(0, 1)   # [hkv, prefix, d]
        pv = st["v_cache"][shared].flatten(0, 1)[: c["prefix"]].float().transpose(0, 1)
        sp = torch.matmul(q, pk.transpose(1, 2)) * scale
        parts.append((sp, pv.expand(reqs, -1, -1, -1)))
    out, lse = _join(parts, dt)
    out = out.unflatten(2, (most, group)).transpose(1, 2).flatten(2, 3)[req, place]
    return out, lse.unflatten(2, (most, group)).transpose(1, 2).flatten(2, 3)[req, place]


def _selected_plain(st):
    c = st["case"]
    hq, hkv, d, dt = c["hq"], c["hkv"], c["d"], st["q"].dtype
    group, scale = hq // hkv, d ** -0.5
    req, _ = _requests(st)
    real = st["topk"] >= 0
    at = st["topk"].clamp(min=0).long()
    page = torch.gather(st["block_table"].long()[req], 1, at // PAGE)
    keys = st["k_cache"][page, at % PAGE].float().transpose(1, 2)                      # [rows, hkv, k, d]
    values = st["v_cache"][page, at % PAGE].float().transpose(1, 2)
    q = st["q"].float().unflatten(1, (hkv, group))
    s = torch.matmul(q, keys.transpose(2, 3)) * scale
    out, lse = _join([(torch.where(real[:, None, None], s, float("-inf")), values)], dt)
    return out.flatten(1, 2), lse.flatten(1, 2)


def run(st):
    c = st["case"]
    if own:
        from sparse_attention_indexer_score_gb300 import dsa

        if c["op"] == "append":
            q = dsa.kv_append(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], st["positions"],
                              st["cos_sin"], q=st["q"], interleaved=c["interleaved"])
            return q, st["k_cache"], st["v_cache"]
        if "workspace" not in st:                        # a serving loop's, kept from step to step
            st["workspace"] = dsa.new_workspace(
                dsa.attend_workspace_size(st["q"].shape[0], c["requests"], c["hq"], c["hkv"], c["d"], st["qlen"],
                                          c.get("k", 0)), "cuda")
        if c["op"] == "paged":
            return dsa.attend_paged(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["starts"],
                                    st["row_ends"], st["qlen"], prefix_pages=st["prefix_pages"],
                                    prefix_len=c["prefix"], want_lse=True, workspace=st["workspace"])
        return dsa.attend_selected(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["starts"],
                                   st["row_ends"], st["topk"], want_lse=True, workspace=st["workspace"])
    if c["op"] == "append":
        return _append_plain(st)
    return _paged_plain(st) if c["op"] == "paged" else _selected_plain(st)


def work(case):
    c = case
    kv = 2 * c["hkv"] * c["d"] * 2                       # one token's key and value bytes
    row = 2 * c["hq"] * c["d"]                           # one query row in 16 bits
    if c["op"] == "append":
        n = c["tokens"]
        # a position past the table's end starts over, so a long step shares some angles
        return {"bytes": n * (2 * row + 2 * kv + 16) + min(n, c["max_pos"]) * c["rot"] * 4,
                "flops": n * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    lens, rows = _sizes(c)
    n = sum(rows)
    if c["op"] == "paged":
        seen = sum(sum(max(0, m - r + i + 1) for i in range(r)) for m, r in zip(lens, rows))
        seen += n * c["prefix"]
        keys = sum(lens) + c["prefix"]
        lists = sum(-(-m // PAGE) for m in lens) * 4 + n * 4
    else:
        k = c["k"]
        took = [[min(k, max(0, m - r + i + 1)) for i in range(r)] for m, r in zip(lens, rows)]
        seen = sum(map(sum, took))
        # the largest row's keys, and half of every other row's (never more than the request has)
        keys = sum(min(m, t[-1] + sum(t[:-1]) // 2) for m, t in zip(lens, took))
        lists = n * k * 4
    return {"bytes": keys * kv + n * (2 * row + c["hq"] * 4) + lists, "flops": 4 * seen * c["hq"] * c["d"]}


def _exact_rows(q, keys, values, seen, scale):
    """q [hkv, m, d], keys and values [hkv, t, d], seen [m, t], all in 64 bits."""
    s = torch.einsum("hmd,htd->hmt", q, keys) * scale
    s = s.masked_fill(~seen, float("-inf"))
    lse = torch.logsumexp(s, dim=-1) if s.shape[-1] else s.new_full(s.shape[:2], float("-inf"))
    w = torch.exp(s - lse.masked_fill(lse == float("-inf"), 0.0)[..., None])
    return torch.einsum("hmt,htd->hmd", w, values), lse


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    q = st["q"].double()
    if c["op"] == "append":
        half = c["rot"] // 2
        w = st["cos_sin"].double()[st["positions"]]
        turn = torch.complex(w[:, :half], w[:, half:])[:, None, :]

        def turned(x):
            x = x.double().clone()
            if c["interleaved"]:
                z = torch.view_as_complex(x[..., : 2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
                x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2] = z.real, z.imag
            else:
                z = torch.complex(x[..., :half].contiguous(), x[..., half: 2 * half].contiguous()) * turn
                x[..., :half], x[..., half: 2 * half] = z.real, z.imag
            return x

        k_cache, v_cache = st["k_cache"].double().contiguous(), st["v_cache"].double().contiguous()
        keep = torch.nonzero(st["slots"] >= 0)[:, 0]
        k_cache.flatten(0, 1)[st["slots"][keep]] = turned(st["k"])[keep]
        v_cache.flatten(0, 1)[st["slots"][keep]] = st["v"].double()[keep]
        return turned(q), k_cache, v_cache
    hkv, group, d = c["hkv"], c["hq"] // c["hkv"], c["d"]
    scale = 1.0 / math.sqrt(d)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], float("-inf"), device="cuda", dtype=torch.float64)
    starts, ends = st["starts"].tolist(), st["row_ends"].tolist()
    flat = [st[x].reshape(-1, hkv, d) for x in ("k_cache", "v_cache")]

    def tokens(pages, positions):
        return pages.long()[positions // PAGE] * PAGE + positions % PAGE

    shared = tokens(st["prefix_pages"], torch.arange(c.get("prefix", 0), device="cuda"))
    for j, table in enumerate(st["block_table"]):
        rows = range(starts[j], starts[j + 1])
        if c["op"] == "paged":
            most = max(ends[r] for r in rows)
            at = torch.cat([shared, tokens(table, torch.arange(most, device="cuda"))])
            place = torch.arange(at.numel(), device="cuda") - shared.numel()
            blocks = [(list(rows), at, torch.stack([place < ends[r] for r in rows]))]
        else:
            blocks = []
            for r in rows:
                p = st["topk"][r].long()
                at = tokens(table, p[p >= 0])
                blocks.append(([r], at, torch.ones((1, at.numel()), dtype=torch.bool, device="cuda")))
        for which, at, seen in blocks:
            x = q[which].unflatten(1, (hkv, group)).transpose(0, 1).flatten(1, 2)       # [hkv, rows * group, d]
            k, v = (f[at].double().transpose(0, 1) for f in flat)
            o, l = _exact_rows(x, k, v, seen.repeat_interleave(group, 0), scale)
            out[which] = o.unflatten(1, (len(which), group)).transpose(0, 1).flatten(1, 2)
            lse[which] = l.unflatten(1, (len(which), group)).transpose(0, 1).flatten(1, 2)
    return out, lse
