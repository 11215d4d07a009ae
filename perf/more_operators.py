"""Workloads of the 4-bit key/value cache: the append that rotates and quantises, the reading back, and the
attention over all keys of a request or over the indexer's selected keys.

A cache section (one page of 64 tokens, one head) holds 64 rows of d / 2 bytes of key codes, 64 rows of value codes,
then 64 rows of scales: the key's d / 16, padded to a multiple of 4, and the value's likewise.  Codes are E2M1, column
2j in the low half of byte j; every 16 columns have an E4M3 scale s, and a code c stands for c * s * g, g being the
cache's FP32 scale of keys or of values.

``run`` computes a case in plain torch operations, or through the library's calls where ``own`` is set.
"""

import math

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # One new token of one request, written and read back: the smallest append, where the calls' latency is all.
        dict(name="append one token", op="append", tokens=1, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", max_pos=131072, g=1.0),
        # The rows of a speculative-verify step (128 requests, up to 4 rows and 4 padding rows), partial rotation.
        dict(name="append verify rows", op="append", tokens=333, hq=64, hkv=8, d=128, rot=64, interleaved=True,
             dtype="fp16", max_pos=65536, g=0.25),
        # A prompt's chunk of tokens going into the cache.
        dict(name="append prompt chunk", op="append", tokens=16384, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", max_pos=131072, g=1.0),
        # One request's context taken back out of the cache, an odd length and an odd head.
        dict(name="read one request", op="read", tokens=1001, hkv=8, d=80, dtype="fp16", g=0.5),
        # Many requests' keys and values read back for a prompt's later chunk.
        dict(name="read long contexts", op="read", tokens=65536, hkv=8, d=128, dtype="bf16", g=1.0),
        # One request, one row, a short context: latency.
        dict(name="paged one request", op="paged", requests=1, qlen=1, lo=1000, hi=1000, hq=32, hkv=8, d=128,
             dtype="bf16", layers=1, g=1.0),
        # A decode batch: the cache is read once.
        dict(name="paged decode", op="paged", requests=64, qlen=1, lo=4096, hi=8192, hq=32, hkv=8, d=128,
             dtype="bf16", layers=1, g=1.0),
        # A few long contexts under one key head (all query heads share it), two layers' pages in one pool.
        dict(name="paged long one head", op="paged", requests=8, qlen=1, lo=131071, hi=131071, hq=16, hkv=1, d=128,
             dtype="fp16", layers=2, g=0.5),
        # The verify rows of a large batch, some requests with hardly a page.
        dict(name="paged verify batch", op="paged", requests=128, qlen=4, lo=64, hi=8192, hq=64, hkv=8, d=128,
             dtype="bf16", layers=1, g=1.0),
        # One row's selected keys: latency.
        dict(name="selected one row", op="selected", requests=1, qlen=1, k=2048, lo=8192, hi=8192, hq=32, hkv=8, d=128,
             dtype="bf16", layers=1, g=1.0),
        # The indexer's decode batch: 2048 keys a row out of 4096 to 8192.
        dict(name="selected decode", op="selected", requests=64, qlen=1, k=2048, lo=4096, hi=8192, hq=32, hkv=8, d=128,
             dtype="bf16", layers=1, g=1.0),
        # Verify rows, some with fewer keys than k; rows of a request share half of their keys.
        dict(name="selected verify rows", op="selected", requests=40, qlen=4, k=1000, lo=500, hi=32768, hq=48, hkv=4,
             d=64, dtype="fp16", layers=2, g=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "paged", "paged", "selected", "selected"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, hkv=hkv, d=rng.choice([64, 80, 96, 128]), dtype=rng.choice(["bf16", "fp16"]),
             g=rng.choice([1.0, 0.25, 0.37]))
    if op == "read":
        return c | dict(tokens=_log(rng, 1, 65536))
    c |= dict(hq=hkv * rng.choice([1, 2, 3, 4, 6, 8, 16]))
    if op == "append":
        return c | dict(tokens=_log(rng, 1, 8192), rot=rng.choice([c["d"], 32, 64]),
                        interleaved=rng.choice([False, True]), max_pos=_log(rng, 4096, 131072))
    c |= dict(requests=_log(rng, 1, 128), qlen=rng.choice([1, 1, 2, 3, 4]), layers=rng.choice([1, 1, 2]))
    # at most 384 K keys of one request each in all, so that no case costs more than the largest listed one
    most = min(131072, max(512, 393216 // c["requests"]))
    hi = _log(rng, 64, most)
    if op == "paged":
        return c | dict(lo=rng.randint(0, hi // 2), hi=hi)
    return c | dict(k=_log(rng, 16, 2048), lo=rng.randint(1, hi), hi=hi)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], both ends among them where there is room."""
    return [hi] if n == 1 else [lo + (hi - lo) * j // (n - 1) for j in range(n)]


def _sizes(c):
    """Key counts and row counts of the requests, before they are shuffled together (the sums are the case's)."""
    lens = _spread(c["requests"], c["lo"], c["hi"])
    rows = [1 + j % c["qlen"] for j in range(c["requests"])]
    return [max(n, q) if c["lo"] > 0 else n for n, q in zip(lens, rows)], rows


def _scale_row(d):
    return 4 * -(-d // 64)


def _section(d):
    return PAGE * (d + 2 * _scale_row(d))


def _cache(c, pages, g):
    """A pool of pages whose codes are spread over the grid and whose scales give columns a size of about g."""
    layers = c.get("layers", 1)
    t = torch.randint(0, 256, (pages, layers, c["hkv"], _section(c["d"])), generator=g, device="cuda",
                      dtype=torch.uint8)[:, layers - 1]
    s = t[..., PAGE * c["d"]:]
    # 0x28 to 0x2f: 0.25 to 0.47, which makes the codes' root mean square (2.9) one
    s.copy_(torch.randint(0x28, 0x30, s.shape, generator=g, device="cuda", dtype=torch.uint8))
    return t


def _pages(lens, g):
    """Block table over a shuffled pool (unused entries -1), and the pool's size."""
    need = [-(-n // PAGE) for n in lens]
    total = sum(need)
    perm = torch.randperm(max(total, 1), generator=g, device="cuda").to(torch.int32)
    counts = torch.tensor(need, device="cuda")
    first = torch.cumsum(counts, 0) - counts
    col = torch.arange(max(max(need), 1), device="cuda")
    at = (first[:, None] + col).clamp(max=max(total - 1, 0))
    table = torch.where(col < counts[:, None], perm[at].to(torch.int64), -1).to(torch.int32)
    return table.contiguous(), max(total, 1)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] in ("append", "read"):
        n, hkv, d = c["tokens"], c["hkv"], c["d"]
        pages = -(-n // PAGE) + 2
        slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:n]
        if n > 4:
            slots[-4:] = -1                                            # padding rows of the step
        st |= dict(slots=slots.contiguous(), cache=_cache(c, pages, g))
    if c["op"] == "read":
        return st
    if c["op"] == "append":
        hq = c["hq"]
        packed = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device="cuda")   # one projection's output
        # a few columns of a layer's keys are far larger than the others
        packed[:, hq * d: (hq + hkv) * d] *= torch.where(
            torch.rand(hkv * d, generator=g, device="cuda") < 0.03, 8.0, 1.0)
        q, k, v = (packed * (2 * c["g"])).to(dt).split([hq * d, hkv * d, hkv * d], dim=1)
        st |= dict(q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hkv, d)), v=v.unflatten(1, (hkv, d)))
        start = int(torch.randint(0, max(1, c["max_pos"] - n), (1,), generator=g, device="cuda"))
        st["positions"] = torch.arange(n, device="cuda") % (c["max_pos"] - start) + start
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        ang = torch.arange(c["max_pos"], device="cuda", dtype=torch.float64)[:, None] * freq
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32)
        return st
    lens, rows = _sizes(c)
    order = torch.randperm(c["requests"], generator=g, device="cuda").tolist()
    lens, rows = [lens[j] for j in order], [rows[j] for j in order]
    table, total = _pages(lens, g)
    n = sum(rows)
    ends, starts = [], [0]
    for m, r in zip(lens, rows):
        ends += [max(0, m - r + i + 1) for i in range(r)]
        starts.append(starts[-1] + r)
    # heads from diffuse to sharp, as the heads of a layer are
    heat = torch.linspace(0.5, 4.0, c["hq"], device="cuda")[:, None] / c["g"]
    st["q"] = (torch.randn((n, c["hq"], c["d"]), generator=g, device="cuda") * heat).to(dt)
    st |= dict(cache=_cache(c, total, g), block_table=table,
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


def _split(sections, d):
    """Key codes, value codes [..., 64, d / 2], key scales and value scales [..., 64, d / 16] of sections."""
    w, sr = d // 2, _scale_row(d)
    k, v, s = sections.split([PAGE * w, PAGE * w, PAGE * 2 * sr], dim=-1)
    s = s.unflatten(-1, (PAGE, 2 * sr))
    return k.unflatten(-1, (PAGE, w)), v.unflatten(-1, (PAGE, w)), s[..., : d // 16], s[..., sr: sr + d // 16]


def _values(codes, scales, g):
    """What codes and scales stand for, in FP32: (code * scale) * g."""
    grid = torch.tensor(GRID + [-x for x in GRID], device=codes.device)
    byte = torch.arange(256, device=codes.device)
    x = torch.stack([grid[byte & 15], grid[byte >> 4]], dim=1)[codes.int()].flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * s[..., None] * g).flatten(-2)


def _quantise(x, g):
    """Codes and scales of FP32 rows: s = E4M3(amax / (6 g)) a block of 16, code = E2M1(x / (s g))."""
    b = x.unflatten(-1, (-1, 16))
    g = torch.tensor(g, device=x.device, dtype=torch.float32)
    s = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = torch.where(s.float()[..., None] > 0, b / (s.float() * g)[..., None], 0.0 * b).flatten(-2)
    a = y.abs()
    code = sum((a > t if even else a >= t).to(torch.uint8)            # ties to the even code
               for t, even in ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False),
                               (5.0, True)))
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _rotate(x, cos, sin, interleaved):
    """x [n, heads, d] in FP32 with its first columns turned by the angles [n, rot / 2]."""
    half = cos.shape[1]
    c, s = cos[:, None, :], sin[:, None, :]
    r = x[..., : 2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, w = a * c - b * s, b * c + a * s
    turned = torch.stack([u, w], dim=-1).flatten(-2) if interleaved else torch.cat([u, w], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _read_plain(st):
    c = st["case"]
    real = st["slots"] >= 0
    slots = st["slots"].clamp(min=0)
    parts = [t.transpose(1, 2)[slots // PAGE, slots % PAGE] for t in _split(st["cache"], c["d"])]
    out = [_values(parts[i], parts[i + 2], c["g"]).to(DTYPES[c["dtype"]]) for i in (0, 1)]
    return tuple(torch.where(real[:, None, None], x, torch.zeros_like(x)) for x in out)


def _append_plain(st):
    c = st["case"]
    half = c["rot"] // 2
    table = st["cos_sin"][st["positions"]]
    cos, sin = table[:, :half], table[:, half:]
    q = _rotate(st["q"].float(), cos, sin, c["interleaved"]).to(st["q"].dtype)
    kc, ks = _quantise(_rotate(st["k"].float(), cos, sin, c["interleaved"]), c["g"])
    vc, vs = _quantise(st["v"].float(), c["g"])
    real = st["slots"] >= 0
    slots = st["slots"][real]
    for to, new in zip(_split(st["cache"], c["d"]), (kc, vc, ks, vs)):
        to.transpose(1, 2)[slots // PAGE, slots % PAGE] = new[real]
    return (q,) + _read_plain(st)


def _requests(st):
    """The request of every row and its place there."""
    at = torch.arange(st["row_ends"].numel(), device="cuda")
    req = (at[:, None] >= st["starts"][1:]).sum(1)
    return req, at - st["starts"][req]


def _softmax(s, values, dt):
    """Scores (-inf where masked) over values; zeros and -inf for a row that sees nothing."""
    top = s.amax(-1) if s.shape[-1] else torch.full(s.shape[:-1], float("-inf"), device=s.device)
    base = torch.where(top == float("-inf"), 0.0, top)[..., None]
    w = (s - base).exp()
    total = w.sum(-1)
    out = torch.matmul(w, values)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    return out.to(dt), torch.where(total > 0, base[..., 0] + total.log(), float("-inf"))


def _paged_plain(st):
    c = st["case"]
    hq, hkv, d, dt = c["hq"], c["hkv"], c["d"], st["q"].dtype
    group, scale = hq // hkv, d ** -0.5
    req, place = _requests(st)
    reqs, most = c["requests"], st["qlen"]
    kc, vc, ks, vs = _split(st["cache"][st["block_table"].clamp(min=0).long()], d)     # [requests, pages, hkv, 64, .]
    keys = _values(kc, ks, c["g"]).transpose(1, 2).flatten(2, 3)                       # [requests, hkv, keys, d]
    values = _values(vc, vs, c["g"]).transpose(1, 2).flatten(2, 3)
    width = keys.shape[2]
    q = torch.zeros((reqs, most, hq, d), device="cuda")
    q[req, place] = st["q"].float()
    ends = torch.zeros((reqs, most), device="cuda", dtype=torch.int64)
    ends[req, place] = st["row_ends"].long()
    q = q.unflatten(2, (hkv, group)).transpose(1, 2).flatten(2, 3)                     # [requests, hkv, most * group, d]
    s = torch.matmul(q, keys.transpose(2, 3)) * scale
    seen = torch.arange(width, device="cuda") < ends.repeat_interleave(group, 1)[:, None, :, None]
    out, lse = _softmax(torch.where(seen, s, float("-inf")), values, dt)
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
    kc, vc, ks, vs = (t.transpose(1, 2)[page, at % PAGE].transpose(1, 2) for t in _split(st["cache"], d))
    keys, values = _values(kc, ks, c["g"]), _values(vc, vs, c["g"])                    # [rows, hkv, k, d]
    q = st["q"].float().unflatten(1, (hkv, group))
    s = torch.matmul(q, keys.transpose(2, 3)) * scale
    out, lse = _softmax(torch.where(real[:, None, None], s, float("-inf")), values, dt)
    return out.flatten(1, 2), lse.flatten(1, 2)


def run(st):
    c = st["case"]
    if own:
        from sparse_attention_indexer_score_gb300 import dsa

        scales = dict(k_scale=c["g"], v_scale=c["g"])
        if c["op"] == "append":
            q = dsa.kv_append_fp4(st["k"], st["v"], st["slots"], st["cache"], st["positions"], st["cos_sin"],
                                  q=st["q"], interleaved=c["interleaved"], **scales)
            return (q,) + tuple(dsa.kv_read_fp4(st["slots"], st["cache"], c["d"], DTYPES[c["dtype"]], **scales))
        if c["op"] == "read":
            return tuple(dsa.kv_read_fp4(st["slots"], st["cache"], c["d"], DTYPES[c["dtype"]], **scales))
        if "workspace" not in st:                        # a serving loop's, kept from step to step
            st["workspace"] = dsa.new_workspace(
                dsa.attend_workspace_size_fp4(st["q"].shape[0], c["requests"], c["hq"], c["hkv"], c["d"], st["qlen"],
                                              c.get("k", 0)), "cuda")
        if c["op"] == "paged":
            return dsa.attend_paged_fp4(st["q"], st["cache"], st["block_table"], st["starts"], st["row_ends"],
                                        st["qlen"], want_lse=True, workspace=st["workspace"], **scales)
        return dsa.attend_selected_fp4(st["q"], st["cache"], st["block_table"], st["starts"], st["row_ends"],
                                       st["topk"], want_lse=True, workspace=st["workspace"], **scales)
    if c["op"] == "append":
        return _append_plain(st)
    if c["op"] == "read":
        return _read_plain(st)
    return _paged_plain(st) if c["op"] == "paged" else _selected_plain(st)


def work(case):
    c = case
    kv = c["hkv"] * (c["d"] + c["d"] // 8)               # one token's codes and scales, keys and values
    wide = 2 * c["hkv"] * c["d"] * 2                     # ... in 16 bits
    if c["op"] == "read":
        n = c["tokens"]
        return {"bytes": n * (8 + kv + wide), "flops": n * 2 * c["hkv"] * c["d"] * 2}
    row = 2 * c["hq"] * c["d"]                           # one query row in 16 bits
    if c["op"] == "append":
        n = c["tokens"]
        # queries in and out, keys and values in, codes out; then the codes in and the values they stand for out
        return {"bytes": n * (2 * row + 2 * wide + 2 * kv + 16) + min(n, c["max_pos"]) * c["rot"] * 4,
                "flops": n * ((c["hq"] + c["hkv"]) * c["rot"] * 3 + 2 * c["hkv"] * c["d"] * 6)}
    lens, rows = _sizes(c)
    n = sum(rows)
    if c["op"] == "paged":
        seen = sum(sum(max(0, m - r + i + 1) for i in range(r)) for m, r in zip(lens, rows))
        keys = sum(lens)
        lists = sum(-(-m // PAGE) for m in lens) * 4 + n * 4
    else:
        k = c["k"]
        took = [[min(k, max(0, m - r + i + 1)) for i in range(r)] for m, r in zip(lens, rows)]
        seen = sum(map(sum, took))
        # the largest row's keys, and half of every other row's (never more than the request has)
        keys = sum(min(m, t[-1] + sum(t[:-1]) // 2) for m, t in zip(lens, took))
        lists = n * k * 4
    return {"bytes": keys * kv + n * (2 * row + c["hq"] * 4) + lists, "flops": 4 * seen * c["hq"] * c["d"]}


def _exact_values(codes, scales, g):
    """Codes [..., d / 2] and scales [..., d / 16] from the formats' bits, in 64 bits."""
    nibble = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()
    e, m = (nibble >> 1) & 3, (nibble & 1).double()
    x = torch.where(e > 0, torch.ldexp(1 + m / 2, e - 1), m / 2) * (1 - 2 * (nibble >> 3)).double()
    b = scales.int()
    e, m = (b >> 3) & 15, (b & 7).double()
    s = torch.where(e > 0, torch.ldexp(1 + m / 8, e - 7), torch.ldexp(m / 8, torch.full_like(e, -6)))
    s = s * (1 - 2 * (b >> 7)).double()
    return x * s.repeat_interleave(16, -1) * g


def _exact_rounded(x, bits, low, most):
    """x >= 0 in a format of `bits` bits behind the leading one, exponents from `low`, values up to `most`; ties to even."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** (low - 1)))).clamp(min=low)
    step = torch.exp2(e - bits)
    return (torch.round(x / step) * step).clamp(max=most)


def _exact_stored(x, g):
    """What rows in 64 bits become in the cache: the values their codes stand for."""
    b = x.unflatten(-1, (-1, 16))
    s = _exact_rounded(b.abs().amax(-1, keepdim=True) / (6 * g), 3, -6, 448.0)
    y = torch.where(s > 0, b / (s * g).clamp(min=1e-300), 0.0 * b)
    return (_exact_rounded(y.abs(), 1, 0, 6.0) * torch.sign(y) * s * g).flatten(-2)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    d, hkv, g = c["d"], c["hkv"], float(torch.tensor(c["g"], dtype=torch.float32))    # (the cache's scales are FP32)
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

        keep = (st["slots"] >= 0).double()[:, None, None]
        return turned(st["q"]), _exact_stored(turned(st["k"]), g) * keep, _exact_stored(st["v"].double(), g) * keep

    # tokens of the pool, one behind the other: [pages * 64, hkv, .]
    flat = [t.transpose(1, 2).flatten(0, 1) for t in _split(st["cache"], d)]

    def tokens(at):
        return tuple(_exact_values(flat[i][at], flat[i + 2][at], g) for i in (0, 1))

    if c["op"] == "read":
        keep = (st["slots"] >= 0).double()[:, None, None]
        return tuple(x * keep for x in tokens(st["slots"].clamp(min=0)))
    q = st["q"].double()
    group, scale = c["hq"] // hkv, 1.0 / math.sqrt(d)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], float("-inf"), device="cuda", dtype=torch.float64)
    starts, ends = st["starts"].tolist(), st["row_ends"].tolist()
    for j, table in enumerate(st["block_table"]):
        rows = range(starts[j], starts[j + 1])
        if c["op"] == "paged":
            p = torch.arange(max(ends[r] for r in rows), device="cuda")
            blocks = [(list(rows), p, torch.stack([p < ends[r] for r in rows]))]
        else:
            blocks = []
            for r in rows:
                p = st["topk"][r].long()
                p = p[p >= 0]
                blocks.append(([r], p, torch.ones((1, p.numel()), dtype=torch.bool, device="cuda")))
        for which, p, seen in blocks:
            if not p.numel():
                continue
            k, v = (x.transpose(0, 1) for x in tokens(table.long()[p // PAGE] * PAGE + p % PAGE))
            x = q[which].unflatten(1, (hkv, group)).transpose(0, 1).flatten(1, 2)       # [hkv, rows * group, d]
            s = torch.einsum("hmd,htd->hmt", x, k) * scale
            s = s.masked_fill(~seen.repeat_interleave(group, 0), float("-inf"))
            l = torch.logsumexp(s, dim=-1)
            o = torch.einsum("hmt,htd->hmd", torch.exp(s - l.masked_fill(l == float("-inf"), 0.0)[..., None]), v)
            out[which] = o.unflatten(1, (len(which), group)).transpose(0, 1).flatten(1, 2)
            lse[which] = l.unflatten(1, (len(which), group)).transpose(0, 1).flatten(1, 2)
    return out, lse
