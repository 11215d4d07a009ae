"""Values that are not finite and that a row sees, in every kind of tile: an output column with such values of one
sign is infinite of that sign, with both signs or a NaN among them it is NaN, and no other column changes by a bit."""

import pytest
import torch

from attend_case import Case, choose

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

# narrow tiles of 8 and 16 rows, wide ones, one request alone (an output without a join) and many pieces of one row
FORMS = [dict(hq=8, hkv=2, dim=64), dict(hq=16, hkv=1, dim=128), dict(hq=40, hkv=2, dim=80), dict(hq=128, hkv=1, dim=128)]
IDS = [f"{f['hq']}x{f['hkv']}x{f['dim']}" for f in FORMS]


def place(c, j, t):
    """(page, token) of key t of request j, or of the prefix (j = -1)."""
    return int(c.prefix_pages[t // 64] if j < 0 else c.block_table[j, t // 64]), t % 64


def plant(c, spots):
    """spots: (request, key, head, column, value); returns the columns' outputs as {(request, head, column): value}."""
    want = {}
    for j, t, h, x, value in spots:
        p, i = place(c, j, t)
        c.v[p, i, h, x] = value
        have = want.get((j, h, x))
        want[j, h, x] = value if have is None else have + value     # inf - inf is NaN
    return want


def check(c, before, after, want, sees):
    """`sees(row, request)`: whether the row sees the request's (or prefix's, -1) planted values."""
    out, ref = after[0].float().cpu(), before[0].float().cpu()
    assert torch.isfinite(ref).all() and torch.equal(before[1], after[1])     # the log-sum-exp has no values in it
    group = out.shape[1] // c.k.shape[2]
    touched = torch.zeros(out.shape, dtype=torch.bool)
    for r in range(out.shape[0]):
        for (j, h, x), value in want.items():
            if not sees(r, j):
                continue
            for g in range(h * group, (h + 1) * group):
                touched[r, g, x] = True
                got = float(out[r, g, x])
                assert got == value or (value != value and got != got), (r, g, x, value, got)
    assert torch.equal(out[~touched], ref[~touched])


def spots(j, n, dim, hkv):
    """Columns with one infinity, two of one sign, both signs, NaN; first and last keys, heads and columns."""
    last = hkv - 1
    return [(j, 0, 0, 0, INF), (j, n - 1, last, dim - 1, -INF), (j, n // 2, 0, 5, INF), (j, n // 3, 0, 5, INF),
            (j, n // 2, 0, 17, -INF), (j, n - 1, 0, 17, INF), (j, n // 3, last, 33, NAN), (j, n // 2, last, 40, -INF)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("lens", [[70], [200, 33, 131], [9000, 100]], ids=str)
def test_values_that_every_row_sees(cuda_lib, lens, form, dtype):
    c = Case(lens, [1] * len(lens), dtype=dtype, **form)
    topk = choose(c, max(lens))                                       # every key, in another order, with holes
    before, listed = c.paged(cuda_lib), c.selected(cuda_lib, topk)
    want = {}
    for j, n in enumerate(lens):
        want |= plant(c, spots(j, n, form["dim"], form["hkv"]))
    check(c, before, c.paged(cuda_lib), want, lambda r, j: r == j)
    check(c, listed, c.selected(cuda_lib, topk), want, lambda r, j: r == j)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_values_that_only_the_last_row_sees(cuda_lib, form, dtype):
    lens = [150, 64, 2000]
    c = Case(lens, [3, 2, 4], dtype=dtype, **form)
    before = c.paged(cuda_lib)
    want = {}
    for j, n in enumerate(lens):
        want |= plant(c, [(j, n - 1, 0, 3, INF), (j, n - 1, 0, 9, NAN), (j, n - 1, form["hkv"] - 1, 47, -INF)])
    check(c, before, c.paged(cuda_lib), want, lambda r, j: r == [2, 4, 8][j])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_values_of_a_prefix(cuda_lib, form, dtype):
    c = Case([40, 200, 0], [1, 2, 1], prefix=700, dtype=dtype, **form)
    before = c.paged(cuda_lib)
    want = plant(c, spots(-1, 700, form["dim"], form["hkv"]))
    check(c, before, c.paged(cuda_lib), want, lambda r, j: True)


def test_values_of_a_long_prefix_in_pairs_of_row_tiles(cuda_lib):
    c = Case([(37 * j) % 150 for j in range(65)], [1] * 65, prefix=7301, hq=128, hkv=1, dim=64, dtype="fp16")
    assert 33 * -(-7301 // 128) > 12 * torch.cuda.get_device_properties(0).multi_processor_count
    before = c.paged(cuda_lib)
    want = plant(c, spots(-1, 7301, 64, 1))
    check(c, before, c.paged(cuda_lib), want, lambda r, j: True)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (40, 2)])
def test_an_infinite_value_of_a_small_weight(cuda_lib, hq, hkv):
    """A weight of 2^-60 is zero in FP16, but not in the sum: the output is infinite all the same."""
    c = Case([130], [1], hq=hq, hkv=hkv, dim=64, dtype="fp16")
    p, i = place(c, 0, 64)
    c.q.fill_(1.0)
    c.k[c.block_table[0].clamp(min=0).long()] = 0.0
    c.k[p, i] = -60 * 0.6931 / 8                                      # score 64 * this / 8
    before = c.paged(cuda_lib)
    want = plant(c, [(0, 64, 0, 7, INF), (0, 64, hkv - 1, 8, -INF)])
    check(c, before, c.paged(cuda_lib), want, lambda r, j: True)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (128, 1)])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_a_cache_full_of_one_such_value(cuda_lib, value, hq, hkv):
    """Every column of every row, long pieces among them, without a wait running out."""
    c = Case([30000, 100], [1, 2], prefix=5000, hq=hq, hkv=hkv, dim=128)
    topk = choose(c, 2000)
    c.v.fill_(value)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out, _ in (c.paged(cuda_lib, status=status), c.selected(cuda_lib, topk, status=status)):
        assert torch.isnan(out).all() if value != value else (out == value).all()
    assert int(status) == 0
