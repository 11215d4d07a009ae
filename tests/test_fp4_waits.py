"""Waits of the 4-bit attention kernels, read from their source (CPU only: a wait that runs out is not provoked on a
GPU): every one has a limit, and a warp whose wait ran out lets its copies land and starts no more."""

import re

from test_attend_waits import code


def kernel(src, name):
    body = src[src.index(f"\n{name}(const Att4Params p)") if f"\n{name}(const Att4Params p)" in src else
               src.index(f" {name}(const Att4Params p)"):]
    return body[:body.index("\n}\n")]


def test_no_wait_without_a_limit():
    src = code("attend_fp4.cuh")
    assert not re.findall(r"\"[^\"]*\b(?:bar|barrier)\.(?:cta\.)?(?:sync|red|arrive)\b", src)
    assert not re.findall(r"\bmbar_try_wait\b", src)


def test_a_warp_that_gave_up_starts_no_more_copies():
    src = code("attend_fp4.cuh")
    cluster = kernel(src, "attend_fp4_cluster_kernel")
    failed = cluster[cluster.index("if (!__all_sync(0xFFFFFFFFu, ok))"):]
    failed = failed[:failed.index("break;")]
    assert "mbar_drain(" in failed and "count = 0;" in failed
    copy = cluster[cluster.index("auto copy = [&](int tile, int i)"):]
    copy = copy[:copy.index("\n    };\n")]
    assert copy.count("i < count") == 2                      # of either kind of keys
    axis = kernel(src, "attend_fp4_kernel")
    failed = axis[axis.index("if (!__all_sync(0xFFFFFFFFu, landed))"):]
    assert "gave_up = true;" in failed[:failed.index("break;")]
    assert "while (i < count && !gave_up)" in axis and "else if (gave_up)" in axis


def test_block_and_cluster_barriers_are_reached_by_every_warp():
    """No return, and none of them inside a unit's loop, where a warp may leave."""
    cluster = kernel(code("attend_fp4.cuh"), "attend_fp4_cluster_kernel")
    assert not re.findall(r"\breturn;", cluster)
    units = cluster[cluster.index("for (int i = 0; i < count && x.nq > 0; ++i)"):]
    units = units[:units.index("\n        }\n")]
    assert "__syncthreads" not in units and "cluster.sync" not in units
    assert cluster.count("__syncthreads") == 1 and cluster.count("cluster.sync()") == 2
