"""Where a segment goes on the axis when requests overlap (CPU only: the arithmetic of the plan, in its own types).

The bounds of requests are device data: 512 of them, every other one over all of 2^24 rows in tiles of one row, claim
2^32 segments before the plan's first chunk ends.  The place of a segment has to stay past the last one then."""

import os
import re

import numpy as np

CU = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                  "sparse_attention_indexer_score_gb300", "csrc", "attend.cu")
TYPES = {"int": np.int32, "int64_t": np.int64}


def test_the_place_of_a_segment_does_not_wrap():
    with open(CU) as f:
        src = f.read()
    body = src[src.index("__device__ int64_t lay_out("):]
    kind, expr = re.search(r"const (\w+) at = ([^;]*block_scan64[^;]*);", body).groups()
    rows, threads = 1 << 24, 512
    max_segs = rows + threads
    claims = np.where(np.arange(threads) % 2 == 0, rows, 0).astype(np.int64)
    before = np.cumsum(claims) - claims
    assert before.max() > 2 ** 31
    narrowed = "static_cast<int>(" in expr
    place = (before.astype(np.int32) if narrowed else before).astype(TYPES[kind])
    assert ((place >= 0) & ((before < max_segs) | (place >= max_segs))).all()
