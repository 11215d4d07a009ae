"""Where the scoring and top-k calls of different sizes keep what in one workspace (CPU only: the layout is host code).

Histograms and counters have to be zero when a call starts, and a call clears its own.  So no call may leave other
bytes where another one counts, whatever their rows, widths and kinds, as long as the workspace was sized for all."""

import itertools
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_indexer_score_gb300", "csrc")
PROGRAM = """
#include <stdio.h>
#include "workspace.h"
int main() {
    long long rows, width, bytes;
    int plan, logits;
    while (scanf("%lld %lld %d %d %lld", &rows, &width, &plan, &logits, &bytes) == 5) {
        const dsa::WsLayout L = dsa::workspace_layout(rows, width, plan, logits, bytes);
        printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu %zu %zu\\n", L.hist, L.counters, L.zeroed, L.info, L.segs,
               L.seg_prefix, L.eff_end, L.cta, L.cand, L.logits, L.total);
    }
}
"""


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("layout")
    (d / "layout.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", f"-I{CSRC}", str(d / "layout.cpp"), "-o", str(d / "layout")], check=True)

    def run(calls):
        text = "\n".join(" ".join(map(str, c)) for c in calls)
        out = subprocess.run([str(d / "layout")], input=text, capture_output=True, text=True, check=True).stdout
        return [list(map(int, line.split())) for line in out.splitlines()]

    return run


def regions(call, at):
    """(start, end) of the counting regions, and of all others."""
    rows, width, plan, logits, _ = call
    hist, counters, zeroed, info, segs, prefix, ends, cta, cand, lg, _ = at
    counts = [(hist, hist + rows * 8192), (counters, counters + rows * 16)]
    other = [(cand, cand + rows * 65536)]
    if plan:
        other += [(info, info + 32), (segs, segs + 16 * (rows + 1)), (prefix, prefix + 4 * (rows + 2)),
                  (ends, ends + 4 * rows), (cta, cta + 16 * 1024)]
    if logits:
        other.append((lg, lg + rows * width * 4))
    return [r for r in counts if r[1] > r[0]], [r for r in other if r[1] > r[0]]


def apart(a, b):
    return a[1] <= b[0] or b[1] <= a[0]


@pytest.mark.parametrize("seed", range(20))
def test_no_call_leaves_bytes_where_another_counts(layout, seed):
    rng = random.Random(seed)
    most_rows, most_width = rng.randint(1, 400), rng.choice([0, 64, 640, 65536]) * rng.randint(1, 3)
    need = layout([(most_rows, most_width, 1, 1, 0)])[0][-1]
    size = need + rng.choice([0, 0, 1, 255, 4096, 10 ** 6])
    calls = [(rng.randint(1, most_rows), rng.randint(0, most_width), plan, logits and plan, size)
             for plan, logits in itertools.product((0, 1), repeat=2) for _ in range(6)] + \
            [(most_rows, most_width, 1, 1, size)]
    laid = [regions(c, at) for c, at in zip(calls, layout(calls))]
    for counts, other in laid:
        every = counts + other
        assert all(0 <= s and e <= size for s, e in every) and all(s % 256 == 0 for s, _ in every)
        assert all(apart(a, b) for a, b in itertools.combinations(every, 2))
        for counts2, _ in laid:
            assert all(apart(a, b) for a in other for b in counts2)


def test_sizes_have_not_changed(layout):
    """A workspace of the size that a call asks for is one just large enough, whatever its kind."""
    for rows, width, plan, logits in [(1, 64, 1, 1), (335, 65536, 1, 1), (335, 65536, 1, 0), (64, 0, 0, 0)]:
        exact = layout([(rows, width, plan, logits, 0)])[0]
        assert layout([(rows, width, plan, logits, exact[-1])])[0] == exact
        counts, other = regions((rows, width, plan, logits, 0), exact)
        assert exact[-1] == max(-(-e // 256) * 256 for _, e in counts + other)
