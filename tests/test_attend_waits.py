"""Waits of the attention kernel, read from its source (CPU only: a wait that runs out is not provoked on a GPU).

Its roles may give up separately, so no role may wait for another without a limit: a named barrier has none, and a
warp that has left leaves its partner there for good.  What stays are the mbarrier waits with a time limit, and the
block-wide barriers that every thread reaches whatever its role did.
"""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_indexer_score_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_role_waits_at_a_named_barrier():
    assert not re.findall(r"\"[^\"]*\b(?:bar|barrier)\.(?:cta\.)?(?:sync|red|arrive)\b", code("attend.cu"))


def test_every_mbarrier_wait_has_a_limit():
    src = code("attend.cu")
    assert not re.findall(r"\bmbar_try_wait\b", src)                 # only inside the bounded waits
    body = code("common.cuh")
    for name in ("mbar_wait", "mbar_drain"):
        text = body[body.index(f"bool {name}("):]
        text = text[:text.index("\n}\n")]
        assert "globaltimer()" in text and "return false" in text, name


def test_block_barriers_stand_outside_the_roles():
    """__syncthreads in the kernel: before the roles part and after they have met again."""
    src = code("attend.cu")
    kernel = src[src.index("    attend_kernel(const __grid_constant__"):]
    kernel = kernel[:kernel.index("\n}\n")]
    roles, done = kernel.index("if (warp < 2 || copies)"), kernel.index("done:")
    assert "__syncthreads" not in kernel[roles:done]
    assert kernel[done:].count("__syncthreads") == 1
