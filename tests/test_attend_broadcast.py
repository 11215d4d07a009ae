"""Outputs and caches that are broadcast, several elements in one place, are refused (CPU only: no call here reaches
the GPU); one element may have a stride of zero."""

import pytest

from test_attend_args import APPEND, PAGED, SELECTED, call, dsa   # noqa: F401  (the fixture)


@pytest.mark.parametrize("fn,base", [("dsa_attend_paged", PAGED), ("dsa_attend_selected", SELECTED)])
def test_outputs_of_attention(dsa, fn, base):   # noqa: F811
    assert call(dsa, fn, base, None, rows=2, orow=0) == -1
    assert call(dsa, fn, base, None, oh=0) == -1
    # one row: past this check, to the workspace's size
    assert call(dsa, fn, base, None, orow=0, wsb=0) == -1 == call(dsa, fn, base, None, wsb=0)


def test_outputs_of_the_append(dsa):   # noqa: F811
    for kw in (dict(ot=0), dict(oh=0)):
        assert call(dsa, "dsa_kv_append", APPEND, None, **kw) == -1
    for name in ("k_page_stride", "v_page_stride", "k_token_stride", "v_token_stride", "k_head_stride", "v_head_stride"):
        assert call(dsa, "dsa_kv_append", APPEND, {name: 0}) == -1, name
