"""Flags that are neither true nor false (CPU only: refused before the device is looked at)."""

import pytest
import torch

from test_attend_devices import append_args, attend_args, dsa   # noqa: F401  (the fixture)


class Neither:
    def __bool__(self):
        raise RuntimeError("neither")


@pytest.mark.parametrize("flag", [torch.zeros(2), Neither()], ids=["tensor", "object"])
def test_a_flag_that_is_neither(dsa, flag):   # noqa: F811
    with pytest.raises(ValueError, match="true or false"):
        dsa.kv_append(**append_args("cpu"), interleaved=flag)
    args = attend_args("cpu", 1 << 20)
    with pytest.raises(ValueError, match="true or false"):
        dsa.attend_paged(**args, max_query_len=1, want_lse=flag)
    with pytest.raises(ValueError, match="true or false"):
        dsa.attend_selected(**args, topk=torch.zeros(2, 4, dtype=torch.int32), want_lse=flag)
    dsa.attend_workspace_size(1, 1, 8, 2, 64, 1)      # and no error is left behind for the next call
