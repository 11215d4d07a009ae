"""A dispatch mode (a memory tracker, a tracer) sees the outputs that the append and attention calls allocate, and
results are the same under it and under deterministic algorithms."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import attend_case
import fp4_case

pytestmark = pytest.mark.gpu


class Empties(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.sizes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.sizes.append(tuple(out.shape))
        return out


def calls(dsa):
    """name: (call, the shapes it allocates as outputs)"""
    a = attend_case.Case([70, 200], [1, 2], hq=8, hkv=2, dim=64)
    f = fp4_case.Case([70, 200], [1, 2], hq=8, hkv=2, dim=64)
    lists = [x(c, 30) for x, c in ((attend_case.choose, a), (fp4_case.choose, f))]
    q, lse, kv = (3, 8, 64), (3, 8), (3, 2, 64)
    rows = torch.randn((3, 2, 64), device="cuda").bfloat16()
    slots = torch.tensor([3, 64, -1], device="cuda")
    append = (rows, rows, slots)
    caches = (torch.zeros((2, 64, 2, 64), dtype=torch.bfloat16, device="cuda"),) * 2
    cache = dsa.new_kv_cache_fp4(2, 2, 64, "cuda")
    return {"kv_append": (lambda: dsa.kv_append(*append, caches[0], caches[1].clone(), q=a.q), [q]),
            "attend_paged": (lambda: a.paged(dsa), [q]),
            "attend_selected": (lambda: a.selected(dsa, lists[0]), [q]),
            "kv_append_fp4": (lambda: dsa.kv_append_fp4(*append, cache, q=f.q), [q]),
            "kv_read_fp4": (lambda: dsa.kv_read_fp4(slots, cache, 64), [kv, kv]),
            "attend_paged_fp4": (lambda: f.paged(dsa), [q, lse]),
            "attend_selected_fp4": (lambda: f.selected(dsa, lists[1]), [q, lse])}


NAMES = ["kv_append", "attend_paged", "attend_selected", "kv_append_fp4", "kv_read_fp4", "attend_paged_fp4",
         "attend_selected_fp4"]


def tensors(x):
    return [t for t in (x if isinstance(x, tuple) else (x,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_a_dispatch_mode_sees_the_outputs(cuda_lib, name):
    call, shapes = calls(cuda_lib)[name]
    want = tensors(call())
    with Empties() as seen:
        got = tensors(call())
    for s in shapes:
        assert s in seen.sizes, (s, seen.sizes)
        seen.sizes.remove(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("name", NAMES)
def test_under_deterministic_algorithms(cuda_lib, name):
    call, _ = calls(cuda_lib)[name]
    want = tensors(call())
    torch.use_deterministic_algorithms(True)
    try:
        got = tensors(call())
    finally:
        torch.use_deterministic_algorithms(False)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
