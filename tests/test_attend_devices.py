"""Every tensor of the append and attention calls has to be on the caches' device: one of them elsewhere is refused
before anything is launched.  On the CPU the one elsewhere is a meta tensor, on the GPU a host tensor."""

import pytest
import torch

BF = torch.bfloat16
I32, I64, U8 = torch.int32, torch.int64, torch.uint8


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_indexer_score_gb300 import build
    try:
        build.build()
    except RuntimeError as e:   # no nvcc on this machine
        pytest.skip(str(e))
    from sparse_attention_indexer_score_gb300 import dsa as d
    return d


def append_args(device):
    z = lambda *n, dtype: torch.zeros(n, dtype=dtype, device=device)   # noqa: E731
    return dict(k=z(3, 2, 64, dtype=BF), v=z(3, 2, 64, dtype=BF), slots=z(3, dtype=I64), k_cache=z(2, 64, 2, 64, dtype=BF),
                v_cache=z(2, 64, 2, 64, dtype=BF), positions=z(3, dtype=I64), cos_sin=z(9, 64, dtype=torch.float32),
                q=z(3, 4, 64, dtype=BF), q_out=z(3, 4, 64, dtype=BF), status=z(1, dtype=I32))


def attend_args(device, size):
    z = lambda *n, dtype: torch.zeros(n, dtype=dtype, device=device)   # noqa: E731
    return dict(q=z(2, 8, 64, dtype=BF), k_cache=z(3, 64, 2, 64, dtype=BF), v_cache=z(3, 64, 2, 64, dtype=BF),
                block_table=z(1, 3, dtype=I32), starts=z(2, dtype=I32), row_ends=z(2, dtype=I32),
                out=z(2, 8, 64, dtype=BF), workspace=z(size, dtype=U8), status=z(1, dtype=I32))


APPEND = ["k", "v", "slots", "k_cache", "v_cache", "positions", "cos_sin", "q", "q_out", "status"]
ATTEND = ["q", "k_cache", "v_cache", "block_table", "starts", "row_ends", "out", "workspace", "status"]


def calls(dsa, device):
    size = max(dsa.attend_workspace_size(2, 1, 8, 2, 64, 2), dsa.attend_workspace_size(2, 1, 8, 2, 64, 2, 4))
    shared = attend_args(device, size)
    return {"append": (dsa.kv_append, append_args(device)),
            "paged": (dsa.attend_paged, dict(shared, max_query_len=2, prefix_len=64,
                                             prefix_pages=torch.zeros(1, dtype=I32, device=device))),
            "selected": (dsa.attend_selected, dict(shared, topk=torch.zeros(2, 4, dtype=I32, device=device)))}


CASES = [("append", n) for n in APPEND] + [("paged", n) for n in ATTEND + ["prefix_pages"]] + \
        [("selected", n) for n in ATTEND + ["topk"]]


@pytest.mark.parametrize("call,name", CASES)
def test_a_tensor_on_another_device_is_refused(dsa, call, name):
    fn, args = calls(dsa, "cpu")[call]
    with pytest.raises(ValueError, match="device"):
        fn(**dict(args, **{name: args[name].to("meta")}))


@pytest.mark.gpu
@pytest.mark.parametrize("call,name", CASES)
def test_a_host_tensor_among_gpu_tensors_is_refused(cuda_lib, call, name):
    fn, args = calls(cuda_lib, "cuda")[call]
    with pytest.raises(ValueError, match="device"):
        fn(**dict(args, **{name: args[name].cpu()}))
    with pytest.raises(ValueError, match="device"):
        fn(**dict(args, **{name: args[name].cpu().pin_memory()}))


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["append", "paged", "selected"])
def test_the_same_tensors_on_one_gpu_are_taken(cuda_lib, call):
    fn, args = calls(cuda_lib, "cuda")[call]
    fn(**args)
    torch.cuda.synchronize()
    assert int(args["status"]) == 0


def test_a_workspace_with_gaps_is_refused(dsa):
    """Its size counts elements, its span is what the kernels would write."""
    for call in ("paged", "selected"):
        fn, args = calls(dsa, "cpu")[call]
        n = args["workspace"].numel()
        for ws in (torch.zeros(2 * n, dtype=U8)[::2], torch.zeros(1, dtype=U8).expand(n)):
            with pytest.raises(ValueError, match="contiguous"):
                fn(**dict(args, workspace=ws))
