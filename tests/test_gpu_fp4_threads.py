"""Host threads that call the 4-bit attention at the same time, each with a stream and a workspace of its own, and
calls over heads of several widths in either order: results are those of each call alone."""

import ctypes
import hashlib
import os
import subprocess
import sys
import threading

import pytest
import torch

from fp4_case import Case

pytestmark = pytest.mark.gpu

DIMS = (16, 48, 64, 80, 112, 128)


def cases(dims):
    return [Case([300 + 40 * j for j in range(9)], [2] * 9, hq=8, hkv=8 if dim < 100 else 2, dim=dim, seed=dim) for dim in dims]


def hashes(dsa, dims):
    return {c.dim: hashlib.sha256(c.paged(dsa)[0].view(torch.int16).cpu().numpy().tobytes()).hexdigest() for c in cases(dims)}


def test_the_first_width_does_not_decide_for_the_others(cuda_lib):
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "from sparse_attention_indexer_score_gb300 import dsa\nimport test_gpu_fp4_threads as t\n"
            "print(sorted(t.hashes(dsa, [int(x) for x in sys.argv[1:]]).items()))" % (os.path.dirname(here), here))
    got = [subprocess.run([sys.executable, "-c", code, *map(str, dims)], capture_output=True, text=True, timeout=300)
           for dims in (DIMS, DIMS[::-1])]
    assert [g.returncode for g in got] == [0, 0], got[0].stderr + got[1].stderr
    assert got[0].stdout == got[1].stdout and "112" in got[0].stdout


def test_threads_at_once(cuda_lib):
    dsa, cs = cuda_lib, cases(DIMS)
    want = [c.paged(dsa)[0] for c in cs]
    outs = [[torch.zeros_like(c.q) for _ in range(20)] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    args = []
    for c, stream in zip(cs, streams):
        rows, hq, dim = c.q.shape
        t = c.cache
        cache = dsa.KvCacheFp4(t.data_ptr(), t.stride(0), t.stride(1), t.shape[0], t.shape[1], dim, 1.0, 1.0)
        ws = torch.empty(dsa.attend_workspace_size_fp4(rows, 9, hq, c.hkv, dim, 2), dtype=torch.uint8, device="cuda")
        args.append((cache, ws, [ctypes.addressof(cache), 0, c.q.data_ptr(), hq * dim, dim, hq, c.block_table.data_ptr(),
                                 c.block_table.stride(0), c.block_table.shape[1], c.starts.data_ptr(),
                                 c.row_ends.data_ptr(), 9, rows, 2, c.scale], stream))
    torch.cuda.synchronize()
    gate, codes = threading.Barrier(len(cs)), []

    def work(i):
        _, ws, first, stream = args[i]
        hq, dim = cs[i].q.shape[1:]
        gate.wait()
        for out in outs[i]:
            codes.append(dsa.lib().dsa_attend_paged_fp4(*first, out.data_ptr(), hq * dim, dim, None, ws.data_ptr(),
                                                        ws.numel(), None, stream.cuda_stream))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [0] * 20 * len(cs)
    for w, os_ in zip(want, outs):
        assert all(torch.equal(w, o) for o in os_)
