"""Build the CUDA library ``libdsa.so`` in-tree for sm_103a (GB300), and the
small Python extension that binds its append and attention calls.

Each translation unit is compiled in parallel (nvcc; the host compiler for the
extension), then linked into shared libraries next to this file.  No CMake; a
minute or two on an Arm GB300 host.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libdsa.so")
BINDING = os.path.join(HERE, "_dsa_binding.so")
BUILT_WITH = os.path.join(BUILD_DIR, "built_with.txt")
SOURCES = ["quant.cu", "layout.cu", "score.cu", "topk.cu", "norm.cu", "probe.cu", "kvcache.cu", "attend.cu",
           "kvfp4.cu", "attend_fp4_paged.cu", "attend_fp4_selected.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: set CUDA_HOME or put nvcc on PATH")
    return found


def _tools() -> str:
    """What the extension is compiled against besides the sources: torch and Python, by version and place."""
    import torch

    return "\n".join([torch.__version__, torch.__file__, sys.version])


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    try:
        with open(BUILT_WITH) as f:
            if f.read() != _tools():
                return True
    except OSError:
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "dsa.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the libraries if any source is newer than them, or torch or Python is another than they were
    compiled for; return ``libdsa.so``'s path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        binding = pool.submit(_compile_binding)
        objs = list(pool.map(compile_one, SOURCES))
        binding_obj = binding.result()
    tmp = LIB + ".tmp"
    # Shared CUDA runtime: in a process that imported torch, the loader reuses
    # torch's libcudart.so.13, so the library and torch share one runtime
    # (current device, streams, events).  The rpath is the fallback for C callers.
    libdir = os.path.join(os.path.dirname(os.path.dirname(cc)), "lib64")
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs, f"-Xlinker=-rpath,{libdir}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding_obj)
    with open(BUILT_WITH, "w") as f:
        f.write(_tools())
    return LIB


def _run(cmd, what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def _compile_binding() -> str:
    import sysconfig

    import torch

    obj = os.path.join(BUILD_DIR, "binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = [f"-I{d}" for d in (os.path.join(os.path.dirname(torch.__file__), "include"),
                              sysconfig.get_paths()["include"], cuda)]
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
    _run(["g++", "-O2", "-std=c++17", "-fPIC", abi, *inc, "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj],
         "g++ on binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    import torch

    # torch's libraries are in the process already (the package imports torch first);
    # libdsa.so is found next to the extension.
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libdsa.so", f"-L{torch_lib}", "-ltorch_python",
          "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], "link of the binding")
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
