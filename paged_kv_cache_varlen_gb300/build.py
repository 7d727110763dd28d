"""Build ``libpkv.so`` in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel into ``_build/``; the objects are
linked into ``paged_kv_cache_varlen_gb300/libpkv.so`` (static cudart, no
driver-library link: the tensor-map encoder is looked up at run time).
``_marshal.so`` beside it is the Python module that marshals the arguments of
the per-step calls (host code against torch's and Python's headers; it calls
libpkv.so). The library needs nvcc alone: where torch is not installed, it is
all that is built, and a binding module that fails to build leaves it there.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(PKG, "_build")
LIBRARY = os.path.join(PKG, "libpkv.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_SOURCE = "marshal.cpp"
SOURCES = ["kv_write.cu", "decode_mma.cu", "decode_rows.cu", "merge.cu", "prefill_tc.cu",
           "prefill_rows.cu", "copy_blocks.cu", "rope_write.cu", "norm_write.cu",
           "key_weights.cu", "key_weights_tc.cu", "evict.cu", "api.cpp", "budget_api.cpp", "cache8_api.cpp",
           "window_api.cpp", "api_noalloc.cu", "block_manager.cpp"]
HEADERS = [os.path.join(CSRC, "common.cuh"), os.path.join(CSRC, "launch.h"),
           os.path.join(CSRC, "key_weights.cuh"), os.path.join(CSRC, "rope.cuh"),
           os.path.join(CSRC, "wait.cuh"), os.path.join(CSRC, "e4m3.cuh"),
           os.path.join(ROOT, "include", "pkv.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fno-strict-aliasing"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_input() -> float:
    files = ([os.path.join(CSRC, s) for s in SOURCES + [MARSHAL_SOURCE]] + HEADERS
             + [os.path.abspath(__file__)])
    return max(os.path.getmtime(f) for f in files)


def up_to_date() -> bool:
    newest = _newest_input()
    parts = (LIBRARY, MARSHAL) if _have_torch() else (LIBRARY,)
    return all(os.path.exists(f) and os.path.getmtime(f) >= newest for f in parts)


def _have_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _torch_paths() -> tuple[list[str], str]:
    """Include flags of torch, Python and CUDA, and torch's library folder."""
    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    include = os.path.join(root, "include")
    dirs = [include, os.path.join(include, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"]]
    flags = [f"-I{d}" for d in dirs]
    flags.append(f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}")
    return flags, os.path.join(root, "lib")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    if src == MARSHAL_SOURCE:
        cmd += _torch_paths()[0]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
    if verbose and res.stderr:
        print(res.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libpkv.so unless it is newer than every source."""
    if not force and up_to_date():
        return LIBRARY
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        marshal = pool.submit(_compile, MARSHAL_SOURCE, verbose) if _have_torch() else None
        objs = list(pool.map(lambda s: _compile(s, verbose), SOURCES))
        _link(LIBRARY, objs, [])
        if marshal is None:
            return LIBRARY
        obj = marshal.result()
    torch_lib = _torch_paths()[1]
    _link(MARSHAL, [obj],
          [f"-L{os.path.dirname(LIBRARY)}", "-l:libpkv.so", f"-L{torch_lib}", "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           "-Xlinker", "-rpath,$ORIGIN", "-Xlinker", f"-rpath,{torch_lib}"])
    return LIBRARY


def _link(target: str, objs: list[str], extra: list[str]) -> None:
    tmp = target + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, *extra, "-cudart", "static"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, target)


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
