"""Build libpkv.so (the CUDA kernels + the C ABI of include/pkv.h) in-tree for sm_103a.

Each translation unit is compiled by nvcc in parallel, then linked into one shared
library next to this file (``_lib/libpkv.so``).  Beside it goes ``_lib/_pkv_prompt.so``, the
marshalling of the prompt side's calls from torch tensors (``csrc/prompt_bind.cpp``), compiled by the host
compiler against torch's headers.  No CMake, no torch extension machinery.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libpkv.so")
BIND = os.path.join(OUT_DIR, "_pkv_prompt.so")
SOURCES = ["pkv_api.cu", "append.cu", "decode_bf16.cu", "decode_e4m3.cu", "pkv_noalloc.cu", "copy_blocks.cu",
           "block_manager.cpp", "cascade_bf16.cu", "cascade_e4m3.cu",
           "decode_mma.cu", "decode_mma_e4m3.cu",
           "merge_partitions.cu", "cascade_prefix_tc.cu", "cascade_prefix_mma.cu", "kv_checksum.cu", "stage_copy.cu",
           "qk_rope_append.cu", "prefill_tc.cu", "merge_prefill.cu", "kv_gather.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
                   "-I", CSRC, *extra]


def _stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BIND)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    inc = os.path.join(ROOT, "include")
    deps = ([os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(inc, f) for f in os.listdir(inc)]
            + [__file__])
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _bind_flags():
    """(compile, link) flags of prompt_bind.cpp: torch's headers and libraries, found without
    importing torch."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(torch, "lib")
    return (["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w", *[x for i in inc for x in ("-isystem", i)]],
            ["-shared", "-L", lib, "-L", OUT_DIR, "-lpkv", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
             "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libpkv.so and _pkv_prompt.so if any source is newer; returns the library's path."""
    if not force and not _stale():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    obj_dir = os.path.join(OUT_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *_flags(extra_flags), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    bind_cc, bind_ld = _bind_flags()
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    bind_obj = os.path.join(obj_dir, "prompt_bind.o")

    def run(cmd, what: str) -> None:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(run, [cxx, *bind_cc, "-c", os.path.join(CSRC, "prompt_bind.cpp"), "-o", bind_obj],
                         "compiling prompt_bind.cpp")
        objs = list(ex.map(compile_one, SOURCES))
        bind.result()
    tmp = LIB + f".tmp{os.getpid()}"
    run([cc, *ARCH, "-shared", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB)
    tmp = BIND + f".tmp{os.getpid()}"
    run([cxx, "-o", tmp, bind_obj, *bind_ld], "link of _pkv_prompt.so")
    os.replace(tmp, BIND)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
