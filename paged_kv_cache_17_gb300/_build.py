"""Build libpkv.so (the CUDA kernels + the C ABI of include/pkv.h) in-tree for sm_103a.

Each translation unit is compiled by nvcc in parallel, then linked into one shared
library next to this file (``_lib/libpkv.so``).  Beside it goes ``_lib/_pkv_prompt.so``, the
marshalling of the prompt side's calls from torch tensors (``csrc/prompt_bind.cpp``), compiled by the host
compiler against torch's headers (left out where those are not installed).  No CMake, no torch extension machinery.
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
BOUND_TO = BIND + ".bound_to"  # the torch and Python it was built against
BIND_LIBS = ("c10", "c10_cuda", "torch_cpu", "torch_python")
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


def _newer(target: str, deps) -> bool:
    """Whether target is missing or older than one of deps."""
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps
                                             if os.path.exists(d))


def _stale_lib() -> bool:
    inc = os.path.join(ROOT, "include")
    return _newer(LIB, [os.path.join(d, f) for d in (CSRC, inc) for f in os.listdir(d) if f != "prompt_bind.cpp"]
                  + [__file__])


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")  # (without importing it)
    return spec.submodule_search_locations[0] if spec else ""


def _bound_to() -> str:
    """What _pkv_prompt.so is bound to: this torch and this Python."""
    version = os.path.join(_torch_dir(), "version.py")
    if not os.path.exists(version):
        return ""
    with open(version) as f:
        return f"{sysconfig.get_config_var('SOABI')} {version} {int(os.path.getmtime(version))}\n{f.read()}"


def _stale_bind() -> bool:
    if _newer(BIND, [os.path.join(CSRC, "prompt_bind.cpp"), os.path.join(ROOT, "include", "pkv.h"), __file__]):
        return True
    if not os.path.exists(BOUND_TO):
        return True
    with open(BOUND_TO) as f:
        return f.read() != _bound_to()


def _bind_lacks() -> str:
    """What is not there to build _pkv_prompt.so with, or ''."""
    torch = _torch_dir()
    if not torch:
        return "torch"
    for path in (os.path.join(torch, "include", "ATen", "ATen.h"),
                 os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                 *(os.path.join(torch, "lib", f"lib{n}.so") for n in BIND_LIBS)):
        if not os.path.exists(path):
            return path
    return ""


def _bind_flags():
    """(compile, link) flags of prompt_bind.cpp: torch's headers and libraries, found without
    importing torch."""
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(torch, "lib")
    return (["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w", *[x for i in inc for x in ("-isystem", i)]],
            ["-shared", "-L", lib, "-L", OUT_DIR, "-lpkv", *(f"-l{n}" for n in BIND_LIBS), "-Wl,-rpath,$ORIGIN",
             "-Wl,-rpath," + lib])


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link what is older than its sources (_pkv_prompt.so also: bound to another torch or Python);
    returns the library's path.  Where torch's or Python's headers are not installed, libpkv.so alone is
    built, with a warning: the prompt side's calls then raise, everything else works."""
    make_lib, make_bind = force or _stale_lib(), force or _stale_bind()
    lacks = _bind_lacks() if make_bind else ""
    if lacks:
        make_bind = False
        for old in (BIND, BOUND_TO):
            if os.path.exists(old):
                os.remove(old)
        print(f"warning: _pkv_prompt.so is not built, {lacks} is missing; the prompt side's calls will raise",
              file=sys.stderr)
    if not make_lib and not make_bind:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    obj_dir = os.path.join(OUT_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()

    def run(cmd, what: str) -> None:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)

    def compile_one(src: str) -> str:
        obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
        run([cc, *_flags(extra_flags), "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc for {src}")
        return obj

    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    bind_obj = os.path.join(obj_dir, "prompt_bind.o")
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        if make_bind:
            bound_to = _bound_to()
            bind_cc, bind_ld = _bind_flags()
            bind = ex.submit(run, [cxx, *bind_cc, "-c", os.path.join(CSRC, "prompt_bind.cpp"), "-o", bind_obj],
                             "compiling prompt_bind.cpp")
        if make_lib:  # in place before a failure of the binding is raised
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + f".tmp{os.getpid()}"
            run([cc, *ARCH, "-shared", "-o", tmp, *objs], "link")
            os.replace(tmp, LIB)
        if make_bind:
            bind.result()
            tmp = BIND + f".tmp{os.getpid()}"
            run([cxx, "-o", tmp, bind_obj, *bind_ld], "link of _pkv_prompt.so")
            os.replace(tmp, BIND)
            tmp = BOUND_TO + f".tmp{os.getpid()}"
            with open(tmp, "w") as f:
                f.write(bound_to)
            os.replace(tmp, BOUND_TO)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
