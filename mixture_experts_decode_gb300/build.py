"""Build libmoedec.so (the C-ABI CUDA library) in-tree for sm_103a, and _block.so
(the compiled binding of the decode block's entry points, linked against it).

Each .cu translation unit is compiled by its own nvcc process (in parallel),
then linked into mixture_experts_decode_gb300/libmoedec.so with the static
CUDA runtime.  A hash of the sources and flags skips up-to-date rebuilds.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoedec.so")
BLOCK = os.path.join(PKG, "_block.so")
BUILD_DIR = os.path.join(ROOT, "_build")
SOURCES = ["api.cu", "gate_up.cu", "down.cu", "grouped.cu", "align.cu", "router.cu", "requant.cu", "decode_fp4.cu",
           "attention.cu", "rope.cu", "norm.cu", "matvec4.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _digest(extra) -> str:
    h = hashlib.sha256()
    files = sorted(os.listdir(CSRC)) + ["../../include/moedec.h"]
    for name in files:
        path = os.path.normpath(os.path.join(CSRC, name))
        if os.path.isfile(path):
            h.update(name.encode())
            with open(path, "rb") as f:
                h.update(f.read())
    h.update(repr((ARCH, NVCC_FLAGS, extra)).encode())
    return h.hexdigest()


def _block_commands():
    """(compile command without -o, its object's link command without -o) of _block.so."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    cxx = os.environ.get("CXX", "g++")
    comp = [cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-isystem{d}" for d in inc], "-c", os.path.join(CSRC, "binding.cpp")]
    link = [cxx, "-shared", "-L" + os.path.join(root, "lib"), "-L" + PKG, "-Wl,-rpath,$ORIGIN"]
    libs = ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-l:libmoedec.so"]
    return comp, link, libs, torch.__version__


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False, extra_flags=(), lib_path: str = LIB) -> str:
    """Compile every CUDA source and link the library (default: the in-tree
    libmoedec.so; extra_flags/lib_path build a variant elsewhere); returns
    the library path."""
    extra = list(extra_flags)
    in_tree = lib_path == LIB
    comp, link, libs, torch_version = _block_commands()
    want = _digest(extra + [torch_version])
    stamp = lib_path + ".src-sha"
    if not force and os.path.exists(lib_path) and os.path.exists(stamp) and (not in_tree or os.path.exists(BLOCK)):
        with open(stamp) as f:
            if f.read().strip() == want:
                return lib_path
    # one object folder per output library (rebuilt in place: the stamp, not
    # the folder, records which sources it holds)
    obj_dir = os.path.join(BUILD_DIR, os.path.basename(lib_path) + ".objs")
    os.makedirs(obj_dir, exist_ok=True)
    nvcc = _nvcc()
    block_obj = os.path.join(obj_dir, "binding.o")

    def compile_one(src):
        if src == "binding.cpp":
            return block_obj, _run([*comp, "-o", block_obj], "g++ for binding.cpp")
        obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
        return obj, _run([nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc for {src}")

    todo = SOURCES + (["binding.cpp"] if in_tree else [])
    with cf.ThreadPoolExecutor(max_workers=len(todo)) as ex:
        results = list(ex.map(compile_one, todo))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = lib_path + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, "-Xlinker", "-soname=libmoedec.so",
          *[o for o, _ in results if o != block_obj]], "link")
    os.replace(tmp, lib_path)
    if in_tree:
        tmp = BLOCK + f".tmp{os.getpid()}"
        _run([*link, "-o", tmp, block_obj, *libs], "link of _block.so")
        os.replace(tmp, BLOCK)
    with open(stamp, "w") as f:
        f.write(want + "\n")
    return lib_path


if __name__ == "__main__":
    flags = [a for a in sys.argv[1:] if a.startswith("-X")]
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, extra_flags=flags))
