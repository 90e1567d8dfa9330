"""In-tree build of libsba.so for sm_103a with nvcc (no cmake, no torch extension).

Each CUDA translation unit is compiled in parallel, then linked into
``selected_block_attention_gb300/_lib/libsba.so``; beside it the Python module of the
calls bound in C++ (``csrc/binding.cpp``, g++ against torch's headers) becomes
``_lib/_paged.so``.  A rebuild is skipped when both are newer than every source and header
and the module was built for this Python and torch.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libsba.so")
MODULE_PATH = os.path.join(LIB_DIR, "_paged.so")
MODULE_STAMP = os.path.join(BUILD_DIR, "_paged.for")  # the Python and torch it was built against

SOURCES = ["api.cu", "sparse_mask.cu", "nsa_select.cu", "nsa_backward.cu", "blocksparse_attn.cu",
           "blocksparse_backward.cu", "rotary.cu", "ragged_decode.cu", "paged_append.cu", "paged_attention.cu", "paged_chunk.cu",
           "paged_select.cu", "probe.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsba")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "sba.h"))
    files.append(os.path.abspath(__file__))
    return files


def _module_target():
    return f"{sys.version.split()[0]} torch {torch.__version__}"


def _module_command(obj):
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    return [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[x for i in inc for x in ("-isystem", i)], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]


def up_to_date():
    if not os.path.exists(LIB_PATH) or not os.path.exists(MODULE_PATH) or not os.path.exists(MODULE_STAMP):
        return False
    with open(MODULE_STAMP) as f:
        if f.read() != _module_target():
            return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(MODULE_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every kernel for sm_103a, link libsba.so and the Python module; returns the
    library's path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, *NVCC_FLAGS, *ARCH, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    module_obj = os.path.join(BUILD_DIR, "binding.o")
    procs.append(("binding.cpp", subprocess.Popen(_module_command(module_obj), stdout=subprocess.PIPE,
                                                  stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append(f"--- {src} ---\n{text}")
        elif verbose and text:
            print(text, file=sys.stderr)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    tmp = LIB_PATH + ".tmp"
    link = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB_PATH)
    tmp = MODULE_PATH + ".tmp"
    link = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, module_obj, "-L", LIB_DIR, "-l:libsba.so",
            "-Wl,-rpath,$ORIGIN", "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, MODULE_PATH)
    with open(MODULE_STAMP, "w") as f:
        f.write(_module_target())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
