"""Build libfa.so in-tree with nvcc for sm_103a, and its compiled binding.

Each .cu file under csrc/ is compiled in parallel to an object file, then all
are linked into ``_lib/libfa.so`` with the CUDA runtime linked statically (so
the library loads next to any PyTorch build).  The driver API is reached
through ``cudaGetDriverEntryPointByVersion``; nothing links libcuda.
``csrc/fa_binding.cpp`` becomes ``_lib/_fa_binding.so``, built against the
headers of the PyTorch that imports it.

    python -m tiled_attention_bwd_gb300.build [--force] [--verbose]
"""
import argparse
import concurrent.futures as cf
import json
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
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libfa.so")
BINDING = os.path.join(OUT_DIR, "_fa_binding.so")
FLAGS = os.path.join(OUT_DIR, "build_flags.json")
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_serve_api.cu",
           "fa_rope.cu", "fa_cache4.cu", "fa_cache4_attn.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required")
    return cand


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
             if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    files.append(os.path.join(INCLUDE, "fa.h"))
    return files


def _stale():
    if not all(os.path.exists(f) for f in (LIB, BINDING, FLAGS)):
        return True
    with open(FLAGS) as f:
        if json.load(f).get("torch") != torch.__version__:
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(f) > t for f in _inputs())


def _build_binding():
    """g++ of the binding (result as subprocess.run's)."""
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    tmp = BINDING + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", INCLUDE, "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           os.path.join(CSRC, "fa_binding.cpp"), "-o", tmp, "-L", lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode == 0:
        os.replace(tmp, BINDING)
    return r


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libfa.so if missing or older than its sources."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_binding)
        results = list(ex.map(compile_one, SOURCES))
        binding = binding.result()
    if binding.returncode != 0:
        sys.stderr.write(binding.stdout + binding.stderr)
        raise RuntimeError("g++ failed on fa_binding.cpp")
    objs = []
    for src, obj, r in results:
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s" % src)
        objs.append(obj)
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of libfa.so failed")
    os.replace(tmp, LIB)
    # The target architecture as built, for the test suite to check without
    # opening the binary.
    with open(FLAGS, "w") as f:
        json.dump({"compile": common, "torch": torch.__version__,
                   "link": ARCH + ["-shared", "-cudart", "static"]}, f,
                  indent=1)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
