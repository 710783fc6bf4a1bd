"""Build libes.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit under ``csrc/`` is compiled in parallel to an
object file, then linked into ``_build/libes.so`` with the static CUDA runtime
(the driver's ``cuTensorMapEncodeTiled`` and module API are fetched at run
time, so the library loads on machines without a GPU driver as well) and
NVRTC, which compiles body programs at run time.  The headers NVRTC needs are
embedded into the library as text (``write_jit_headers``).  Beside it
``_build/es_torch.so``, a Python module that marshals the sequence operators'
tensors, is compiled against the installed PyTorch and again when that changes;
without PyTorch there is libes.so alone, and what goes wrong with the module
leaves libes.so built.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libes.so")
# the tensor marshalling of the sequence operators (a Python module over libes.so and PyTorch)
TORCH_SRC = os.path.join(CSRC, "torch", "es_torch.cpp")
TORCH_LIB = os.path.join(BUILD, "es_torch.so")
TORCH_STAMP = TORCH_LIB + ".built_for"

GEN = os.path.join(BUILD, "gen")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC,
                     "-I", GEN]

# Headers compiled at run time with body programs (NVRTC): embedded in the
# library as text, in this order.
JIT_HEADERS = ["es_ptx.cuh", "skel_common.cuh", "skel_generic.cuh", "skel_generic_bwd.cuh", "skel_lane.cuh",
               "skel_lane_bwd.cuh", "skel_time.cuh", "skel_time_bwd.cuh", "skel_vec.cuh", "skel_vec_bwd.cuh"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libes.so")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def cuda_home() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))


def write_jit_headers() -> str:
    """Write ``gen/es_jit_headers.inc``: the run-time compiled headers as C++
    raw string literals (names and texts for nvrtcCreateProgram)."""
    os.makedirs(GEN, exist_ok=True)
    names, texts = [], []
    for h in JIT_HEADERS:
        path = os.path.join(CSRC, h)
        if not os.path.exists(path):
            continue
        text = open(path).read()
        if ")ES_JIT\"" in text:
            raise RuntimeError("%s contains the raw-string delimiter" % h)
        names.append(h)
        texts.append(text)
    lines = ["// generated by build.py from csrc/: headers for run-time compilation", "#pragma once",
             "static const int kJitHeaderCount = %d;" % len(names),
             "static const char* const kJitHeaderNames[] = {%s};" % ", ".join('"%s"' % n for n in names),
             "static const char* const kJitHeaderSources[] = {"]
    for t in texts:
        lines.append('R"ES_JIT(' + t + ')ES_JIT",')
    lines.append("};")
    out = os.path.join(GEN, "es_jit_headers.inc")
    body = "\n".join(lines) + "\n"
    if not os.path.exists(out) or open(out).read() != body:
        with open(out, "w") as f:
            f.write(body)
    return out


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(INCLUDE, "es.h"), os.path.abspath(__file__)]


def _newer(product: str, deps) -> bool:
    return os.path.exists(product) and all(os.path.getmtime(p) <= os.path.getmtime(product) for p in deps)


def _installed_torch():
    """What es_torch.so is built against: where PyTorch lies and its version (found without importing
    it, which takes seconds), Python's ABI; None without PyTorch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    home = os.path.dirname(spec.origin)
    version = os.path.join(home, "version.py")
    text = open(version).read() if os.path.exists(version) else ""
    return "%s\n%s\n%s" % (home, sys.implementation.cache_tag, text)


def _lib_up_to_date() -> bool:
    return _newer(LIB, _deps())


def _torch_up_to_date() -> bool:
    installed = _installed_torch()
    if installed is None:
        return True
    if not _newer(TORCH_LIB, [TORCH_SRC, os.path.join(INCLUDE, "es.h"), os.path.abspath(__file__)]) or not os.path.exists(TORCH_STAMP):
        return False
    with open(TORCH_STAMP) as f:
        return f.read() == installed


def up_to_date() -> bool:
    return _lib_up_to_date() and _torch_up_to_date()


def _compile_torch(obj: str):
    """g++ on es_torch.cpp against the installed PyTorch's headers."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = ["g++", "-O1", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", INCLUDE, "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda_home(), "include"),
           "-c", TORCH_SRC, "-o", obj]
    return TORCH_SRC, subprocess.run(cmd, capture_output=True, text=True)


def _link_torch(obj: str):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_LIB + ".%d.tmp" % os.getpid()
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-les", "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
                        "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking es_torch.so failed")
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_STAMP, "w") as f:
        f.write(_installed_torch() or "")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    lib, module = force or not _lib_up_to_date(), (force and _installed_torch() is not None) or not _torch_up_to_date()
    if not (lib or module):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    write_jit_headers()
    cc = nvcc()
    srcs = _sources() if lib else []
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [cc] + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r

    torch_obj = os.path.join(BUILD, "es_torch.torch.o")
    # the longest compilations first, so that none of them is left alone at the end
    order = sorted(zip(srcs, objs), key=lambda p: -os.path.getsize(p[0]))
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        bound = ex.submit(_compile_torch, torch_obj) if module else None
        results = list(ex.map(compile_one, order))
    failed = [(s, r) for s, r in results if r.returncode != 0]
    for s, r in results:
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
    if failed:
        raise RuntimeError("compilation failed for: " + ", ".join(os.path.basename(s) for s, _ in failed))
    if lib:
        tmp = LIB + ".%d.tmp" % os.getpid()
        lib64 = os.path.join(cuda_home(), "lib64")
        link = ["-L", lib64, "-lnvrtc", "-Xlinker", "-rpath," + lib64]
        r = subprocess.run([cc] + ARCH + ["-shared", "-o", tmp] + objs + link, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("linking libes.so failed")
        os.replace(tmp, LIB)
    if module:
        src, r = bound.result()
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("compilation failed for: " + os.path.basename(src))
        _link_torch(torch_obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
