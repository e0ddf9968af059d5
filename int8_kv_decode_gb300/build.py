"""Build libkattn.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel; the shared library links the CUDA
runtime statically so it does not depend on which libcudart the process
loaded first.  Object files go to ``_build/`` next to this file.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkattn.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC,-ffp-contract=off",
          "-I", INCLUDE, "-I", CSRC]

# Per-file extra flags.  The exact-mode scan and the host constant generator
# must not contract multiply-add pairs.
SOURCES = {
    "kattn_api.cu": [],
    "quantize.cu": [],
    "qk_debug.cu": [],
    "decode_fast.cu": [],
    "decode_fast_paged.cu": [],
    "decode_tc.cu": [],
    "decode_noalloc.cu": [],
    "decode_exact.cu": ["--fmad=false"],
    "expf_constants.cu": ["--fmad=false"],
    "hash_rows.cu": [],
    "decode_diff.cu": [],
    "norm_quant.cu": [],
    "pages.cu": [],
    "rope.cu": [],
    "blocks.cu": [],
    "decode_blocks.cu": [],
}


def nvcc_path() -> str:
    env = os.environ.get("NVCC")
    if env:
        return env
    found = shutil.which("nvcc")
    if found:
        return found
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _headers():
    hs = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    hs += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}")
    if verbose and r.stdout.strip():
        print(r.stdout, flush=True)
    return r.stdout


# The checks and calls of the block-scaled operators in one step from Python (bind.cpp), a
# module against the torch and Python that run this; the stamp names them.  The library needs
# neither: it is built and linked without torch, and api.py calls it without this module.
BIND = os.path.join(PKG, "_bind.so")
_STAMP = os.path.join(BUILD, "bind.stamp")


def _has_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def _bind_stamp() -> str:
    import torch
    return f"{sys.version} {torch.__version__} {torch.__file__}"


def _bind_outdated() -> bool:
    return _stale(BIND, [os.path.join(CSRC, "bind.cpp"), os.path.join(INCLUDE, "kattn.h"), __file__])


def _bind_stale() -> bool:
    if _bind_outdated():
        return True
    try:
        with open(_STAMP, encoding="utf-8") as f:
            return f.read() != _bind_stamp()
    except OSError:
        return True


def _build_bind(verbose: bool) -> None:
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    lib = os.path.join(base, "lib")
    tmp = BIND + ".tmp"
    cmd = ["g++", "-shared", "-O2", "-std=c++17", "-fPIC", os.path.join(CSRC, "bind.cpp"), "-o", tmp,
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), f"-DKATTN_TORCH_VERSION=\"{torch.__version__}\"",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
           "-lc10"]
    try:
        _run(cmd, verbose)
    except RuntimeError:
        if os.path.exists(BIND):
            os.remove(BIND)                       # (of an earlier source)
        raise
    os.replace(tmp, BIND)
    with open(_STAMP, "w", encoding="utf-8") as f:
        f.write(_bind_stamp())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link libkattn.so and, where there is torch, the binding module; returns
    the library's path.  Rebuilds what is stale."""
    nvcc = nvcc_path()
    os.makedirs(BUILD, exist_ok=True)
    headers = _headers()
    jobs = []
    objs = []
    for src, extra in SOURCES.items():
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, __file__] + headers):
            cmd = [nvcc, "-c", s, "-o", o] + ARCH + COMMON + extra
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)
    outputs = []
    binding = None
    bind = _has_torch() and (force or _bind_stale())
    if not bind and os.path.exists(BIND) and _bind_outdated():
        os.remove(BIND)                           # (its calls may not be the library's any more)
    if jobs or bind:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
            binding = ex.submit(_build_bind, verbose) if bind else None
            outputs = list(ex.map(lambda c: _run(c, verbose), jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        _run([nvcc, "-shared", "-o", tmp] + ARCH + objs + ["-cudart", "static"], verbose)
        os.replace(tmp, LIB)
    if binding:
        binding.result()                          # (a failure of its own, once the library is there)
    if ptxas_verbose:
        for out in outputs:
            print(out)
    return LIB


# Test-only build: exact mode's hand-off waits give up after this many polls
# (0: at once), so that a test can check the give-up path -- NaN rows and the
# KATTN_DEVERR_TIMEOUT bit -- with no wait that could block.  Never loaded by
# the package; only tests/test_gpu_exact_timeout.py loads it.
TIMEOUT_VARIANT_LIB = os.path.join(BUILD, "libkattn_exact_spin0.so")


def build_exact_timeout_variant(verbose: bool = False) -> str:
    """libkattn.so with decode_exact.cu built with KATTN_EXACT_SPIN_LIMIT = 0
    (every other object shared with the library); returns its path."""
    build(verbose=verbose)
    nvcc = nvcc_path()
    src = os.path.join(CSRC, "decode_exact.cu")
    obj = os.path.join(BUILD, "decode_exact_spin0.o")
    deps = [src, __file__] + _headers()
    if _stale(obj, deps):
        _run([nvcc, "-c", src, "-o", obj] + ARCH + COMMON + SOURCES["decode_exact.cu"]
             + ["-DKATTN_EXACT_SPIN_LIMIT=0u"], verbose)
    objs = [os.path.join(BUILD, f.replace(".cu", ".o")) for f in SOURCES if f != "decode_exact.cu"]
    if _stale(TIMEOUT_VARIANT_LIB, objs + [obj]):
        tmp = TIMEOUT_VARIANT_LIB + ".tmp"
        _run([nvcc, "-shared", "-o", tmp] + ARCH + objs + [obj, "-cudart", "static"], verbose)
        os.replace(tmp, TIMEOUT_VARIANT_LIB)
    return TIMEOUT_VARIANT_LIB


# Test-only builds: a warp of decode_diff.cu finds no further copy ready after
# `limit` stages, for the maps in the bit mask `maps`, so that a test can check how
# the two warps of a pair part, with no wait that could block.  Never loaded by the
# package; only tests/test_gpu_diff_timeout.py loads them.
def build_diff_timeout_variant(limit: int, maps: int, verbose: bool = False) -> str:
    """libkattn.so with decode_diff.cu built to run out of copies; returns its path."""
    build(verbose=verbose)
    nvcc = nvcc_path()
    src = os.path.join(CSRC, "decode_diff.cu")
    obj = os.path.join(BUILD, f"decode_diff_limit{limit}_maps{maps}.o")
    lib = os.path.join(BUILD, f"libkattn_diff_limit{limit}_maps{maps}.so")
    if _stale(obj, [src, __file__] + _headers()):
        _run([nvcc, "-c", src, "-o", obj] + ARCH + COMMON + SOURCES["decode_diff.cu"]
             + [f"-DKATTN_DIFF_STAGE_LIMIT={limit}", f"-DKATTN_DIFF_STAGE_MAPS={maps}"], verbose)
    objs = [os.path.join(BUILD, f.replace(".cu", ".o")) for f in SOURCES if f != "decode_diff.cu"]
    if _stale(lib, objs + [obj]):
        tmp = lib + ".tmp"
        _run([nvcc, "-shared", "-o", tmp] + ARCH + objs + [obj, "-cudart", "static"], verbose)
        os.replace(tmp, lib)
    return lib


# Likewise for decode_blocks.cu: the warps in the bit mask `warps` of a block of four find no
# further copy ready after `limit` stages.  Only tests/test_gpu_blocks_timeout.py loads them.
def build_blocks_timeout_variant(limit: int, warps: int, verbose: bool = False) -> str:
    """libkattn.so with decode_blocks.cu built to run out of copies; returns its path."""
    build(verbose=verbose)
    nvcc = nvcc_path()
    src = os.path.join(CSRC, "decode_blocks.cu")
    obj = os.path.join(BUILD, f"decode_blocks_limit{limit}_warps{warps}.o")
    lib = os.path.join(BUILD, f"libkattn_blocks_limit{limit}_warps{warps}.so")
    if _stale(obj, [src, __file__] + _headers()):
        _run([nvcc, "-c", src, "-o", obj] + ARCH + COMMON + SOURCES["decode_blocks.cu"]
             + [f"-DKATTN_BLOCKS_STAGE_LIMIT={limit}", f"-DKATTN_BLOCKS_STAGE_WARPS={warps}"], verbose)
    objs = [os.path.join(BUILD, f.replace(".cu", ".o")) for f in SOURCES if f != "decode_blocks.cu"]
    if _stale(lib, objs + [obj]):
        tmp = lib + ".tmp"
        _run([nvcc, "-shared", "-o", tmp] + ARCH + objs + [obj, "-cudart", "static"], verbose)
        os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
    print(LIB)
