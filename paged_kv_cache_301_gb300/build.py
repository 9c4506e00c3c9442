"""Compile libpagedattn.so in-tree for GB300 (sm_103a).

Each translation unit is compiled in parallel with nvcc into _build/, then
linked into paged_kv_cache_301_gb300/libpagedattn.so; the Python binding of some
calls (_binding.so, host code against PyTorch's headers) is linked to it.  A stamp
records the host machine and the Python and PyTorch versions, so that what was built
for others is rebuilt.
"""
from __future__ import annotations

import concurrent.futures
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedattn.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "pa_binding.cpp")
STAMP = os.path.join(BUILD, "machine.txt")

SOURCES = [
    "pa_api.cu",
    "pa_cache.cu",
    "pa_decode_simt.cu",
    "pa_block_manager.cpp",
    "pa_allocsim.cpp",
    "pa_decode_noalloc.cu",
    "pa_decode_tc.cu",
    "pa_decode_tcg.cu", "pa_blocks.cu", "pa_prefill_tc.cu", "pa_prefill_simt.cu",
    "pa_stream.cu",
    "pa_rope.cu", "pa_decode_q8.cu", "pa_expand_q8.cu",
]
HEADERS = [
    os.path.join(ROOT, "include", "pagedattn.h"),
    os.path.join(CSRC, "pa_common.cuh"),
    os.path.join(CSRC, "pa_internal.h"),
]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"] + ARCH


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedattn")
    return cand


def _built_for() -> str:
    import torch
    return f"{platform.machine()} python {platform.python_version()} torch {torch.__version__}"


def _stale() -> bool:
    if not all(os.path.exists(p) for p in (LIB, BINDING, STAMP)):
        return True
    with open(STAMP) as f:
        if f.read().strip() != _built_for():
            return True
    lib_t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS + [BINDING_SOURCE]
    deps += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return any(os.path.getmtime(d) > lib_t for d in deps)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), "-c", os.path.join(CSRC, src), "-o", obj] + NVCC_FLAGS
    if verbose and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        sys.stderr.write(res.stdout + res.stderr)
    return obj


def _compile_binding() -> str:
    """The host-only object of the Python binding."""
    import torch
    obj = os.path.join(BUILD, "pa_binding.o")
    headers = os.path.join(torch.__path__[0], "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [headers, os.path.join(headers, "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-c", BINDING_SOURCE, "-o", obj, "-O2", "-std=c++17", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    res = subprocess.run(cmd + [x for i in includes for x in ("-isystem", i)],
                         capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on pa_binding.cpp:\n{res.stdout}\n{res.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:" + os.path.basename(LIB),
           "-Wl,-rpath,$ORIGIN"]
    cmd += ["-L" + os.path.join(torch.__path__[0], "lib"), "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build (if needed) and return the path of libpagedattn.so."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding.result())
    with open(STAMP, "w") as f:
        f.write(_built_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
