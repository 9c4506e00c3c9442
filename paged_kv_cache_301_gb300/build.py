"""Compile libpagedattn.so in-tree for GB300 (sm_103a).

Each translation unit is compiled in parallel with nvcc into _build/, then
linked into paged_kv_cache_301_gb300/libpagedattn.so, which is all that users of the C ABI
need; a stamp records the host machine, so that a library built on another architecture
is rebuilt.  The Python binding of some calls (_binding.so) is host code against Python's
and PyTorch's headers, linked to the library, with a stamp of their versions.  Where it
cannot be built the library is made all the same.
"""
from __future__ import annotations

import concurrent.futures
import os
import platform
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedattn.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "pa_binding.cpp")
STAMP = os.path.join(BUILD, "machine.txt")
BINDING_STAMP = os.path.join(BUILD, "binding.txt")

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
    "pa_latent_cache.cu", "pa_latent_decode.cu", "pa_latent_prefill.cu", "pa_decode_tree.cu",
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


def _stale(target: str, stamp: str, built_for: str, deps: list) -> bool:
    if not os.path.exists(target) or not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        if f.read().strip() != built_for:
            return True
    made = os.path.getmtime(target)
    return any(os.path.getmtime(d) > made for d in deps)


def _library_stale() -> bool:
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    deps += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return _stale(LIB, STAMP, platform.machine(), deps)


def _binding_stale() -> bool:
    return _stale(BINDING, BINDING_STAMP, _built_for(), [BINDING_SOURCE] + HEADERS)


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


def _build_library(verbose: bool) -> None:
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    with open(STAMP, "w") as f:
        f.write(platform.machine())


def _compile_stale_binding(force: bool):
    """The binding's object where it has to be linked anew, else None."""
    return _compile_binding() if force or _binding_stale() else None


def build(force: bool = False, verbose: bool = False, need_binding: bool = False) -> str:
    """Build (if needed) and return the path of libpagedattn.so.  Without a binding there is a
    warning, or with need_binding an error, once the library is made."""
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_stale_binding, force)
        if force or _library_stale():
            _build_library(verbose)
    try:
        obj = binding.result()
        if obj:
            _link_binding(obj)
            with open(BINDING_STAMP, "w") as f:
                f.write(_built_for())
    except Exception as e:                   # a tool or a header that is not there
        for p in (BINDING, BINDING_STAMP):   # nor one that was built for others
            if os.path.exists(p):
                os.remove(p)
        if need_binding:
            raise
        warnings.warn(f"libpagedattn.so is built, its Python binding is not (pa_rope_append and "
                      f"the 8-bit cache's calls need it): {e}", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
