"""Build libbi.so (the CUDA kernels behind the C ABI in include/bi.h) in-tree.

Every translation unit is compiled for sm_103a only, in parallel, then linked
into ``invariant_bi_rmsnorm_gb300/libbi.so``.  nvcc cross-compiles without a
GPU, so this also runs on a machine with no device.  The library links the
CUDA runtime statically and resolves the one driver call
it needs (cuTensorMapEncodeTiled) at run time, so it does not link libcuda.

Beside it, ``_call_fp8``: the 8-bit linear path's calls from Python, compiled by
the host compiler against the torch that is installed, and again for another torch
(an accessor of torch's tensors is compiled in, and with it their layout).  Where that cannot be
done the build says so and goes on: the library does not need them.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

from . import _lib

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbi.so")
CALLS = os.path.join(PKG, "_call_fp8" + sysconfig.get_config_var("EXT_SUFFIX"))
OBJ_DIR = os.path.join(PKG, "_build")
CALLS_FOR = os.path.join(OBJ_DIR, "call_fp8.torch")  # the torch that CALLS was built for

SOURCES = ["api.cu", "rmsnorm.cu", "gemm.cu", "decode_attention.cu", "prefill_attention.cu",
           "decoder_ops.cu", "logprobs.cu", "kv4_cache.cu", "kv4_attention.cu",
           "logprobs_top.cu", "fp8_quant.cu", "gemm_fp8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths.append(os.path.join(INCLUDE, "bi.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _with_calls() -> bool:
    import torch
    return torch.version.cuda is not None  # else there are no tensors to call with


def _calls_command(built_for: str, out: str) -> list[str]:
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBUILT_FOR="{built_for}"',
            *(f"-isystem{d}" for d in (os.path.join(home, "include"), os.path.join(cuda, "include"),
                                       sysconfig.get_paths()["include"])),
            "-I" + INCLUDE, os.path.join(CSRC, "call_fp8.cpp"), "-o", out,
            "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _build_calls() -> None:
    built_for = _lib.torch_build()
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=PKG)
    os.close(fd)
    try:
        r = subprocess.run(_calls_command(built_for, tmp), capture_output=True, text=True)
        why = f"{r.stdout}\n{r.stderr}" if r.returncode else None
    except (OSError, RuntimeError) as e:  # no such compiler, or no toolkit
        why = str(e)
    if why is None:
        os.replace(tmp, CALLS)
        with open(CALLS_FOR, "w") as f:
            f.write(built_for)
        return
    os.unlink(tmp)
    if os.path.exists(CALLS):  # of other sources, or for another torch
        os.unlink(CALLS)
    sys.stderr.write(f"call_fp8.cpp did not build, and the 8-bit calls go through Python:\n{why}\n")


def _built_for() -> str | None:
    try:
        with open(CALLS_FOR) as f:
            return f.read()
    except OSError:
        return None


def _link(cmd: list[str]) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")


def _build_lib(ex: ThreadPoolExecutor, extra: list[str]) -> None:
    objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=PKG)
    os.close(fd)
    try:
        _link([nvcc(), *ARCH, "-shared", *objs, "-o", tmp, "-cudart", "static"])
    except RuntimeError:
        os.unlink(tmp)
        raise
    os.replace(tmp, LIB)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libbi.so and _call_fp8, each unless it is newer than every source (and
    the second was built for this torch)."""
    newest = _deps_mtime()

    def current(f):
        return not force and os.path.exists(f) and os.path.getmtime(f) >= newest

    lib = not current(LIB)
    calls = _with_calls() and not (current(CALLS) and _built_for() == _lib.torch_build())
    if not lib and not calls:
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        made = ex.submit(_build_calls) if calls else None
        if lib:
            _build_lib(ex, ["-Xptxas", "-v"] if verbose_ptxas else [])
        if made is not None:
            made.result()
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
