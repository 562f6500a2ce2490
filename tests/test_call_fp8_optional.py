"""The compiled calls of the 8-bit path are an accelerator of the host's part: without them the
library loads, and every call goes its way through Python."""
import os
import subprocess
import sys

import pytest
import torch

from invariant_bi_rmsnorm_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, *args):
    return subprocess.run([sys.executable, "-c", code, *args], cwd=ROOT, capture_output=True, text=True, timeout=600)


# an entry of None makes the import of that module fail, as a missing file does
WITHOUT = """
import sys, warnings
import torch
import __graft_entry__
__graft_entry__.build()
for name in [n for n in sys.modules if n.startswith("invariant_bi_rmsnorm_gb300")]:
    del sys.modules[name]
sys.modules["invariant_bi_rmsnorm_gb300._call_fp8"] = None
import invariant_bi_rmsnorm_gb300 as bi
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    assert bi.abi_version() == 2
    assert bi.status_string(0) == "BI_OK" and bi._lib.fp8_calls is None
said = [str(w.message) for w in said if w.category is RuntimeWarning]
assert len(said) == (torch.version.cuda is not None) and all("_call_fp8" in s for s in said), said
x = torch.zeros(3, 64, dtype=torch.bfloat16)
q, s = x.to(torch.float8_e4m3fn), torch.zeros(bi.fp8_scales_shape(3, 64), dtype=torch.uint8)
for call in (lambda: bi.rmsnorm(x, x[0]), lambda: bi.quantize_fp8(x, out=q, scales=s), lambda: bi.gemm_fp8(q, s, q, s, out=x)):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("not refused")
print("loaded")
"""


def test_the_library_loads_without_them():
    r = run(WITHOUT)
    assert r.returncode == 0 and "loaded" in r.stdout, r.stderr[-2000:]


# a tree of its own, whose compiler for the calls fails: libbi.so is made all the same, and the
# next build tries only what is missing
BUILDS = """
import os, shutil, sys
root = sys.argv[1]
for d in ("invariant_bi_rmsnorm_gb300", "include"):
    shutil.copytree(d, os.path.join(root, d), ignore=shutil.ignore_patterns("*.so", "_build", "__pycache__"))
os.chdir(root)
sys.path.insert(0, root)
from invariant_bi_rmsnorm_gb300 import build
compiled = []
build._compile = lambda src, extra: compiled.append(src) or src
def link(cmd):
    open(cmd[cmd.index("-o") + 1], "w").close()
build._link = link
os.environ["CXX"] = "false"
assert build.build() == build.LIB and os.path.exists(build.LIB) and sorted(compiled) == sorted(build.SOURCES)
made = os.path.getmtime(build.LIB)
compiled.clear()
assert build.build() == build.LIB and not compiled and os.path.getmtime(build.LIB) == made
print("built")
"""


def test_the_library_is_built_where_they_cannot_be(tmp_path):
    r = run(BUILDS, str(tmp_path))
    assert r.returncode == 0 and "built" in r.stdout, r.stderr[-2000:]
    assert "call_fp8.cpp" in r.stderr


@pytest.mark.skipif(torch.version.cuda is None, reason="a torch without CUDA has no such calls")
def test_a_current_library_needs_no_toolkit(monkeypatch, tmp_path, capfd):
    import __graft_entry__
    from invariant_bi_rmsnorm_gb300 import build
    __graft_entry__.build()

    def nvcc():
        raise RuntimeError("nvcc not found")
    monkeypatch.setattr(build, "nvcc", nvcc)
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "calls.so"))
    assert build.build() == build.LIB and "nvcc not found" in capfd.readouterr().err


def test_what_is_current_is_left_alone(monkeypatch):
    """A tree that cannot be written to is no trouble then."""
    import __graft_entry__
    from invariant_bi_rmsnorm_gb300 import build
    __graft_entry__.build()
    monkeypatch.setattr(build.os, "makedirs", lambda *a, **k: pytest.fail("nothing is to be made"))
    monkeypatch.setattr(build.tempfile, "mkstemp", lambda *a, **k: pytest.fail("nothing is to be made"))
    assert build.build() == build.LIB


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["quantize_fp8", "fp8_read", "rmsnorm_fp8", "add_rmsnorm_fp8", "gemm_fp8", "gemm_fp8_swiglu"])
def test_the_same_bytes_without_them(name, monkeypatch):
    from tests.test_fp8_calls_gpu import args_of
    _lib.load()
    assert _lib.fp8_calls is not None
    got = []
    for calls in (_lib.fp8_calls, None):
        monkeypatch.setattr(_lib, "fp8_calls", calls)
        f, a, outs = args_of(name)
        f(*a, **outs)
        got.append({k: v.view(torch.uint8) for k, v in outs.items()})
    assert all(torch.equal(got[0][k], got[1][k]) for k in got[0])
