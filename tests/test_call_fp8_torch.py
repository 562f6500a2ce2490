"""The compiled calls read torch's own objects by the layout that they were compiled against, so
they are bound to that torch: another's are refused at load and built again (no GPU)."""
import importlib.machinery
import os
import subprocess
import sys

import pytest
import torch

from invariant_bi_rmsnorm_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with_cuda = pytest.mark.skipif(torch.version.cuda is None, reason="a torch without CUDA has no such calls")

OF_ANOTHER_TORCH = """
import sys, types, warnings
import torch
import __graft_entry__
__graft_entry__.build()
for name in [n for n in sys.modules if n.startswith("invariant_bi_rmsnorm_gb300")]:
    del sys.modules[name]
import invariant_bi_rmsnorm_gb300 as bi
calls = types.ModuleType("invariant_bi_rmsnorm_gb300._call_fp8")
BUILT_FOR
def bind(*addresses):
    raise AssertionError("bound")
calls.bind = bind
sys.modules["invariant_bi_rmsnorm_gb300._call_fp8"] = bi._call_fp8 = calls
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    assert bi.abi_version() == 2 and bi._lib.fp8_calls is None
assert [w for w in said if w.category is RuntimeWarning and "torch" in str(w.message)], [str(w.message) for w in said]
print("refused")
"""


@with_cuda
@pytest.mark.parametrize("built_for", ["", "calls.built_for = '1.0.0 abc'", "calls.built_for = torch.__version__ + ' abc'"])
def test_calls_of_another_torch_are_refused(built_for):
    r = subprocess.run([sys.executable, "-c", OF_ANOTHER_TORCH.replace("BUILT_FOR", built_for)], cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "refused" in r.stdout, r.stderr[-2000:]


@with_cuda
def test_they_say_what_they_were_built_for():
    import __graft_entry__
    __graft_entry__.build()
    _lib.load()
    assert _lib.fp8_calls.built_for == _lib.torch_build()
    assert torch.__version__ in _lib.torch_build()
    # a file that only this interpreter's import finds
    assert build.CALLS.endswith("_call_fp8" + importlib.machinery.EXTENSION_SUFFIXES[0])
    assert _lib.fp8_calls.__file__ == build.CALLS


@with_cuda
def test_another_torch_builds_them_again(monkeypatch, tmp_path):
    """And nothing else: the library knows no torch."""
    import __graft_entry__
    __graft_entry__.build()
    monkeypatch.setattr(build, "_compile", lambda *a: pytest.fail("libbi.so is current"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "calls.so"))
    monkeypatch.setattr(build, "CALLS_FOR", str(tmp_path / "calls.txt"))
    monkeypatch.setattr(_lib, "torch_build", lambda: "one")
    ran = []

    def compile_calls(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", compile_calls)
    build.build()
    build.build()
    assert len(ran) == 1 and any('"one"' in a for a in ran[0])
    monkeypatch.setattr(_lib, "torch_build", lambda: "two")
    build.build()
    build.build()
    assert len(ran) == 2 and any('"two"' in a for a in ran[1])
