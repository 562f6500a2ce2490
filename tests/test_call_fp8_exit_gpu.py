"""A daemon thread inside a compiled 8-bit call while the interpreter ends: the thread is unwound at
the call's return, and the process ends as it would have."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# in place of the library's entry, one that takes a second (and launches nothing)
SLOW = """
#include <unistd.h>
int slow(void) { usleep(1000000); return 0; }
"""

ENDS = """
import ctypes, sys, threading, time
import torch
import invariant_bi_rmsnorm_gb300 as bi
x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
q, s = bi.quantize_fp8(x)
torch.cuda.synchronize()
slow = ctypes.cast(ctypes.CDLL(sys.argv[1]).slow, ctypes.c_void_p).value
calls = bi._lib.fp8_calls
calls.bind(*[slow] * 6)

class Late:  # goes with the interpreter's last names, and takes longer than the call
    def __del__(self, sleep=time.sleep):
        sleep(3.0)
sys.late = Late()
threading.Thread(target=calls.quantize_fp8, args=(x, q, s), daemon=True).start()
time.sleep(0.2)
print("ending", flush=True)
"""


def test_the_interpreter_ends_during_a_call(tmp_path):
    (tmp_path / "slow.c").write_text(SLOW)
    so = str(tmp_path / "slow.so")
    subprocess.run(["gcc", "-shared", "-fPIC", str(tmp_path / "slow.c"), "-o", so], check=True)
    r = subprocess.run([sys.executable, "-c", ENDS, so], capture_output=True, text=True, timeout=300)
    assert "ending" in r.stdout and r.returncode == 0, (r.returncode, r.stderr[-2000:])
