"""The binding without a device (no GPU): what it looks up when it is imported,
and what a call says when there is no device to make it on."""
import os
import subprocess
import sys

import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# a torch without CUDA has no _cuda_getCurrentRawStream
WITHOUT_CUDA = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import invariant_bi_rmsnorm_gb300 as bi
x = torch.zeros(2, 128, dtype=torch.bfloat16)
for call in (lambda: bi.rmsnorm(x, x[0]), lambda: bi.logprobs_top(x, None, 1)):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("not refused")
torch.cuda.current_stream = lambda device: type("Stream", (), {"cuda_stream": 1000 + device})()
torch.cuda.current_device = lambda: 5
assert bi._stream(None) == 1005
"""


def test_imports_and_refuses_on_a_torch_without_cuda():
    r = subprocess.run([sys.executable, "-c", WITHOUT_CUDA], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


def test_no_device_is_reported_in_torchs_words(monkeypatch):
    def no_device():
        raise RuntimeError("Found no NVIDIA driver on your system.")
    monkeypatch.setattr(torch.cuda, "current_device", no_device)
    with pytest.raises(RuntimeError, match="Found no NVIDIA driver"):
        bi._stream(None)
    # a tensor that is there all the same is no CUDA tensor
    with pytest.raises(ValueError, match="CUDA tensor"):
        bi.logprobs_top(torch.zeros(2, 8, dtype=torch.bfloat16), None, 1)
