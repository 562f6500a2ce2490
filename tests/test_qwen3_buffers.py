"""An engine has the step buffers that its own steps use, and no others (no GPU)."""
import pytest
import torch

from invariant_bi_rmsnorm_gb300 import fp8_scales_shape, qwen3

ALL = {"res", "n", "qkv", "q", "attn", "o", "d"}
CFG = qwen3.Qwen3Config(hidden=272, layers=1, ffn=544, heads=2, kv_heads=1, vocab=40, max_pos=64)


@pytest.mark.parametrize("kw,more", [
    (dict(), {"h": (300, 544)}),
    (dict(ops="torch"), {"gu": (300, 1088), "h": (300, 544)}),
    (dict(linear_bits=8), {"n8": (300, 272), "n8s": fp8_scales_shape(300, 272), "attn8": (300, 256),
                           "attn8s": fp8_scales_shape(300, 256), "h8": (300, 544), "h8s": fp8_scales_shape(300, 544)})])
def test_step_buffers(kw, more, monkeypatch):
    monkeypatch.setattr(qwen3, "quantize_fp8", lambda w: (w, None))  # the library's takes CUDA tensors
    w = qwen3.Qwen3Weights(CFG, seed=1, device="cpu")
    eng = qwen3.Engine(w, num_pages=4, max_tokens_per_step=300, device="cpu", **kw)
    assert set(eng.buf) == ALL | set(more)
    for name, shape in more.items():
        assert tuple(eng.buf[name].shape) == shape
        assert eng.buf[name].dtype == (torch.uint8 if name.endswith("s") else torch.float8_e4m3fn if "8" in name else torch.bfloat16)
