"""The decoder on 8-bit weights and activations.

Bit for bit: the engine's logits are those of the layer's calls made one after the other
by hand over a whole prompt, and a request's logits are the same alone, batched, with
prompts cut anywhere, through captured graphs, and over either cache's own decode and
prefill forms.  The calls themselves are compared with the fp64 oracle in
tests/test_fp8_gpu.py."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import qwen3
from tests._util import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def two_layer():
    cfg = qwen3.Qwen3Config(layers=2, max_pos=1024)
    return cfg, qwen3.Qwen3Weights(cfg, seed=2000)


def by_hand(cfg, w, tokens):
    """Logits of a whole prompt, every call of a layer in its place."""
    T, pages = len(tokens), -(-len(tokens) // 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    pos = torch.arange(T, **i32)
    table, lens = torch.arange(pages, **i32)[None], torch.tensor([T], **i32)
    rope = qwen3.rope_table(cfg.max_pos, cfg.rope_theta, device="cuda")
    res, d = w.embed[torch.tensor(tokens, device="cuda")].clone(), None
    for L in w.layers:
        n = bi.rmsnorm_fp8(res, L["in_norm"], cfg.eps) if d is None else bi.add_rmsnorm_fp8(d, res, L["in_norm"], cfg.eps)
        kc, vc = (torch.zeros(pages, cfg.kv_heads, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = bi.qk_norm_rope_append(bi.gemm_fp8(*n, *bi.quantize_fp8(L["qkv"])), cfg.heads, cfg.kv_heads, pos, pos, rope,
                                   L["q_norm"], L["k_norm"], kc, vc, cfg.eps)
        a = bi.prefill_attention(q, kc, vc, table, lens, torch.tensor([0, T], **i32), T, T)
        o = bi.gemm_fp8(*bi.quantize_fp8(a.view(T, -1)), *bi.quantize_fp8(L["o"]))
        n = bi.add_rmsnorm_fp8(o, res, L["post_norm"], cfg.eps)
        h = bi.gemm_fp8_swiglu(*n, *bi.quantize_fp8(bi.interleave_gate_up(L["gate_up"])))
        d = bi.gemm_fp8(*h, *bi.quantize_fp8(L["down"]))
    return bi.gemm(bi.add_rmsnorm(d, res, w.final_norm, cfg.eps), w.lm_head)


def test_logits_are_those_of_the_calls_by_hand(two_layer):
    cfg, w = two_layer
    g = torch.Generator().manual_seed(5)
    prompt, forced = (torch.randint(0, cfg.vocab, (n,), generator=g).tolist() for n in (45, 4))
    want = by_hand(cfg, w, prompt + forced[:3])[44:]
    for budget in (17, 512):
        eng = qwen3.Engine(w, num_pages=8, max_tokens_per_step=budget, linear_bits=8)
        logs = eng.generate([qwen3.Sequence(sid=0, prompt=prompt, max_new=4, forced=forced)], record={0})
        for a, b in zip(logs[0], want):
            assert np.array_equal(bits(a), bits(b))
    bi.get_device_error()


@pytest.mark.parametrize("kv_bits", [16, 4])
def test_bits_alone_batched_and_graphed(two_layer, kv_bits):
    cfg, w = two_layer
    track = {0, 3, 9}
    runs = []
    for graphs, budget in ((False, 130), (True, 300)):
        reqs = qwen3.random_requests(10, cfg.vocab, 1, 150, max_new=6, seed=21)
        eng = qwen3.Engine(w, num_pages=10 * 10 + 1, max_tokens_per_step=budget, cuda_graphs=graphs, kv_bits=kv_bits,
                           linear_bits=8)
        runs.append((reqs, eng.generate(reqs, record=track, top=3), eng))
    (r0, l0, _), (r1, l1, e1) = runs
    assert e1.graph_steps > 0
    for sid in track:
        assert r0[sid].generated == r1[sid].generated
        alone = qwen3.Sequence(sid=sid, prompt=list(r0[sid].prompt), max_new=6)
        la = qwen3.Engine(w, num_pages=16, max_tokens_per_step=64, kv_bits=kv_bits, linear_bits=8).generate([alone], record={sid})
        assert alone.generated == r0[sid].generated
        for a, b, c in zip(l0[sid], l1[sid], la[sid]):
            assert np.array_equal(bits(a), bits(b)) and np.array_equal(bits(a), bits(c))
    bi.get_device_error()


def test_engine_refuses_other_widths(two_layer):
    for kw in (dict(linear_bits=4), dict(linear_bits=8, ops="torch")):
        with pytest.raises(ValueError, match="linear_bits"):
            qwen3.Engine(two_layer[1], num_pages=4, **kw)
