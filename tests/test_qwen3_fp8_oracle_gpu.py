"""The 8-bit decoder layer against its definition in 64 bits, stage by stage: what each buffer of a step
holds is compared with what the oracle makes of the buffers before it, from the weights as they are given. So
a call in the wrong place (another norm, weight or input, a quantiser missing or twice) shows, which the same
calls made by hand would repeat.

Norms with weights of their own in every place; layer 0 and layer 1 (its input is what an engine of one layer
leaves); a prompt step and a decode step. Bounds as in tests/test_fp8_gpu.py: exact where the stage is, else the
8-bit values that lie within a rounding of the exact one, carried through the products; RoPE and attention as in
their own tests (2^-6 of a rotated pair, 1e-2 of the largest)."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import inputs, qwen3
from oracle import bf16_to_f64, decoder as odec, fp8, rmsnorm, round_bf16
from tests._util import bits, f64, ulp_distance
from tests.test_fp8_gpu import EPS_NORM, EPS_SILU, check_held, held_bounds, host

pytestmark = pytest.mark.gpu

CFG = qwen3.Qwen3Config(hidden=1040, layers=2, ffn=1552, heads=8, kv_heads=2, vocab=1000, max_pos=256)
PROMPT, MORE = 70, 3


@pytest.fixture(scope="module")
def weights():
    w = qwen3.Qwen3Weights(CFG, seed=3100)
    for i, at in enumerate([(L, n) for L in w.layers for n in ("in_norm", "q_norm", "k_norm", "post_norm")]):
        L, n = at
        L[n] = inputs.rmsnorm_weight(len(L[n]), seed=3200 + i).cuda()
    w.final_norm = inputs.rmsnorm_weight(CFG.hidden, seed=3300).cuda()
    return w


def step(w, n_layers, new):
    """An engine after the step that gives token `new` of one sequence, and the logits of it."""
    g = torch.Generator().manual_seed(17)
    prompt, forced = (torch.randint(0, CFG.vocab, (n,), generator=g).tolist() for n in (PROMPT, MORE))
    eng = qwen3.Engine(w, num_pages=8, max_tokens_per_step=128, n_layers=n_layers, linear_bits=8)
    logs = eng.generate([qwen3.Sequence(sid=0, prompt=prompt, max_new=new, forced=forced)], record={0})
    assert eng.steps == new
    torch.cuda.synchronize()
    rows = PROMPT if new == 1 else 1
    return eng, {k: v[:rows] for k, v in eng.buf.items() if not k.endswith("s") or k == "res"}, logs[0][-1], (prompt + forced)[:PROMPT + new - 1]


def bf16(x):
    return bf16_to_f64(round_bf16(x))


def norm(x, w):
    return x / np.sqrt((x ** 2).mean(1, keepdims=True) + CFG.eps) * f64(w)


def check_product(y, x, W, off=None):
    """y = bf16 of x . W^T, where x is held to within `off`."""
    off = np.zeros_like(x) if off is None else off
    ref, slack = x @ W.T, off @ np.abs(W).T
    mag = (np.abs(x) + off) @ np.abs(W).T
    err = np.abs(f64(y) - ref)
    assert (err <= slack + 2.0 ** -8 * (np.abs(ref) + slack) + x.shape[1] * 2.0 ** -22 * mag).all()


def check_pairs(got, ref):
    pair = np.hypot(ref[..., :64], ref[..., 64:])
    assert (np.abs(got - ref) <= 2.0 ** -6 * np.concatenate([pair, pair], -1) + 1e-30).all()


def heads_of(x, w, pos):
    """Normed and rotated heads x [T, n, 128]."""
    T, n, D = x.shape
    y = bf16(rmsnorm(round_bf16(x.reshape(-1, D)), w, CFG.eps)).reshape(T, n, D)
    return odec.rope(y.transpose(1, 0, 2), pos, CFG.rope_theta).transpose(1, 0, 2)


@pytest.mark.parametrize("layer", [0, 1])
@pytest.mark.parametrize("new", [1, 3])
def test_stages_of_a_layer(weights, layer, new):
    w, L = weights, weights.layers[layer]
    eng, b, logits, tokens = step(w, layer + 1, new)
    R, N, D, Hq, Hkv, F = b["res"].shape[0], len(tokens), 128, CFG.heads, CFG.kv_heads, CFG.ffn
    if layer == 0:
        x = f64(w.embed)[tokens[N - R:]]
    else:  # the residual stream behind one layer: the last norm adds its share
        x = f64(step(w, 1, new)[1]["res"])
    W = {n: fp8.held(f64(L[n])) for n in ("qkv", "o", "gate_up", "down")}

    # the input norm, held in 8 bits, and the query, key and value projections
    n = norm(x, L["in_norm"])
    lo, hi = held_bounds(n, EPS_NORM)
    check_product(b["qkv"], np.sign(n) * (lo + hi) / 2, W["qkv"], (hi - lo) / 2)

    # heads: norms, rotation, the cache's last rows
    qkv, pos = f64(b["qkv"]).reshape(R, Hq + 2 * Hkv, D), np.arange(N - R, N)
    check_pairs(f64(b["q"]), heads_of(qkv[:, :Hq], L["q_norm"], pos))
    k, v = (f64(c[layer].transpose(1, 2)).reshape(-1, Hkv, D)[:N] for c in (eng.k_cache, eng.v_cache))
    check_pairs(k[N - R:], heads_of(qkv[:, Hq:Hq + Hkv], L["k_norm"], pos))
    assert np.array_equal(v[N - R:], qkv[:, Hq + Hkv:])

    # attention over the cache, its output in 8 bits, the output projection
    q = np.zeros((N, Hq, D))
    q[N - R:] = f64(b["q"])
    ref = odec.causal_attention(q, k, v, 1 / np.sqrt(D))[N - R:]
    assert np.abs(f64(b["attn"]) - ref).max() <= 1e-2 * np.abs(ref).max()
    a = f64(b["attn"]).reshape(R, Hq * D)
    codes, tiles = host(b["attn8"], eng.buf["attn8s"])
    want, scale = fp8.quantise(a)
    assert np.array_equal(fp8.code_values()[codes], want)
    assert np.array_equal(fp8.read_scales(tiles, R, Hq * D), scale)
    check_product(b["o"], fp8.held(a), W["o"])

    # the sum, the norm behind attention, gate|up with SwiGLU in 8 bits, down
    mid = bf16(x + f64(b["o"]))
    check_held(b["n8"], eng.buf["n8s"], norm(mid, L["post_norm"]), EPS_NORM)
    n = fp8.read(*host(b["n8"], eng.buf["n8s"]))
    g, u = n @ W["gate_up"][:F].T, n @ W["gate_up"][F:].T
    dg, du = (CFG.hidden * 2.0 ** -22 * (np.abs(n) @ np.abs(W["gate_up"][s]).T) for s in (slice(F), slice(F, None)))
    sig = 1 / (1 + np.exp(-g))
    ref = fp8.swiglu(g, u)
    off = (np.abs(sig * (1 + g * (1 - sig))) + dg) * (np.abs(u) + du) * dg + np.abs(g * sig) * du + EPS_SILU * np.abs(ref)
    h, hs = fp8.read(*host(b["h8"], eng.buf["h8s"])), fp8.read_scales(eng.buf["h8s"].cpu().numpy(), R, F)
    unit = np.repeat(np.ldexp(1.0, hs - 127), 128, axis=1)[:, :F]
    assert (np.abs(h - ref) <= off + np.maximum((np.abs(ref) + off) * 2.0 ** -4, unit * 2.0 ** -10)).all()
    check_product(b["d"], h, W["down"])

    # the last sum and norm, and the logits, in bf16
    total = bf16(mid + f64(b["d"]))
    assert np.array_equal(f64(b["res"]), total)
    assert ulp_distance(bits(b["n"]), round_bf16(norm(total, w.final_norm))).max() <= 2
    check_product(logits[None], f64(b["n"])[-1:], f64(w.lm_head))
    bi.get_device_error()
