"""The decoder served from a 4-bit KV cache, and its per-token report.

Everything is bit for bit.  Served from a 4-bit cache the decoder has to give
the logits of a decoder with a bf16 cache (which is compared with the fp64
oracle elsewhere) whose appended rows pass through the fp64 oracle of the 4-bit
format before anything reads them.  And alone as batched, graphs as eager,
prompts cut anywhere."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import qwen3
from oracle import kv4
from tests._util import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def two_layer():
    cfg = qwen3.Qwen3Config(layers=2, max_pos=1024)
    return cfg, qwen3.Qwen3Weights(cfg, seed=2000)


def test_logits_are_those_of_rows_passed_through_the_format(two_layer, monkeypatch):
    cfg, w = two_layer

    def sequences():
        g = torch.Generator().manual_seed(5)
        out = []
        for i, L in enumerate((12, 20, 7)):
            prompt = torch.randint(0, cfg.vocab, (L,), generator=g).tolist()
            forced = torch.randint(0, cfg.vocab, (4,), generator=g).tolist()
            out.append(qwen3.Sequence(sid=i, prompt=prompt, max_new=4, forced=forced))
        return out
    got = qwen3.Engine(w, num_pages=64, max_tokens_per_step=30, kv_bits=4).generate(sequences(), record={0, 1, 2})
    append = qwen3.qk_norm_rope_append

    def append_through_the_format(qkv, Hq, Hkv, pos, slots, rope, qn, kn, k_cache, v_cache, eps, q_out):
        append(qkv, Hq, Hkv, pos, slots, rope, qn, kn, k_cache, v_cache, eps, q_out=q_out)
        at = slots.long()
        for c in (k_cache, v_cache):
            rows = kv4.values(*kv4.quantise(c[at // 16, :, at % 16].cpu().double().numpy()))
            c[at // 16, :, at % 16] = torch.from_numpy(rows).to(torch.bfloat16).cuda()
    monkeypatch.setattr(qwen3, "qk_norm_rope_append", append_through_the_format)
    want = qwen3.Engine(w, num_pages=64, max_tokens_per_step=30).generate(sequences(), record={0, 1, 2})
    for sid in want:
        assert len(want[sid]) == 4
        for a, b in zip(got[sid], want[sid]):
            assert np.array_equal(bits(a), bits(b))
    bi.get_device_error()


def test_bits_alone_batched_graphed_and_reported(two_layer):
    cfg, w = two_layer
    track = {0, 3, 9}
    runs = []
    for graphs, budget in ((False, 130), (True, 300)):
        reqs = qwen3.random_requests(10, cfg.vocab, 1, 150, max_new=6, seed=21)
        eng = qwen3.Engine(w, num_pages=10 * 10 + 1, max_tokens_per_step=budget, cuda_graphs=graphs, kv_bits=4)
        runs.append((reqs, eng.generate(reqs, record=track, top=5), eng))
    (r0, l0, e0), (r1, l1, e1) = runs
    assert e1.graph_steps > 0
    for sid in track:
        assert r0[sid].generated == r1[sid].generated
        alone = qwen3.Sequence(sid=sid, prompt=list(r0[sid].prompt), max_new=6)
        e1.reset()
        la = qwen3.Engine(w, num_pages=16, max_tokens_per_step=64, kv_bits=4).generate([alone], record={sid})
        assert alone.generated == r0[sid].generated
        for step in range(6):
            row = l0[sid][step]
            assert np.array_equal(bits(row), bits(l1[sid][step])) and np.array_equal(bits(row), bits(la[sid][step]))
            # the report is that of the recorded row, in either run
            lp, _, h, ids, top = bi.logprobs_top(row[None].cuda(), torch.tensor([r0[sid].generated[step]],
                                                                                dtype=torch.int32).cuda(), 5)
            for e in (e0, e1):
                assert torch.equal(e.logprobs[sid][step], lp[0].cpu())
                assert torch.equal(e.entropies[sid][step], h[0].cpu())
                assert torch.equal(e.top[sid][step][0], ids[0].cpu())
                assert torch.equal(e.top[sid][step][1], top[0].cpu())
            assert ids[0, 0].item() == r0[sid].generated[step]  # greedy: the likeliest token was chosen
    bi.get_device_error()


def test_engine_refuses_other_widths_and_reports(two_layer):
    with pytest.raises(ValueError, match="kv_bits"):
        qwen3.Engine(two_layer[1], num_pages=4, kv_bits=8)
    for top in (-1, 33):
        with pytest.raises(ValueError, match="top"):
            qwen3.Engine(two_layer[1], num_pages=4).generate([], top=top)
