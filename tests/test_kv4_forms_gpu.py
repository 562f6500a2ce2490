"""Forms of the 4-bit cache's kernels that only larger calls take: the fused
append of a step's whole token budget, and the fold of many rows of more than 32
chunks.  Bit for bit, as in test_kv4_gpu.py."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import inputs, qwen3
from tests._util import bits
from tests.test_kv4_gpu import _both, _cache_of, _filled

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    bi.get_device_error()


# Four warps a token from 8 tokens per SM on, eight below.
@pytest.mark.parametrize("past", [-1, 0, 37], ids=["below", "at", "above"])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (64, 8), (5, 2), (12, 3), (1, 1), (5, 5), (13, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_fused_append_of_many_tokens(Hq, Hkv, norm, past):
    """bi_qk_norm_rope_append into a bf16 cache, then bi_kv4_append of its rows;
    slots and positions out of range at the ends and in between are skipped."""
    T = 8 * torch.cuda.get_device_properties(0).multi_processor_count + past
    P = T // 16 + 3
    g = torch.Generator(device="cuda").manual_seed(1100 + Hq)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * 128 + 8, generator=g, device="cuda").to(torch.bfloat16)[:, :-8]
    w = [inputs.rmsnorm_weight(128, seed=1101 + i).cuda() if norm else None for i in range(2)]
    c = torch.Generator().manual_seed(1102)
    pos = torch.randint(0, 4000, (T,), generator=c).to(torch.int32).cuda()
    slots = torch.randperm(P * 16, generator=c)[:T].to(torch.int32).cuda()
    rope = qwen3.rope_table(4096, 1e6, device="cuda")
    kb = torch.zeros(P, Hkv, 16, 128, dtype=torch.bfloat16, device="cuda")
    vb = torch.zeros_like(kb)
    q = bi.qk_norm_rope_append(qkv, Hq, Hkv, pos, slots, rope, *w, kb, vb)
    at = slots.long()
    rows = kb[at // 16, :, at % 16], vb[at // 16, :, at % 16]
    want = _filled(P, Hkv)
    bi.kv4_append(*rows, slots, *want)
    got = _filled(P, Hkv)
    q4 = bi.qk_norm_rope_append_kv4(qkv, Hq, Hkv, pos, slots, rope, *w, *got)
    assert np.array_equal(bits(q4), bits(q))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    bi.get_device_error()

    bad = torch.tensor([0, 700, T - 1], device="cuda")
    slots[bad] = torch.tensor([-1, 16 * P, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    pos[5] = 4096
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[bad] = good[5] = False
    want = _filled(P, Hkv)
    bi.kv4_append(rows[0][good], rows[1][good], slots[good], *want)
    got = _filled(P, Hkv)
    q4 = bi.qk_norm_rope_append_kv4(qkv, Hq, Hkv, pos, slots, rope, *w, *got)
    with pytest.raises(bi.BiError, match="BAD_INPUT"):
        bi.get_device_error()
    assert np.array_equal(bits(q4[good]), bits(q[good]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# 512 rows (sequence, query head) and more are folded a warp a row, 32 chunks at a
# time: rows of exactly 32 chunks, one more, three rounds of them, and rows of one
# chunk between.  18 sequences of 8 kv-heads take the one-warp kernel, 64 of one
# kv-head the four-warp kernel, both that fold.
@pytest.mark.parametrize("B,Hq,Hkv,lens", [
    (18, 32, 8, [8192, 8193, 17000, 1, 8449, 256, 16384, 16385, 257]),
    (64, 8, 1, [8193, 12800, 1, 8192, 8449, 256]),
], ids=["one-warp", "four-warps"])
def test_many_rows_of_more_than_32_chunks(B, Hq, Hkv, lens):
    lens = lens + [1 + 61 * i % 900 for i in range(B - len(lens))]
    msl = max(lens)
    table, P = inputs.paged_layout(torch.tensor(lens), seed=1110)
    g = torch.Generator(device="cuda").manual_seed(1111)
    k, v = (torch.randn(P, Hkv, 16, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, Hq, 128, generator=g, device="cuda").to(torch.bfloat16)
    bt, sl = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    # keys that grow along the first two long sequences: the running maximum moves
    # in later rounds too
    for s in (1, 2):
        n = -(-lens[s] // 16)
        grow = torch.linspace(0.1, 3.0, n, device="cuda").to(torch.bfloat16)[:, None, None, None]
        k[bt[s, :n].long()] *= grow
    kc, vc = _cache_of(k, v)
    got, want, _, _ = _both(q, kc, vc, bt, sl, msl)
    assert np.array_equal(bits(got), bits(want)) and torch.isfinite(got).all()
    # a page out of range in the first round, in a later one, in a row's last chunk
    last = [-(-n // 16) - 1 for n in lens]
    bad = bt.clone()
    bad[0, 100], bad[1, last[1]], bad[2, 16 * 40 + 3] = -1, P, 2 ** 31 - 1
    out = torch.full_like(q, 9.0)
    bi.decode_attention_kv4(q, kc, vc, bad, sl, msl, out=out)
    with pytest.raises(bi.BiError, match="BAD_INPUT"):
        bi.get_device_error()
    hit = [0, 1, 2] if lens[2] > 256 * 40 else [0, 1]
    keep = [i for i in range(B) if i not in hit]
    assert (out[hit] == 9).all() and np.array_equal(bits(out[keep]), bits(want[keep]))
