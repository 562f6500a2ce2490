"""Forms of the 4-bit cache's kernels that only larger calls take: the fused
append of a step's whole token budget.  Bit for bit, as in test_kv4_gpu.py."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import inputs, qwen3
from tests._util import bits
from tests.test_kv4_gpu import _filled

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
