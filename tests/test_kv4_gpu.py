"""The 4-bit KV cache on the GPU: writing, reading back, attention over it.

Writing and reading are compared bit for bit with the fp64 oracle of the format
(a row's codes and scales are exact functions of its bf16 values).  Attention
is compared bit for bit with bi_decode_attention over the read-back cache --
its definition -- and with the fp64 oracle within

    |got - ref| <= 2^-8 |ref| + 2^-13 max|v|:

the output's rounding (half a bf16 step, 2^-9 relative, 2^-8 allowed); weights
kept to 16 bits by the hi + lo split (2^-17 of max|v| each way) and scores of
128 fp32 products, each within 128 * 2^-24 * sum|q k| * scale, here at most
2^-17 * 40 = 2^-11.7 in the worst of cases and below 2^-14 typically, which
moves a weighted mean of v by less than 2^-13 max|v|."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
import oracle
from invariant_bi_rmsnorm_gb300 import inputs, qwen3
from oracle import kv4
from tests._util import bits, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    bi.get_device_error()


def _filled(num_pages, Hkv, byte=0xFF):
    """Caches whose unwritten bytes would show: scales of 0xFFFF are NaN."""
    k = torch.full((num_pages, Hkv, bi.KV4_BLOCK_BYTES), byte, dtype=torch.uint8, device="cuda")
    return k, k.clone()


def _cache_of(k, v):
    """4-bit caches of bf16 caches [P, Hkv, 16, 128] through kv4_append."""
    P, Hkv = k.shape[:2]
    kc, vc = _filled(P, Hkv)
    rows = [x.transpose(1, 2).reshape(P * 16, Hkv, 128) for x in (k, v)]
    bi.kv4_append(*rows, torch.arange(P * 16, dtype=torch.int32, device="cuda"), kc, vc)
    return kc, vc


def _read_all(kc, vc):
    """The whole caches read back."""
    P, Hkv = kc.shape[:2]
    ko = torch.zeros(P, Hkv, 16, 128, dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    bi.kv4_read(kc, vc, torch.arange(P, dtype=torch.int32, device="cuda")[None],
                torch.tensor([16 * P], dtype=torch.int32, device="cuda"), 16 * P, ko, vo)
    return ko, vo


# ------------------------------------------------------------------ writing ----
@pytest.mark.parametrize("T,Hkv,strided", [(1, 1, False), (1, 8, True), (7, 3, False), (33, 5, True),
                                           (130, 8, True), (300, 2, False)])
def test_append_writes_the_oracles_bytes(T, Hkv, strided):
    num_pages = T // 16 + 3
    wide = inputs.normal_bf16((T, 2 + 2 * Hkv, 128), seed=900 + T) if strided else None
    k = wide[:, 2:2 + Hkv] if strided else inputs.normal_bf16((T, Hkv, 128), seed=901, std=3.0)
    v = wide[:, 2 + Hkv:] if strided else inputs.normal_bf16((T, Hkv, 128), seed=902, std=0.01)
    if strided:
        w = wide.cuda()
        kd, vd = w[:, 2:2 + Hkv], w[:, 2 + Hkv:]
    else:
        kd, vd = k.cuda(), v.cuda()
    slots = torch.randperm(num_pages * 16, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    kc, vc = _filled(num_pages, Hkv, 0x5A)
    bi.kv4_append(kd, vd, slots.cuda(), kc, vc)
    for got, x, is_v in ((kc, k, False), (vc, v, True)):
        want = np.full((num_pages, Hkv, kv4.BLOCK), 0x5A, dtype=np.uint8)
        for t, s in enumerate(slots.tolist()):
            kv4.write(want[s // 16], is_v, s % 16, f64(x[t]))
        assert np.array_equal(got.cpu().numpy(), want)


def _hard_rows():
    """Groups where a quantiser goes wrong: zeros, one value, every mantissa of
    the largest magnitude with exact ties beside it, the range's two ends, and
    what is not finite."""
    groups = [np.zeros(32), np.eye(32)[3], -np.eye(32)[31] * 2.0 ** -133]
    for m in range(128, 256):
        amax = m / 64
        s = float(kv4._round_sig4(np.array(amax / 7.0)))
        ties = (np.arange(-7, 7) + 0.5) * s
        g = np.concatenate([[amax], ties, -ties[::-1], np.linspace(-amax, amax, 3)])
        groups.append(np.clip(g, -amax, amax))
    for e in (-133, -130, -127, -110, -103, -100, -99, -60, 60, 120):
        groups.append(np.linspace(-1, 1, 32) * 2.0 ** e)
    near = np.linspace(-1, 1, 32) * 2.0 ** 123
    groups += [near * (1 - 2.0 ** -8), near]  # the largest that is kept, and one past it
    for bad in (np.nan, np.inf, -np.inf):
        g = np.linspace(-1, 1, 32)
        g[17] = bad
        groups.append(g)
    while len(groups) % 4:
        groups.append(np.zeros(32))
    return torch.tensor(np.stack(groups).reshape(-1, 1, 128)).to(torch.bfloat16)


def test_append_hard_groups():
    x = _hard_rows()
    T = x.shape[0]
    P = -(-T // 16)
    kc, vc = _filled(P, 1, 0)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    bi.kv4_append(x.cuda(), x.cuda(), slots, kc, vc)
    n, s = kv4.quantise(f64(x))
    want = kv4.values(n, s)[:, 0]
    for c, is_v in ((kc, False), (vc, True)):
        got = kv4.unpack(c.cpu().numpy(), is_v)[:, 0].reshape(-1, 128)[:T]
        assert np.array_equal(got, want, equal_nan=True)
    # and read back they are those bf16 numbers
    for got in _read_all(kc, vc):
        assert np.array_equal(f64(got)[:, 0].reshape(-1, 128)[:T], want, equal_nan=True)


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (3, 1), (12, 3), (5, 5), (64, 8), (4, 2), (1, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_fused_append_is_the_two_calls(Hq, Hkv, norm):
    """bi_qk_norm_rope_append_kv4 = bi_qk_norm_rope_append into a bf16 cache,
    then bi_kv4_append of its rows, bit for bit."""
    T, P = 41, 6
    qkv = inputs.normal_bf16((T, (Hq + 2 * Hkv) * 128 + 8), seed=910, std=1.5).cuda()[:, :-8]
    w = [inputs.rmsnorm_weight(128, seed=911 + i).cuda() if norm else None for i in range(2)]
    g = torch.Generator().manual_seed(912)
    pos = torch.randint(0, 4000, (T,), generator=g).to(torch.int32).cuda()
    slots = torch.randperm(P * 16, generator=g)[:T].to(torch.int32).cuda()
    rope = qwen3.rope_table(4096, 1e6, device="cuda")
    kb = torch.zeros(P, Hkv, 16, 128, dtype=torch.bfloat16, device="cuda")
    vb = torch.zeros_like(kb)
    q = bi.qk_norm_rope_append(qkv, Hq, Hkv, pos, slots, rope, *w, kb, vb)
    want = _filled(P, Hkv)
    at = slots.long()
    bi.kv4_append(kb[at // 16, :, at % 16], vb[at // 16, :, at % 16], slots, *want)
    got = _filled(P, Hkv)
    q4 = bi.qk_norm_rope_append_kv4(qkv, Hq, Hkv, pos, slots, rope, *w, *got)
    assert np.array_equal(bits(q4), bits(q))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_slots_and_positions_are_skipped():
    T, P, Hkv = 5, 2, 3
    k = inputs.normal_bf16((T, Hkv, 128), seed=920).cuda()
    slots = torch.tensor([3, -1, 32, 7, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    kc, vc = _filled(P, Hkv)
    bi.kv4_append(k, k, slots, kc, vc)
    with pytest.raises(bi.BiError, match="BAD_INPUT"):
        bi.get_device_error()
    want = _filled(P, Hkv)
    good = torch.tensor([0, 3], device="cuda")
    bi.kv4_append(k[good], k[good], slots[good], *want)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    # the fused form: a bad position, a bad slot
    qkv = inputs.normal_bf16((3, 4 * 128), seed=921).cuda()
    rope = qwen3.rope_table(16, 1e6, device="cuda")
    kc, vc = _filled(P, 1)
    bi.qk_norm_rope_append_kv4(qkv, 2, 1, torch.tensor([16, 4, 2], dtype=torch.int32, device="cuda"),
                               torch.tensor([0, 40, 5], dtype=torch.int32, device="cuda"), rope, None,
                               None, kc, vc)
    with pytest.raises(bi.BiError, match="BAD_INPUT"):
        bi.get_device_error()
    changed = (kc != 0xFF).any(0).any(0)
    assert changed[:1024].nonzero().min() >= 64 * 5 and changed[:1024].nonzero().max() < 64 * 6


# ------------------------------------------------------------- reading back ----
@pytest.mark.parametrize("lens", [[1], [16], [17, 0, 300], [15, 33, 1, 64, 257]])
@pytest.mark.parametrize("Hkv", [1, 8, 5])
def test_read_back(lens, Hkv):
    table, P = inputs.paged_layout(torch.tensor(lens), seed=931, spare_pages=2)
    rng = np.random.default_rng(930)
    raw = rng.integers(0, 256, (2, P, Hkv, kv4.BLOCK), dtype=np.uint8)
    raw[..., 1024:] = 0xFF  # NaN scales, but for the tokens that a sequence has
    scales = (rng.integers(8, 16, (2, P, Hkv, 16, 4)) * 2.0 ** -5).astype(np.float32).view(np.uint32) >> 16
    for i, L in enumerate(lens):
        for t in range(L):
            p = int(table[i, t // 16])
            sc = scales[:, p, :, t % 16].astype(np.uint16)
            raw[:, p, :, 1024 + 8 * (t % 16):1032 + 8 * (t % 16)] = sc.view(np.uint8).reshape(2, Hkv, 8)
    kc, vc = torch.from_numpy(raw).cuda().unbind(0)
    ko = torch.full((P, Hkv, 16, 128), -77.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    bi.kv4_read(kc.contiguous(), vc.contiguous(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                max(lens), ko, vo)
    for got, is_v in ((ko, False), (vo, True)):
        want = np.full((P, Hkv, 16, 128), -77.0)
        full = kv4.unpack(raw[int(is_v)], is_v)
        for i, L in enumerate(lens):
            for t in range(L):
                p = int(table[i, t // 16])
                want[p, :, t % 16] = full[p, :, t % 16]
        assert np.array_equal(f64(got), want)


def test_read_back_refuses_bad_pages_and_lengths():
    kc, vc = bi.kv4_cache(4, 2)
    ko = torch.full((4, 2, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    table = torch.tensor([[0, 9], [1, -1], [2, 3], [3, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([32, 20, 33, -1], dtype=torch.int32, device="cuda")  # 33 > max, -1
    bi.kv4_read(kc, vc, table, lens, 32, ko, vo)
    with pytest.raises(bi.BiError, match="BAD_INPUT"):
        bi.get_device_error()
    # the good pages were read (zero codes of zero scale: zeros), the others left alone
    assert (ko[:2] == 0).all() and (vo[:2] == 0).all() and (ko[2:] == 5).all() and (vo[2:] == 5).all()


# ---------------------------------------------------------------- attention ----
def _problem(lens, Hq, Hkv, seed, spare=3):
    p = inputs.decode_problem(len(lens), Hq=Hq, Hkv=Hkv, seq_lens=lens, seed=seed, spare_pages=spare,
                              device="cuda")
    kc, vc = _cache_of(p["k_cache"], p["v_cache"])
    return (p["q"].cuda(), kc, vc, p["block_table"].cuda(), p["seq_lens"].cuda())


# Launches of many chunks run a kernel of their own, and chunks of long sequences
# are folded by one; a bound on the lengths far above them makes such a launch of
# any batch.
BOTH_KERNELS = pytest.mark.parametrize("many", [False, True, "long"], ids=["few-chunks", "many-chunks", "long"])


def _bound(many, bt, msl, Hkv):
    """(block table, max_seq_len) of a launch of few or of many chunks."""
    if many == "long":
        msl = 256 * 40
    elif many:
        msl = 256 * -(-42 * 160 // (bt.shape[0] * Hkv))
    wide = torch.full((bt.shape[0], max(bt.shape[1], -(-msl // 16))), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    return wide, msl


def _both(q, kc, vc, bt, lens, msl, **kw):
    got = bi.decode_attention_kv4(q, kc, vc, bt, lens, msl, **kw)
    ko, vo = _read_all(kc, vc)
    want = bi.decode_attention(q, ko, vo, bt, lens, msl, **kw)
    return got, want, ko, vo


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 1), (5, 5), (14, 2), (3, 1), (28, 4), (6, 3), (20, 4), (6, 1)])
@BOTH_KERNELS
def test_attention_has_the_bits_of_the_read_back_cache(Hq, Hkv, many):
    lens = [1, 2, 15, 16, 17, 255, 256, 257, 1000, 1025, 40, 2049]
    q, kc, vc, bt, sl = _problem(lens, Hq, Hkv, 940 + Hq)
    bt, msl = _bound(many, bt, max(lens), Hkv)
    got, want, ko, vo = _both(q, kc, vc, bt, sl, msl)
    assert np.array_equal(bits(got), bits(want))
    ref = oracle.decode_attention(q.cpu(), ko.cpu(), vo.cpu(), bt.cpu(), sl.cpu())
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * float(vo.abs().max())
    assert (np.abs(f64(got) - ref) <= tol).all(), np.abs(f64(got) - ref).max()


@pytest.mark.parametrize("lens,msl", [([1], 1), ([300], 300), ([8192], 8192), ([9000, 3], 9001),
                                      ([256] * 40, 256), ([700] * 70, 4096), ([8192] * 9, 8192),
                                      ([5000, 1] * 130, 8192), ([70000], 70000),
                                      ([20000, 3, 8193, 8192, 257], 131072)])
def test_attention_over_launch_shapes(lens, msl):
    """Few and many sequences, one and many chunks a CTA, and a bound far above
    the lengths: always the read-back cache's bits."""
    q, kc, vc, bt, sl = _problem(lens, 32 if len(lens) < 60 else 8, 8 if len(lens) < 60 else 2, 960)
    if bt.shape[1] * 16 < msl:
        wide = torch.full((len(lens), -(-msl // 16)), -1, dtype=torch.int32, device="cuda")
        wide[:, :bt.shape[1]] = bt
        bt = wide
    got, want, _, _ = _both(q, kc, vc, bt, sl, msl)
    assert np.array_equal(bits(got), bits(want))


def test_more_pairs_than_counters():
    """65544 (sequence, kv-head) pairs, some of several chunks: the workspace has 65536 arrival counters."""
    B, Hkv = 8193, 8
    lens = [1 + (i * 37) % 40 for i in range(B)]
    lens[5], lens[8000] = 1500, 1300
    table, P = inputs.paged_layout(torch.tensor(lens), seed=971)
    g = torch.Generator(device="cuda").manual_seed(972)
    k = torch.randn(P, Hkv, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(P, Hkv, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    kc, vc = _cache_of(k, v)
    q = torch.randn(B, Hkv, 128, generator=g, device="cuda").to(torch.bfloat16)
    got, want, _, _ = _both(q, kc, vc, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 1500)
    assert np.array_equal(bits(got), bits(want))


def test_warps_that_take_several_chunks():
    """4800 (sequence, kv-head) pairs under a bound of 8 chunks: more chunks than
    warps.  A bad page in one sequence's third chunk, another's first and last."""
    B, Hkv = 600, 8
    lens = [1 + (i * 397) % 2000 for i in range(B)]
    lens[7], lens[300] = 1999, 1300
    table, P = inputs.paged_layout(torch.tensor(lens), seed=973)
    g = torch.Generator(device="cuda").manual_seed(974)
    k = torch.randn(P, Hkv, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(P, Hkv, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    kc, vc = _cache_of(k, v)
    q = torch.randn(B, 2 * Hkv, 128, generator=g, device="cuda").to(torch.bfloat16)
    bt, sl = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    got, want, _, _ = _both(q, kc, vc, bt, sl, 2000)
    assert np.array_equal(bits(got), bits(want))
    bt = bt.clone()
    bt[7, 40], bt[300, 0], bt[300, 81] = -1, P, 2 ** 31 - 1
    out = torch.full_like(q, 9.0)
    bi.decode_attention_kv4(q, kc, vc, bt, sl, 2000, out=out)
    with pytest.raises(bi.BiError, match="BAD_INPUT"):
        bi.get_device_error()
    assert (out[[7, 300]] == 9).all()
    keep = torch.ones(B, dtype=torch.bool)
    keep[[7, 300]] = False
    assert np.array_equal(bits(out[keep.cuda()]), bits(want[keep.cuda()]))


def test_read_back_under_a_bound_far_above_the_lengths():
    """More pages under the bound than the launch has CTAs."""
    S, Hkv, bound = 40, 5, 40000
    lens = [0, 1, 16, 17, 39999, 2500] + [3 * i for i in range(S - 6)]
    need = [-(-n // 16) for n in lens]
    P = sum(need) + 1
    kc = torch.randint(0, 256, (P, Hkv, bi.KV4_BLOCK_BYTES), dtype=torch.uint8, device="cuda")
    kc[:, :, 1024:] = torch.tensor([0x80, 0x3F], dtype=torch.uint8, device="cuda").repeat(64)  # scales of 1
    vc = kc.flip(0).contiguous()
    order = torch.randperm(P, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    bt = torch.full((S, bound // 16), -1, dtype=torch.int32)
    used = 0
    for i, n in enumerate(need):
        bt[i, :n] = order[used:used + n]
        used += n
    sl = torch.tensor(lens, dtype=torch.int32)
    outs = [torch.full((P, Hkv, 16, 128), 99.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bi.kv4_read(kc, vc, bt.cuda(), sl.cuda(), bound, *outs)
    bi.get_device_error()
    whole = _read_all(kc, vc)  # every page, all 16 rows
    for got, every in zip(outs, whole):
        want = torch.full_like(got, 99.0)
        for i, L in enumerate(lens):
            for p in range(need[i]):
                n = min(16, L - 16 * p)
                want[int(bt[i, p]), :, :n] = every[int(bt[i, p]), :, :n]
        assert np.array_equal(bits(got), bits(want))


def test_row_alone_and_in_a_batch():
    lens = [5, 8000, 256, 1, 4097, 700, 31]
    q, kc, vc, bt, sl = _problem(lens, 32, 8, 980)
    ws = torch.zeros(bi.decode_attention_workspace_size(7, 32, 128, 8192), dtype=torch.uint8, device="cuda")
    wide = torch.full((7, 512), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    batch = bi.decode_attention_kv4(q, kc, vc, wide, sl, 8192, workspace=ws)
    for i, L in enumerate(lens):
        for msl in (L, 8192):
            one = bi.decode_attention_kv4(q[i:i + 1], kc, vc, wide[i:i + 1].contiguous(), sl[i:i + 1], msl,
                                          workspace=ws)
            assert np.array_equal(bits(one[0]), bits(batch[i])), (L, msl)
    assert not ws[:bi._lib.DECODE_COUNTER_BYTES].any()  # counters are left zero


@pytest.mark.parametrize("scale", [1e-6, 0.5, 30.0])
@BOTH_KERNELS
def test_peaked_and_flat_scores(scale, many):
    lens = [3, 290, 1030]
    q, kc, vc, bt, sl = _problem(lens, 16, 4, 985)
    bt, msl = _bound(many, bt, max(lens), 4)
    got, want, _, _ = _both(q, kc, vc, bt, sl, msl, scale=scale)
    assert np.array_equal(bits(got), bits(want)) and torch.isfinite(got).all()


@BOTH_KERNELS
def test_scores_that_climb_page_after_page(many):
    """Keys that grow along the sequence move the reference maximum on every
    page; keys that shrink leave it at the first; either way down to weights of
    zero.  And queries of -inf and NaN, which show in their own head only."""
    lens = [700, 256, 33]
    q, kc, vc, bt, sl = _problem(lens, 8, 4, 987)
    P = kc.shape[0]
    k, v = _read_all(kc, vc)
    for i, L in enumerate(lens):
        for t in range(L):
            k[int(bt[i, t // 16]), :, t % 16] = ((t + 1) if i == 0 else (L - t)) / 40 * q[i, ::2].sign()
    kc, vc = _cache_of(k, v)
    bt, msl = _bound(many, bt, 700, 4)
    got, want, _, _ = _both(q, kc, vc, bt, sl, msl)
    assert np.array_equal(bits(got), bits(want)) and torch.isfinite(got).all() and P
    bad = q.clone()
    bad[0, 3, 5], bad[1, 2, 7], bad[2, 6, 0] = float("inf"), float("nan"), float("-inf")
    got2, want2, _, _ = _both(bad, kc, vc, bt, sl, msl)
    assert torch.equal(got2.isnan(), want2.isnan())
    assert torch.equal(got2.nan_to_num(0.0), want2.nan_to_num(0.0))
    for i, h in ((0, 3), (1, 2), (2, 6)):
        keep = [j for j in range(8) if j != h]
        assert np.array_equal(bits(got2[i, keep]), bits(got[i, keep]))


@BOTH_KERNELS
def test_what_lies_behind_a_sequence_never_counts(many):
    """Codes and scales of tokens behind the end, NaN scales among them."""
    lens = [1, 9, 23, 511]
    q, kc, vc, bt, sl = _problem(lens, 8, 2, 990)
    bt, msl = _bound(many, bt, 511, 2)
    ref = bi.decode_attention_kv4(q, kc, vc, bt, sl, msl)
    for i, L in enumerate(lens):
        p, r = int(bt[i, (L - 1) // 16]), (L - 1) % 16 + 1
        for c in (kc, vc):
            c[p, :, 1024 + 8 * r:] = 0xFF
        kc[p, :, 64 * r:1024] = 0x99
    assert np.array_equal(bits(bi.decode_attention_kv4(q, kc, vc, bt, sl, msl)), bits(ref))
    assert torch.isfinite(ref).all()


@BOTH_KERNELS
def test_a_nan_group_shows_in_its_own_sequence_only(many):
    lens = [40, 40]
    q, kc, vc, bt, sl = _problem(lens, 4, 1, 992)
    bt, msl = _bound(many, bt, 40, 1)
    ref = bi.decode_attention_kv4(q, kc, vc, bt, sl, msl)
    bad = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    bad[0, 0, 100] = float("inf")
    zero = torch.zeros_like(bad)
    slot = (bt[0, 1] * 16 + 3).reshape(1).to(torch.int32)
    bi.kv4_append(zero, bad, slot, kc, vc)
    got, want, _, _ = _both(q, kc, vc, bt, sl, msl)
    assert np.array_equal(bits(got[1]), bits(ref[1])) and np.array_equal(bits(got), bits(want))
    assert torch.isnan(got[0, :, 96:]).all() and torch.isfinite(got[0, :, :96]).all()


@BOTH_KERNELS
def test_bad_pages_and_lengths_are_reported(many):
    lens = [40, 600, 33, 20]
    q, kc, vc, bt, sl = _problem(lens, 8, 2, 995)
    bt, msl = _bound(many, bt, 2048, 2)
    ws = torch.zeros(bi.decode_attention_workspace_size(4, 8, 128, msl), dtype=torch.uint8, device="cuda")
    ref = bi.decode_attention_kv4(q, kc, vc, bt, sl, msl, workspace=ws)
    for row, col, bad in ((0, 1, kc.shape[0]), (1, 20, -1), (1, 37, 2 ** 31 - 1)):
        t = bt.clone()
        t[row, col] = bad
        out = torch.full_like(q, 9.0)
        bi.decode_attention_kv4(q, kc, vc, t, sl, msl, out=out, workspace=ws)
        with pytest.raises(bi.BiError, match="BAD_INPUT"):
            bi.get_device_error()
        keep = [i for i in range(4) if i != row]
        assert (out[row] == 9).all() and np.array_equal(bits(out[keep]), bits(ref[keep]))
        assert not ws[:bi._lib.DECODE_COUNTER_BYTES].any()
    for bad in (0, -5, msl + 1):
        l2 = sl.clone()
        l2[2] = bad
        out = torch.full_like(q, 9.0)
        bi.decode_attention_kv4(q, kc, vc, bt, l2, msl, out=out, workspace=ws)
        with pytest.raises(bi.BiError, match="BAD_INPUT"):
            bi.get_device_error()
        assert (out[2] == 9).all() and np.array_equal(bits(out[:2]), bits(ref[:2]))
    # and all is well afterwards
    assert np.array_equal(bits(bi.decode_attention_kv4(q, kc, vc, bt, sl, msl, workspace=ws)), bits(ref))


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: its last pages."""
    P, Hkv = 480_000, 8
    kc = torch.zeros(P, Hkv, bi.KV4_BLOCK_BYTES, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 32
    T = 40
    rows = inputs.normal_bf16((2, T, Hkv, 128), seed=997).cuda()
    pages = torch.tensor([[P - 1, 0, P - 2]], dtype=torch.int32, device="cuda")
    t = torch.arange(T, device="cuda")
    slots = (pages[0].long()[t // 16] * 16 + t % 16).to(torch.int32)
    bi.kv4_append(rows[0], rows[1], slots, kc, vc)
    sk, sv = _filled(3, Hkv, 0)
    small = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    bi.kv4_append(rows[0], rows[1], (small[0].long()[t // 16] * 16 + t % 16).to(torch.int32), sk, sv)
    q = inputs.normal_bf16((1, 32, 128), seed=998).cuda()
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    a = bi.decode_attention_kv4(q, kc, vc, pages, lens, T)
    b = bi.decode_attention_kv4(q, sk, sv, small, lens, T)
    assert np.array_equal(bits(a), bits(b))


# -------------------------------------------------------- a run of them ----
def test_prompt_then_decode_as_a_server_runs_them():
    """Prompts written in two chunks and read back for prefill, then decode
    steps: every row has the bits that one prefill over the whole would give."""
    Hq, Hkv = 16, 4
    lens, steps = [70, 5, 300], 3
    total = [n + steps for n in lens]
    table, P = inputs.paged_layout(torch.tensor(total), seed=1001, spare_pages=1)
    bt = table.cuda()
    rope = qwen3.rope_table(1024, 1e6, device="cuda")
    w = [inputs.rmsnorm_weight(128, seed=1002 + i).cuda() for i in range(2)]
    qkv = [inputs.normal_bf16((n, (Hq + 2 * Hkv) * 128), seed=1010 + i).cuda() for i, n in enumerate(total)]
    i32 = dict(dtype=torch.int32, device="cuda")

    def step(caches, spans):
        """spans: (sequence, first, last) -> q rows; writes K/V."""
        rows = torch.cat([qkv[i][a:b] for i, a, b in spans])
        pos = torch.cat([torch.arange(a, b) for _, a, b in spans])
        seq = torch.cat([torch.full((b - a,), i) for i, a, b in spans])
        slots = table[seq, pos // 16] * 16 + pos % 16
        return bi.qk_norm_rope_append_kv4(rows, Hq, Hkv, pos.to(torch.int32).cuda(),
                                          slots.to(torch.int32).cuda(), rope, *w, *caches)

    def prefill(caches, spans):
        q = step(caches, spans)
        ko = torch.full((P, Hkv, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        vo = ko.clone()
        sl = torch.tensor([b for _, _, b in spans], **i32)
        rows = bt[[i for i, _, _ in spans]].contiguous()
        msl = max(b for _, _, b in spans)
        bi.kv4_read(*caches, rows, sl, msl, ko, vo)
        n = [b - a for _, a, b in spans]
        indptr = torch.tensor(np.concatenate([[0], np.cumsum(n)]), **i32)
        out = bi.prefill_attention(q, ko, vo, rows, sl, indptr, max(n), msl)
        return dict(zip([(i, t) for i, a, b in spans for t in range(a, b)], out))

    whole = prefill(_filled(P, Hkv), [(i, 0, n) for i, n in enumerate(total)])
    caches = _filled(P, Hkv)
    got = prefill(caches, [(0, 0, 33), (1, 0, 5)])
    got |= prefill(caches, [(0, 33, 70), (2, 0, 300)])
    for s in range(steps):
        spans = [(i, n + s, n + s + 1) for i, n in enumerate(lens)]
        q = step(caches, spans)
        out = bi.decode_attention_kv4(q, *caches, bt, torch.tensor([b for _, _, b in spans], **i32), max(total))
        got |= {(i, a): o for (i, a, _), o in zip(spans, out)}
    assert set(got) == set(whole)
    for at in whole:
        assert np.array_equal(bits(got[at]), bits(whole[at])), at


@pytest.mark.parametrize("bound", [4096, 65536], ids=["few-chunks", "many-chunks"])
def test_captured_steps_replay_beside_eager_ones(bound):
    """Two captured decode steps with a workspace each, replayed with changed
    inputs while eager calls run on another stream."""
    lens = [700, 30, 4000]
    q, kc, vc, bt, sl = _problem(lens, 32, 8, 1020)
    size = bi.decode_attention_workspace_size(3, 32, 128, bound)
    wide = torch.full((3, bound // 16), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    states = []
    for n in range(2):
        qs, out = q.clone(), torch.empty_like(q)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        bi.decode_attention_kv4(qs, kc, vc, wide, sl, bound, out=out, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bi.decode_attention_kv4(qs, kc, vc, wide, sl, bound, out=out, workspace=ws)
        states.append((g, qs, out))
    side = torch.cuda.Stream()
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for n in range(3):
        new = [inputs.normal_bf16(tuple(q.shape), seed=1030 + 10 * n + i).cuda() for i in range(2)]
        for (g, qs, _), x in zip(states, new):
            qs.copy_(x)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            e = bi.decode_attention_kv4(new[0], kc, vc, wide, sl, bound, workspace=ws)
        for g, _, _ in states:
            g.replay()
        torch.cuda.synchronize()
        for (_, _, out), x in zip(states, new):
            assert np.array_equal(bits(out), bits(bi.decode_attention_kv4(x, kc, vc, wide, sl, bound)))
        assert np.array_equal(bits(e), bits(states[0][2]))


def test_binding_refusals():
    kc, vc = bi.kv4_cache(4, 2)
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(3, dtype=torch.int32, device="cuda")
    rope = torch.zeros(4, 128, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    qkv = torch.zeros(3, 768, dtype=torch.bfloat16, device="cuda")
    bt = idx[:, None].contiguous()

    def refused(match, f, *a, kind=ValueError, **kw):
        with pytest.raises(kind, match=match):
            f(*a, **kw)
    refused("side by side", bi.kv4_append, rows.transpose(0, 1).contiguous().transpose(0, 1), rows, idx, kc, vc)
    refused("k_cache", bi.kv4_append, rows[:, :1], rows[:, :1], idx, kc, vc)
    refused("same shape", bi.kv4_append, rows, rows[:2], idx, kc, vc)
    refused("slots", bi.kv4_append, rows, rows, idx[:2], kc, vc)
    refused("int32", bi.kv4_append, rows, rows, idx.long(), kc, vc)
    refused("bfloat16", bi.kv4_append, rows.float(), rows, idx, kc, vc)
    refused("1152", bi.kv4_append, rows, rows, idx, kc[..., :1024].contiguous(), vc[..., :1024].contiguous())
    refused("contiguous", bi.kv4_append, rows, rows, idx, kc, vc.expand(4, 2, 1152).transpose(0, 1).contiguous().transpose(0, 1))
    refused("CUDA", bi.kv4_append, rows, rows, idx.cpu(), kc, vc)
    refused("uint8", bi.decode_attention_kv4, rows, kc.float(), vc, bt, idx, 16)
    refused("v_cache", bi.decode_attention_kv4, rows, kc, vc[:3], bt, idx, 16)
    refused("seq_lens", bi.decode_attention_kv4, rows, kc, vc, bt, idx[:2], 16)
    refused("block_table", bi.decode_attention_kv4, rows, kc, vc, bt[:2], idx, 16)
    refused("out", bi.decode_attention_kv4, rows, kc, vc, bt, idx, 16, out=rows[:2].clone())
    refused("q must be contiguous", bi.decode_attention_kv4, rows.transpose(0, 1), kc, vc, bt, idx, 16)
    refused("CUDA", bi.decode_attention_kv4, rows, kc, vc, bt, idx, 16, workspace=torch.zeros(64))
    refused("TOO_SMALL", bi.decode_attention_kv4, rows, kc, vc, torch.zeros(3, 32, dtype=torch.int32, device="cuda"),
            idx, 512, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"), kind=bi.BiError)
    refused("k_out", bi.kv4_read, kc, vc, bt, idx, 16, rows, rows)
    refused("seq_lens", bi.kv4_read, kc, vc, bt, idx[:1], 16, rows, rows)
    fused = bi.qk_norm_rope_append_kv4
    refused("k_cache", fused, qkv, 2, 1, idx, idx, rope, None, None, kc, vc)
    refused("whole rows", fused, qkv[:, :700], 2, 2, idx, idx, rope, None, None, kc, vc)
    refused("rope", fused, qkv, 2, 2, idx, idx, rope.double(), None, None, kc, vc)
    refused("positions", fused, qkv, 2, 2, idx[:1], idx, rope, None, None, kc, vc)
    refused("k_norm_w", fused, qkv, 2, 2, idx, idx, rope, w, w[:64], kc, vc)
    refused("q_out", fused, qkv, 2, 2, idx, idx, rope, w, w, kc, vc, q_out=qkv)


def test_tensors_made_for_another_stream():
    """Output and workspace of a call on another stream come from that stream:
    the current one is busy, and the memory it had held is full of ones."""
    lens = [700, 30, 4000]
    q, kc, vc, bt, sl = _problem(lens, 32, 8, 1050)
    want = bi.decode_attention_kv4(q, kc, vc, bt, sl, 4000)
    size = bi.decode_attention_workspace_size(3, 32, 128, 4000)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.ones(8192, 8192, device="cuda")
    for stream in (side, side.cuda_stream):
        dirty = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        del dirty
        for _ in range(3):
            busy @ busy
        got = bi.decode_attention_kv4(q, kc, vc, bt, sl, 4000, stream=stream)
        side.synchronize()
        bi.get_device_error(side)
        assert np.array_equal(bits(got), bits(want))
