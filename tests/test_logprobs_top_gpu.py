"""bi_logprobs_top against fp64: ids exactly, numbers within fp32's error.

Tolerances.  lse and log-probabilities within bi_logprobs' 1e-4 + 1e-6 |ref|,
and its bits for logits within +-1024.  Entropy = ln S - ln 2 T / S, nothing cancels: S
and T are sums of at most 594 terms a thread and 256 threads, each addition
within 2^-24 of a partial sum that its total bounds, so |dS / S| and |dT / T|
<= 602 * 2^-24 + 2^-21 (ex2, and the rounding of its argument up to 127 * 2^-24
for terms that count) < 1e-4 / 2; both |ln S| and |T / S| ln 2 are at most the
entropy: |got - ref| <= 1e-4 + 1e-4 ref."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import inputs


pytestmark = pytest.mark.gpu

V = 151936


def _reference(x, k):
    """(lse, entropy, ids, values) in fp64 of a bf16 CPU tensor [rows, vocab]."""
    d = x.double().numpy()
    m = d.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        lse = m[:, 0] + np.log(np.exp(d - m).sum(1))
        lp = d - lse[:, None]
        p = np.exp(lp)
        h = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(1)
    ids = np.argsort(-d, axis=1, kind="stable")[:, :k]
    return lse, h, ids, np.take_along_axis(d, ids, 1)


def _check(x, k, targets=None):
    xd = x.cuda()
    t = targets if targets is not None else torch.arange(x.shape[0], dtype=torch.int32) % x.shape[1]
    lp, lse, h, ids, top = bi.logprobs_top(xd, t.cuda(), k)
    lp0, lse0 = bi.logprobs(xd, t.cuda())
    near = ((x.float().abs() <= 1024) | (x == float("-inf"))).all(1)
    for got, other in ((lse, lse0), (lp, lp0)):
        assert torch.equal(got.cpu().view(torch.int32)[near], other.cpu().view(torch.int32)[near])
    rlse, rh, rids, rval = _reference(x, k)
    for got, ref in ((lse, rlse), (lp, x.double().numpy()[np.arange(len(x)), t.numpy()] - rlse)):
        assert (np.abs(got.cpu().double().numpy() - ref) <= 1e-4 + 1e-6 * np.abs(ref)).all()
    assert np.array_equal(ids.cpu().numpy(), rids)
    hd = h.cpu().double().numpy()
    assert (np.abs(hd - rh) <= 1e-4 + 1e-4 * np.abs(rh)).all(), np.abs(hd - rh).max()
    # exactly x - lse in fp32
    want = rval.astype(np.float32) - lse.cpu().numpy()[:, None]
    assert np.array_equal(top.cpu().numpy(), want, equal_nan=True)
    bi.get_device_error()


@pytest.mark.parametrize("vocab,k", [(8, 1), (8, 8), (32, 32), (40, 7), (256, 20), (2040, 5), (2048, 32),
                                     (2056, 20), (8192, 1), (65544, 20), (V, 20), (V, 32)])
def test_ordinary_rows(vocab, k):
    _check(inputs.normal_bf16((5, vocab), seed=1100 + k, std=2.0), k)


@pytest.mark.parametrize("vocab", [304, 4096, V])
def test_rows_with_an_order_or_ties(vocab):
    """Constant rows, rising and falling ones, few distinct values, both zeros,
    large values in one thread's vectors only, one value far above the rest."""
    g = torch.Generator().manual_seed(1110)
    j = torch.arange(vocab, dtype=torch.float32)
    rows = torch.zeros(11, vocab)
    rows[0] = 1.5
    rows[1] = j / 64
    rows[2] = -j / 64
    rows[3] = torch.randint(0, 3, (vocab,), generator=g).float()
    rows[4] = torch.where(torch.rand(vocab, generator=g) < 0.5, 0.0, -0.0)
    rows[5] = torch.randn(vocab, generator=g)
    rows[5, (torch.arange(vocab) % 2048) < 8] += 40.0   # one thread of 256 holds every large value
    rows[6] = torch.randn(vocab, generator=g)
    rows[6, vocab // 3] = 300.0
    rows[7] = torch.randn(vocab, generator=g)
    rows[7, (torch.arange(vocab) % 2048) < 16] = 7.0    # ties by the hundred, in two threads
    rows[8] = -1e30
    rows[8, vocab - 1] = 3e38
    rows[9] = 0.25
    rows[9, -9:] = 0.5                                  # the ties that count lie at the end
    rows[10] = (j % 2048) / 2048
    x = rows.to(torch.bfloat16)
    _check(x, 20)
    x[8, vocab - 1] = 1.5e38
    _check(x[8:9], 20)


@pytest.mark.parametrize("vocab", [64, 5000 * 8, V])
def test_masked_rows(vocab):
    """-inf logits: all but one, all but fewer than k, all but some, the first
    or the last half."""
    g = torch.Generator().manual_seed(1120)
    x = torch.randn(6, vocab, generator=g) * 3
    x[0] = float("-inf")
    x[0, vocab // 2 + 1] = -2.0
    keep = torch.randperm(vocab, generator=g)[:5]
    row = x[1].clone()
    x[1] = float("-inf")
    x[1, keep] = row[keep]
    x[2, torch.rand(vocab, generator=g) < 0.9] = float("-inf")
    x[3, :vocab // 2] = float("-inf")
    x[4, vocab // 2:] = float("-inf")
    x = x.to(torch.bfloat16)
    t = torch.tensor([vocab // 2 + 1, int(keep[0]), 3, vocab - 1, 0, 7], dtype=torch.int32)
    t[2] = int((x[2] != float("-inf")).nonzero()[0])
    _check(x, 20, t)
    for mask in (-1e9, -1e30, torch.finfo(torch.bfloat16).min):  # masks of finite values
        _check(torch.where(x == float("-inf"), torch.tensor(mask, dtype=torch.bfloat16), x), 20, t)


def test_rows_without_a_number():
    """Nothing visible, NaN among the logits, nothing but NaN, an infinity."""
    vocab = 4096
    x = inputs.normal_bf16((5, vocab), seed=1130)
    x[0] = float("-inf")
    x[1, 100] = float("nan")
    x[1, 3000] = 50.0
    x[2] = float("nan")
    x[3, 77] = float("inf")
    x[4, 10:] = float("nan")   # ten numbers, then NaN: they rank last, by id
    lp, lse, h, ids, top = [t.cpu() for t in bi.logprobs_top(x.cuda(), torch.zeros(5, dtype=torch.int32).cuda(), 20)]
    assert lse[0] == float("-inf") and torch.isnan(lse[1:]).all()
    assert torch.isnan(h).all() and torch.isnan(top).all()
    assert ids[0].tolist() == list(range(20)) and ids[2].tolist() == list(range(20))
    assert ids[1, 0] == 3000 and 100 not in ids[1].tolist()
    assert ids[3, 0] == 77
    ten = torch.argsort(-x[4, :10].double(), stable=True).tolist()
    assert ids[4].tolist() == ten + list(range(10, 20))
    bi.get_device_error()


def test_rows_alone_batched_and_strided():
    x = inputs.normal_bf16((9, V + 64), seed=1140, std=2.0).cuda()
    t = torch.arange(9, dtype=torch.int32, device="cuda") * 1000
    a = bi.logprobs_top(x[:, :V], t, 20)
    for r in (0, 4, 8):
        b = bi.logprobs_top(x[r:r + 1, :V], t[r:r + 1], 20)
        assert all(torch.equal(p[r:r + 1], q) for p, q in zip(a, b))
    few = bi.logprobs_top(x[:, :V], None, 3)
    assert few[0] is None and torch.equal(few[3], a[3][:, :3]) and torch.equal(few[4], a[4][:, :3])


def test_many_rows_and_a_wide_vocabulary():
    """More than 2^31 logits, whose last rows lie past 32-bit offsets; a
    vocabulary with more than one round of vectors in every segment."""
    rows = 2 ** 31 // V + 40
    x = torch.empty(rows, V, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1145))
    a = bi.logprobs_top(x, None, 4)
    for r in (0, rows // 2, rows - 1):
        assert all(torch.equal(p[r:r + 1], q) for p, q in zip(a[1:], bi.logprobs_top(x[r:r + 1].clone(), None, 4)[1:]))
    del x
    _check(inputs.normal_bf16((2, 1_310_728), seed=1146, std=2.0), 32)


def test_a_captured_call_and_other_streams():
    x = inputs.normal_bf16((6, 8000), seed=1150).cuda()
    t = torch.arange(6, dtype=torch.int32, device="cuda")
    bi.logprobs_top(x, t, 8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bi.logprobs_top(x, t, 8)
    side = torch.cuda.Stream()
    for seed in (1151, 1152):
        x.copy_(inputs.normal_bf16((6, 8000), seed=seed))
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            other = bi.logprobs_top(x, t, 8)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, other))


def test_refusals_and_bad_targets():
    x = inputs.normal_bf16((2, 1024), seed=1160).cuda()
    lp, *_ = bi.logprobs_top(x, torch.tensor([3, 5000], dtype=torch.int32, device="cuda"), 4)
    with pytest.raises(bi.BiError, match="BAD_INPUT"):
        bi.get_device_error()
    assert torch.isnan(lp[1]) and not torch.isnan(lp[0])
    for k in (33, 2000):
        with pytest.raises(bi.BiError, match="UNSUPPORTED"):
            bi.logprobs_top(x, None, k)
    with pytest.raises(ValueError, match="at least 1"):
        bi.logprobs_top(x, None, 0)
    with pytest.raises(ValueError, match="targets"):
        bi.logprobs_top(x, torch.zeros(3, dtype=torch.int32, device="cuda"), 4)
    assert bi.logprobs_top(x[:0], None, 4)[3].shape == (0, 4)


def test_bits_do_not_depend_on_the_call():
    x = inputs.normal_bf16((64, V), seed=1170, std=3.0).cuda()
    a = bi.logprobs_top(x, None, 20)
    for _ in range(3):
        b = bi.logprobs_top(x, None, 20)
        assert all(torch.equal(p, q) for p, q in zip(a[1:], b[1:]))
