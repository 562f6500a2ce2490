"""The entropy of bi_logprobs_top where a row's parts have different maxima.

d = x log2(e) - m log2(e) is formed with a rounded m log2(e), up to 2^-14 off at
|m| = 1024 and differently for every maximum, so the parts of a row that were
formed under different ones have to be brought together by more than 2^((m - m')
log2(e)).

Tolerance.  H = ln S - ln 2 T / S with S and T sums of terms of one sign.  Let
every term be within a factor 1 + e of its value:
    (V / 256 + 12) 2^-24   additions: V / 256 a thread, 5 in a warp, 7 of warps
    moves * 2^-21          a rescaling that is not by 1: exp2f 2^-22, its three
                           products and sums 2^-24 each, and 2^-24 to spare
    2^-22                  ex2.approx of the term
    2^-23 R                the exponents' roundings, 2^-24 of each, and that of
                           log2(e), 2^-25.9 of each: they add up to R nats at most,
                           the row's range
    2^-18 ln 2             between parts with maxima within +-44, whose roundings
                           (2^-19 each) are left in
Then S and T are within a factor 1 + e, T / S within 1 + 2e, and, |T / S| ln 2
being at most H and the division, the product and the difference costing 2^-23 of
H together, |got - H| <= e + (2e + 2^-22) H.  For 2047 values and one 8 above
them that is 4.8e-5; with larger maxima's roundings left in too it is 8.8e-5 off."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi

pytestmark = pytest.mark.gpu


def _entropy(x):
    d = x.double().numpy()
    d = d - d.max(1, keepdims=True)
    p = np.exp(d)
    s = p.sum(1)
    return np.log(s) - (p * d).sum(1) / s


def _check(rows, moves):
    x = torch.stack(rows).to(torch.bfloat16)
    assert torch.equal(x.double(), torch.stack(rows).double())  # bf16 numbers, all of them
    V = x.shape[1]
    t = torch.zeros(len(rows), dtype=torch.int32, device="cuda")
    lp, lse, h, *_ = bi.logprobs_top(x.cuda(), t, 1)
    lp0, lse0 = bi.logprobs(x.cuda(), t)
    assert torch.equal(lp, lp0) and torch.equal(lse, lse0)
    ref = _entropy(x)
    R = (x.double().amax(1) - x.double().amin(1)).numpy()
    e = (V / 256 + 12) * 2.0 ** -24 + moves * 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -23 * R + 2.0 ** -18 * np.log(2)
    off = np.abs(h.cpu().double().numpy() - ref)
    assert (off <= e + (2 * e + 2.0 ** -22) * ref).all(), (off / (e + (2 * e + 2.0 ** -22) * ref)).max()
    bi.get_device_error()


BASES = [1012, 996, 928, 700, 520, 40, 0, -44, -520, -704, -928, -1008]


@pytest.mark.parametrize("V", [2048, 8192, 151936])
@pytest.mark.parametrize("gap", [4, 8, 12])
def test_one_logit_above_the_rest(V, gap):
    """In the first vector, in the last, in a thread's middle: the others' maximum
    moves at one point, within their thread or where threads meet."""
    rows = []
    for b in BASES:
        for at in (5, V // 2 + 1, V - 1):
            r = torch.full((V,), float(b))
            r[at] += gap
            rows.append(r)
    _check(rows, 1)


@pytest.mark.parametrize("V", [2048, 8192, 151936])
def test_threads_of_four_maxima(V):
    thread = torch.arange(V) // 8 % 256
    _check([b - 4.0 * (thread * 7 % 4) for b in BASES], 3)


@pytest.mark.parametrize("V", [8192, 16384])
def test_maxima_that_climb_and_fall(V):
    """Vector after vector: the maximum moves in every thread and every vector, or
    in the first alone."""
    vector = torch.arange(V) // 2048
    n = V // 2048 - 1
    bases = BASES[:-1]  # down to -956, within +-1024
    _check([b - 4.0 * (n - vector) for b in bases] + [b - 4.0 * vector for b in bases], n)
