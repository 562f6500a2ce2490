"""The 8-bit calls' two ways from Python: compiled where all outputs are given and the stream
is the current one, in Python for the rest.  They take and refuse the same, and give the same bits."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_gb300 as bi
from invariant_bi_rmsnorm_gb300 import _lib
from tests._util import bits

pytestmark = pytest.mark.gpu

F8, BF, U8 = torch.float8_e4m3fn, torch.bfloat16, torch.uint8
ROWS, N, F, K = 37, 136, 144, 528


def empty(shape, t):
    return torch.zeros(shape, dtype=U8 if t is F8 else t, device="cuda").view(t) if t is F8 else torch.zeros(shape, dtype=t, device="cuda")


def matrix(rows, cols):
    return [empty((rows, cols), F8), empty(bi.fp8_scales_shape(rows, cols), U8)]


def args_of(name, rows=ROWS):
    """(function, positional arguments, outputs by name) of a call, fresh each time."""
    g = torch.Generator(device="cuda").manual_seed(5)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    x, q8 = normal(rows, K), lambda r, c: list(bi.quantize_fp8(normal(r, c)))  # noqa: E731
    out, scales = matrix(rows, K)
    if name == "quantize_fp8":
        return bi.quantize_fp8, [x], {"out": out, "scales": scales}
    if name == "fp8_read":
        return bi.fp8_read, q8(rows, K), {"out": empty((rows, K), BF)}
    if name == "rmsnorm_fp8":
        return bi.rmsnorm_fp8, [x, normal(K), 1e-6], {"out": out, "scales": scales}
    if name == "add_rmsnorm_fp8":
        return bi.add_rmsnorm_fp8, [x, normal(rows, K), normal(K), 1e-6], {"residual_out": empty((rows, K), BF), "out": out, "scales": scales}
    if name == "gemm_fp8":
        return bi.gemm_fp8, q8(rows, K) + q8(N, K), {"out": empty((rows, N), BF)}
    h, hs = matrix(rows, F)
    return bi.gemm_fp8_swiglu, q8(rows, K) + q8(2 * F, K), {"out": h, "scales": hs}


NAMES = ["quantize_fp8", "fp8_read", "rmsnorm_fp8", "add_rmsnorm_fp8", "gemm_fp8", "gemm_fp8_swiglu"]


class Counted:
    """_lib.fp8_calls with the statuses it gave."""

    def __init__(self, calls):
        self.calls, self.statuses = calls, []

    def __getattr__(self, name):
        def call(*a):
            self.statuses.append(getattr(self.calls, name)(*a))
            return self.statuses[-1]
        return call


@pytest.fixture
def counted(monkeypatch):
    _lib.load()
    c = Counted(_lib.fp8_calls)
    monkeypatch.setattr(_lib, "fp8_calls", c)
    return c


def both(name, change, counted, rows=ROWS):
    """What the compiled call and the Python one give or raise: (results, whether compiled made it)."""
    got = []
    for stream in (None, torch.cuda.current_stream()):
        f, a, outs = args_of(name, rows)
        change(a, outs)
        counted.statuses.clear()
        try:
            f(*a, **outs, stream=stream)
            torch.cuda.synchronize()
            got.append({k: bits(v) if v.dtype is BF else v.view(U8).cpu().numpy() for k, v in outs.items()})
        except (ValueError, bi.BiError) as e:
            got.append((type(e), str(e)))
        if stream is None:
            assert len(counted.statuses) == 1
            made = counted.statuses[0] >= 0
        else:
            assert not counted.statuses
    return got, made


@pytest.mark.parametrize("rows", [1, ROWS, 129])
@pytest.mark.parametrize("name", NAMES)
def test_the_same_bits(name, rows, counted):
    (a, b), made = both(name, lambda a, o: None, counted, rows)
    assert made and isinstance(a, dict)
    for k in a:
        assert np.array_equal(a[k], b[k]), k
    bi.get_device_error()


def strided(t):
    """t's values in rows that lie 32 elements further apart."""
    wide = torch.zeros(t.shape[0], t.shape[1] + 32, dtype=torch.uint8 if t.dtype is F8 else t.dtype, device=t.device)
    wide = wide.view(t.dtype) if t.dtype is F8 else wide
    view = wide[:, :t.shape[1]]
    view.view(U8 if t.dtype is F8 else t.dtype).copy_(t.view(U8 if t.dtype is F8 else t.dtype))
    return view


@pytest.mark.parametrize("name", NAMES)
def test_strided_rows(name, counted):
    def change(a, o):
        for i, t in enumerate(a):
            if torch.is_tensor(t) and t.dim() == 2 and t.dtype is not U8:
                a[i] = strided(t)
        for k, t in o.items():
            if t.dim() == 2 and t.dtype is not U8:
                o[k] = strided(t)
    (a, b), made = both(name, change, counted)
    plain, _ = both(name, lambda a, o: None, counted)
    assert made and isinstance(a, dict)
    for k in a:
        assert np.array_equal(a[k], b[k]) and np.array_equal(a[k], plain[0][k]), k
    bi.get_device_error()


WRONG = {
    "on the CPU": lambda t: t.cpu(),
    "another type": lambda t: t.float() if t.dtype is BF else t.view(torch.int8),
    "a row more": lambda t: torch.cat([t, t[:1]]) if t.dtype is not F8 else torch.cat([t.view(U8), t.view(U8)[:1]]).view(F8),
    "a column less": lambda t: t[..., :-16],
    "a dimension more": lambda t: t[None],
    "columns apart": lambda t: torch.stack([t, t], -1)[..., 0] if t.dtype is not F8 else torch.stack([t.view(U8)] * 2, -1).view(F8)[..., 0],
}


@pytest.mark.parametrize("how", list(WRONG))
@pytest.mark.parametrize("name", NAMES)
def test_the_same_refusals(name, how, counted):
    """Every tensor of the call in turn is wrong in one way.  (x alone may have another row count
    or K: then the others no longer fit.)"""
    _, a, outs = args_of(name)
    where = [("a", i) for i, t in enumerate(a) if torch.is_tensor(t)] + [("o", k) for k in outs]
    for kind, key in where:
        def change(a, o):
            into = a if kind == "a" else o
            into[key] = WRONG[how](into[key])
        (x, y), made = both(name, change, counted)
        assert isinstance(x, tuple) and x == y, f"{kind} {key}: {x}, {y}"
    bi.get_device_error()


@pytest.mark.parametrize("name", NAMES)
def test_the_same_errors_of_the_library(name, counted):
    """A status, not a refusal: codes that do not start on 16 bytes."""
    def change(a, o):
        key = "out" if name != "fp8_read" else None
        t = o["out"] if key else a[0]
        size = t.element_size()
        room = torch.zeros(t.numel() * size + 16, dtype=U8, device="cuda")[8:8 + t.numel() * size]
        t = room.view(t.dtype).view(t.shape)
        if key:
            o["out"] = t
        else:
            a[0] = t
    (x, y), made = both(name, change, counted)
    assert made and x == y and x[0] is bi.BiError, (x, y)
    bi.get_device_error()


def test_the_current_stream_is_the_call_s(counted):
    """Behind work that takes a while on a side stream, and captured."""
    f, a, outs = args_of("gemm_fp8")
    want = bits(f(*a))
    side = torch.cuda.Stream()
    x = torch.zeros_like(a[0].view(U8))
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        x.copy_(a[0].view(U8))
        f(x.view(F8), *a[1:], **outs)
    assert counted.statuses == [0]
    side.synchronize()
    assert np.array_equal(bits(outs["out"]), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f(x.view(F8), *a[1:], **outs)
    outs["out"].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert counted.statuses == [0, 0] and np.array_equal(bits(outs["out"]), want)
    bi.get_device_error()
