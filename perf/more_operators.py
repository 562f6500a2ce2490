"""What the 8-bit linear path is measured on.

Each case is one call, or one run of calls, that a forward step makes:

  norm     rmsnorm_fp8 or add_rmsnorm_fp8, then fp8_read: the norm with an output in 8 bits, read back
  linear   quantize_fp8, then gemm_fp8: a projection of activations that no norm produced (attention's output)
  project  rmsnorm_fp8 or add_rmsnorm_fp8, then gemm_fp8: the norm and the projection behind it
  mlp      add_rmsnorm_fp8, gemm_fp8_swiglu, gemm_fp8: a decoder layer's whole feed-forward block

The format: 128 consecutive values of a row (the last block of a row may be shorter) are held as e4m3
numbers q and one scale 2^(b - 127), b a byte, and stand for q * 2^(b - 127).  b is the least that keeps
max|x| within 448 scales, 8 at least; q is x / scale rounded to nearest even.  Scales lie in tiles of
128 rows by 4 blocks, [ceil(rows / 128), ceil(K / 512), 512] bytes: that of row r's block c is byte
16 (r % 32) + 4 (r % 128 // 32) + c % 4 of tile [r // 128, c // 4].
"""
import math

import torch

own = False

BLOCK, ATOM, EPS = 128, 512, 1e-6
HIDDEN, FFN, QKV = 4096, 12288, 6144


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one token's row: latency is all there is
        {"name": "norm 1 x 4096", "op": "norm", "M": 1, "K": HIDDEN, "add": False},
        # a long prompt's rows, residual added
        {"name": "norm 16384 x 4096", "op": "norm", "M": 16384, "K": HIDDEN, "add": True},
        # one token's attention output through the output projection
        {"name": "linear 1", "op": "linear", "M": 1, "N": HIDDEN, "K": HIDDEN},
        # odd sizes: a block and a scale tile that end short, output tiles that end inside
        {"name": "linear 37 x 1000 x 2064", "op": "linear", "M": 37, "N": 1000, "K": 2064},
        # a few short prompts, between a decode batch and a whole step
        {"name": "linear 300", "op": "linear", "M": 300, "N": HIDDEN, "K": HIDDEN},
        # a step's whole token budget
        {"name": "linear 8192", "op": "linear", "M": 8192, "N": HIDDEN, "K": HIDDEN},
        # a decode batch: the first layer's norm, then the query, key and value projections
        {"name": "project 64", "op": "project", "M": 64, "N": QKV, "K": HIDDEN, "add": False},
        {"name": "project 4096", "op": "project", "M": 4096, "N": QKV, "K": HIDDEN, "add": True},
        # the feed-forward block for one user, for a small batch, for a ragged prompt and for a whole step
        {"name": "mlp 1", "op": "mlp", "M": 1, "K": HIDDEN, "F": FFN},
        {"name": "mlp 24", "op": "mlp", "M": 24, "K": HIDDEN, "F": FFN},
        {"name": "mlp 511", "op": "mlp", "M": 511, "K": HIDDEN, "F": FFN},
        {"name": "mlp 8192", "op": "mlp", "M": 8192, "K": HIDDEN, "F": FFN},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "project", "mlp", "mlp"])
    if op == "norm":
        K = 16 * _log(rng, 1, 1024)
        return {"op": op, "M": _log(rng, 1, min(16384, 16384 * HIDDEN // K)), "K": K, "add": rng.random() < 0.5}
    M = _log(rng, 1, 8192)
    if op == "mlp":
        return {"op": op, "M": M, "K": 16 * _log(rng, 4, HIDDEN // 16), "F": 16 * _log(rng, 4, FFN // 16)}
    case = {"op": op, "M": M, "N": 8 * _log(rng, 4, 16384 // 8), "K": 16 * _log(rng, 1, FFN // 16)}
    return case | {"add": rng.random() < 0.5} if op == "project" else case


def work(c):
    M, K = c["M"], c["K"]
    held = lambda rows, k: rows * k + rows * -(-k // BLOCK)  # 8-bit values and their scales  # noqa: E731
    x = M * K * 2 * (3 if c.get("add", c["op"] == "mlp") else 1) + (2 * K if c["op"] != "linear" else 0)
    if c["op"] == "norm":
        return {"bytes": x + M * K * 2, "flops": 6 * M * K}
    if c["op"] == "mlp":
        F = c["F"]
        return {"bytes": x + held(2 * F, K) + held(K, F) + M * K * 2, "flops": 2 * M * K * 3 * F}
    return {"bytes": x + held(c["N"], K) + M * c["N"] * 2, "flops": 2 * M * K * c["N"]}


# ------------------------------------------------------------- the 8-bit format ----
def _blocks(x):
    """x [rows, K] as fp32 blocks [rows, ceil(K / 128), 128], zeros behind a row's end."""
    x = x.float()
    return torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))


def _quantise(x):
    """Values q [rows, blocks, 128] (fp32, each an e4m3 number) and scale bytes b [rows, blocks]."""
    g = _blocks(x)
    top = g.abs().amax(-1).view(torch.int32)
    b = (((top + 0x1FFFFF) >> 23) - 8).clamp(min=8)  # carries where the mantissa is above 1.75: 448 = 1.75 * 2^8
    q = (g * ((254 - b) << 23).view(torch.float32)[..., None]).to(torch.float8_e4m3fn).float()
    return q, b


def _values(q, b, K):
    return (q * (b << 23).view(torch.float32)[..., None]).flatten(1)[:, :K]


def _pack(b):
    """Scale bytes [rows, blocks] -> tiles [ceil(rows / 128), ceil(blocks / 4), 512] uint8."""
    rows, n = b.shape
    b = torch.nn.functional.pad(b, (0, -n % 4, 0, -rows % 128)).to(torch.uint8)
    return b.view(-(-rows // 128), 4, 32, -(-n // 4), 4).permute(0, 3, 2, 1, 4).reshape(-(-rows // 128), -(-n // 4), 512).contiguous()


def _read(q, tiles):
    """What an 8-bit matrix (q [rows, K] e4m3, scale tiles) stands for, fp32 [rows, K]."""
    rows, K = q.shape
    R, S, _ = tiles.shape
    b = tiles.view(R, S, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, S * 4)[:rows, :-(-K // BLOCK)].to(torch.int32)
    return _values(_blocks(q), b, K)


# ------------------------------------------------------------------ inputs ----
def _weight(n, k, gen, device):
    """A weight [n, k] ~ N(0, 0.02) held in 8 bits, as a program has it from its checkpoint."""
    q, b = _quantise((torch.randn(n, k, generator=gen, device=device) * 0.02).to(torch.bfloat16))
    return q.flatten(1)[:, :k].to(torch.float8_e4m3fn).contiguous(), _pack(b)


def _interleaved(w):
    """Gate rows, then up rows -> groups of 8 gate rows with the 8 matching up rows behind them."""
    return w.unflatten(0, (2, -1, 8)).transpose(0, 1).flatten(0, 2).contiguous()


def _tiles_shape(rows, k):
    return -(-rows // 128), -(-k // ATOM), 512


def prepare(c, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=device)  # noqa: E731
    st = dict(c)
    M, K = c["M"], c["K"]
    x = normal(M, K)
    if c["op"] == "linear":
        # attention's output: heads of their own size
        x = x * torch.exp(0.5 * normal(1, -(-K // 128))).repeat_interleave(128, 1)[:, :K]
    else:
        # one value in a hundred stands out, as in a residual stream
        x = torch.where(torch.rand(M, K, generator=gen, device=device) < 0.01, 100 * x, x)
        st["w"] = (1 + 0.1 * normal(K)).to(torch.bfloat16)
    st["x"] = x.to(torch.bfloat16)
    st["add"] = c.get("add", c["op"] == "mlp")
    empty = lambda shape, t: torch.empty(shape, dtype=t, device=device)  # noqa: E731
    if st["add"]:
        st["residual"] = (4 * normal(M, K)).to(torch.bfloat16)
        st["residual_out"] = torch.empty_like(st["residual"])
    st["q"], st["qs"] = empty((M, K), torch.float8_e4m3fn), empty(_tiles_shape(M, K), torch.uint8)
    if c["op"] == "norm":
        st["out"] = empty((M, K), torch.bfloat16)
    elif c["op"] == "mlp":
        F = c["F"]
        q, b = _quantise(_interleaved((normal(2 * F, K) * 0.02).to(torch.bfloat16)))
        st["W_gu"] = q.flatten(1)[:, :K].to(torch.float8_e4m3fn).contiguous(), _pack(b)
        st["W_down"] = _weight(K, F, gen, device)
        st["h"], st["hs"] = empty((M, F), torch.float8_e4m3fn), empty(_tiles_shape(M, F), torch.uint8)
        st["out"] = empty((M, K), torch.bfloat16)
    else:
        st["W"] = _weight(c["N"], K, gen, device)
        st["out"] = empty((M, c["N"]), torch.bfloat16)
    return st


# ------------------------------------------------------------- plain forms ----
def _held(x):
    """x as 8 bits hold it."""
    return _values(*_quantise(x), x.shape[1])


def _plain_norm(st):
    x, res = st["x"].float(), None
    if st["add"]:
        res = (x + st["residual"].float()).to(torch.bfloat16)
        x = res.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * st["w"].float()
    return _held(n), res


def run(st):
    op = st["op"]
    if own:
        return _run_own(st)
    if op == "linear":
        return {"y": torch.matmul(_held(st["x"]), _read(*st["W"]).t()).to(torch.bfloat16)}
    n, res = _plain_norm(st)
    if op == "norm":
        y = n
    elif op == "project":
        y = torch.matmul(n, _read(*st["W"]).t())
    else:
        gu = torch.matmul(n, _read(*st["W_gu"]).t()).unflatten(1, (-1, 2, 8))
        g, u = gu[:, :, 0].flatten(1), gu[:, :, 1].flatten(1)
        y = torch.matmul(_held(g / (1 + torch.exp(-g)) * u), _read(*st["W_down"]).t())
    return {"y": y.to(torch.bfloat16)} | ({"residual": res} if st["add"] else {})


def _run_own(st):
    import invariant_bi_rmsnorm_gb300 as bi
    op, x, out = st["op"], st["x"], {"y": st["out"]}
    if op == "linear":
        q, qs = bi.quantize_fp8(x, out=st["q"], scales=st["qs"])
        bi.gemm_fp8(q, qs, *st["W"], out=st["out"])
        return out
    if st["add"]:
        out["residual"] = st["residual_out"]
        q, qs = bi.add_rmsnorm_fp8(x, st["residual"], st["w"], EPS, residual_out=st["residual_out"], out=st["q"],
                                   scales=st["qs"])
    else:
        q, qs = bi.rmsnorm_fp8(x, st["w"], EPS, out=st["q"], scales=st["qs"])
    if op == "norm":
        bi.fp8_read(q, qs, out=st["out"])
    elif op == "project":
        bi.gemm_fp8(q, qs, *st["W"], out=st["out"])
    else:
        h, hs = bi.gemm_fp8_swiglu(q, qs, *st["W_gu"], out=st["h"], scales=st["hs"])
        bi.gemm_fp8(h, hs, *st["W_down"], out=st["out"])
    return out


# ---------------------------------------------------- the definition, in 64 bits ----
def _two_to(e):
    """2^e for whole numbers e from -1022 to 1023, fp64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _held64(x):
    """What rows x are held as, in 64 bits: block by block, powers of two and rounding by the definition."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[1], BLOCK):
        g = x[:, at:at + BLOCK].double()
        m, e = torch.frexp(g.abs().amax(-1, keepdim=True))  # m in [0.5, 1): 448 = 0.875 * 2^9
        scale = _two_to(torch.clamp(torch.where(m > 0.875, e - 8, e - 9), min=-119))
        v = g / scale
        _, e = torch.frexp(v)
        step = _two_to(torch.clamp(e - 1, min=-6) - 3)  # four significant bits, subnormals below 2^-6
        out[:, at:at + BLOCK] = torch.round(v / step) * step * scale
    return out


def _read64(q, tiles):
    """An 8-bit matrix from its bytes by the format's formula."""
    rows, K = q.shape
    c = q.view(torch.uint8).to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _two_to(e - 10))
    r = torch.arange(rows, device=q.device)[:, None]
    k = torch.arange(K, device=q.device) // BLOCK
    b = tiles[r // 128, k // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + k % 4]
    return torch.where(c >= 128, -mag, mag) * _two_to(b.long() - 127)


def exact(c, seed):
    st = prepare(c, seed)
    x = st["x"].double()
    if c["op"] == "linear":
        return {"y": _held64(x) @ _read64(*st["W"]).t()}
    res = {}
    if st["add"]:
        x = (x + st["residual"].double()).to(torch.bfloat16).double()
        res = {"residual": x}
    n = _held64(x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS) * st["w"].double())
    if c["op"] == "norm":
        y = n
    elif c["op"] == "project":
        y = n @ _read64(*st["W"]).t()
    else:
        W = _read64(*st["W_gu"])
        row = torch.arange(W.shape[0], device=W.device)
        g, u = n @ W[row % 16 < 8].t(), n @ W[row % 16 >= 8].t()
        del W
        y = _held64(g * torch.sigmoid(g) * u) @ _read64(*st["W_down"]).t()
    return {"y": y} | res
