"""What the 4-bit KV cache and the per-token log-prob report are measured on.

Each case is one call, or one run of calls, that a serving step makes:

  decode   decode_attention_kv4: one query row per sequence over a cache held in 4 bits
  step     qk_norm_rope_append_kv4, then decode_attention_kv4: a decode step's path through one layer
  prompt   qk_norm_rope_append_kv4, kv4_read, prefill_attention: a prompt step's path through one layer
  write    kv4_append, then kv4_read: keys and values computed elsewhere, written and read back
  report   logprobs_top: log-probability of the chosen token, entropy, top alternatives

The format of the cache: a group of 32 consecutive dims of one token and kv-head is held as 4-bit
codes n + 8, n in -7 .. 7, and a scale s, a bf16 number of 4 significant bits, and stands for n * s.
A (page, kv-head) block of K or V has 1152 bytes: the codes of its 16 tokens, 64 bytes each, then 16
rows of 4 scales.  Codes lie in little-endian 32-bit words of 8, code i at bits 4i .. 4i + 3.  Dim
d = 32j + 8p + 2t + e (p, t < 4, e < 2) of token r of K is code p + 4e of word 16r + 4t + j; dim
d = 64w + 32h + 8p + g (g < 8) of token r = 8a + 2b + c (c < 2) of V is code 4h + p of word
128a + 16g + 4b + 2c + w.
"""
import math

import torch

own = False

PAGE, D, GROUP = 16, 128, 32
RECORD = PAGE * 64 + PAGE * 8  # bytes of one (page, kv-head) block of K or of V
THETA, EPS = 1e6, 1e-6
VOCAB = 151936
HEADS = [(32, 8), (28, 4), (16, 2), (8, 1), (5, 5), (64, 8)]


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one user with a long context: a few warps per sequence must find all of the bandwidth
        {"name": "decode 1 x 8192", "op": "decode", "B": 1, "lo": 8192, "hi": 8192, "Hq": 32, "Hkv": 8},
        # odd head counts, lengths from one token on, pages that end inside every chunk
        {"name": "decode 17 x 1-3001", "op": "decode", "B": 17, "lo": 1, "hi": 3001, "Hq": 28, "Hkv": 4},
        # an ordinary serving batch
        {"name": "decode 64 x 1-8192", "op": "decode", "B": 64, "lo": 1, "hi": 8192, "Hq": 32, "Hkv": 8},
        # the largest batch that the decoder's step graphs hold
        {"name": "decode 256 x 1-8192", "op": "decode", "B": 256, "lo": 1, "hi": 8192, "Hq": 32, "Hkv": 8},
        # a short chat: latency is all there is
        {"name": "step 1 x 300", "op": "step", "B": 1, "lo": 300, "hi": 300, "Hq": 32, "Hkv": 8},
        {"name": "step 24 x 37-2048", "op": "step", "B": 24, "lo": 37, "hi": 2048, "Hq": 32, "Hkv": 8},
        # a step's budget filled with short prompts
        {"name": "prompt 29 x 32-512", "op": "prompt", "S": 29, "past": 0, "lo": 32, "hi": 512, "Hq": 32, "Hkv": 8},
        # one chunk of a long prompt, after what was cached before it
        {"name": "prompt 1 x 511 after 6000", "op": "prompt", "S": 1, "past": 6000, "lo": 511, "hi": 511, "Hq": 32, "Hkv": 8},
        # a handful of tokens, and a step's whole token budget
        {"name": "write 37", "op": "write", "S": 3, "lo": 1, "hi": 24, "Hq": 5, "Hkv": 5},
        {"name": "write 8192", "op": "write", "S": 16, "lo": 64, "hi": 960, "Hq": 32, "Hkv": 8},
        # one sampled token, and the tokens of a scoring pass
        {"name": "report 1", "op": "report", "rows": 1, "vocab": VOCAB, "top": 20},
        {"name": "report 1024", "op": "report", "rows": 1024, "vocab": VOCAB, "top": 20},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "step", "prompt", "write", "report"])
    Hq, Hkv = rng.choice(HEADS)
    if op in ("decode", "step"):
        B = _log(rng, 1, 256)
        hi = _log(rng, 1, min(16384, 1048576 * 32 // (max(32, Hq) * B)))
        return {"op": op, "B": B, "lo": rng.randint(1, hi), "hi": hi, "Hq": Hq, "Hkv": Hkv}
    if op == "prompt":
        S = _log(rng, 1, 32)
        hi = _log(rng, 1, 512)
        most = 250_000_000 // (S * hi * Hq)  # scores of the plain form
        past = rng.choice([0, _log(rng, 1, max(1, min(8192, most - hi)))])
        return {"op": op, "S": S, "past": past, "lo": rng.randint(1, hi), "hi": hi, "Hq": Hq, "Hkv": Hkv}
    if op == "write":
        S = _log(rng, 1, 64)
        hi = _log(rng, 1, 8192 // S)
        return {"op": op, "S": S, "lo": rng.randint(1, hi), "hi": hi, "Hq": Hq, "Hkv": Hkv}
    return {"op": op, "rows": _log(rng, 1, 1024), "vocab": 8 * _log(rng, 4, VOCAB // 8), "top": rng.randint(1, 32)}


def _lens(n, lo, hi):
    """n lengths from lo to hi, evenly spread."""
    return [hi] if n == 1 else [lo + (i * (hi - lo)) // (n - 1) for i in range(n)]


def work(c):
    op = c["op"]
    if op == "report":
        n = c["rows"]
        return {"bytes": n * (2 * c["vocab"] + 4 + 12 + 8 * c["top"]), "flops": 6 * n * c["vocab"]}
    Hq, Hkv = c["Hq"], c["Hkv"]
    row4, row16, width = 144 * Hkv, 512 * Hkv, 256 * (Hq + 2 * Hkv)
    if op in ("decode", "step"):
        lens = _lens(c["B"], c["lo"], c["hi"])
        tokens = sum(lens)
        rest = c["B"] * (2 * 256 * Hq if op == "decode" else width + row4 + 2 * 256 * Hq + 512)
        return {"bytes": tokens * row4 + rest, "flops": 4 * tokens * Hq * D}
    new = _lens(c["S"], c["lo"], c["hi"])
    T = sum(new)
    if op == "write":
        return {"bytes": T * (2 * row16 + 2 * row4), "flops": 8 * T * Hkv * D}
    pairs = sum(n * c["past"] + n * (n + 1) // 2 for n in new)
    return {"bytes": T * (width + row4 + 2 * 256 * Hq + 512) + c["S"] * c["past"] * row4, "flops": 4 * pairs * Hq * D}


# ----------------------------------------------------------- the 4-bit format ----
def _places(device):
    """(word, lowest bit) of token r's dim d, [16, 128] each, in a K block and in a V block."""
    r, d = torch.arange(PAGE, device=device)[:, None], torch.arange(D, device=device)
    p, t, e = (d % 32) // 8, (d % 8) // 2, d % 2
    h = (d // 32) % 2
    return ((16 * r + 4 * t + d // 32, (4 * (p + 4 * e)).expand(PAGE, -1)),
            (128 * (r // 8) + 16 * (d % 8) + 4 * ((r % 8) // 2) + 2 * (r % 2) + d // 64, (4 * (4 * h + p)).expand(PAGE, -1)))


def _quantise(x):
    """Codes n (float) and scales [..., 4] of rows x [..., 128]."""
    g = x.float().unflatten(-1, (4, GROUP))
    amax = g.abs().amax(-1)
    b = (amax / torch.full_like(amax, 7.0)).view(torch.int32)  # a quotient, where a product with 1/7 would miss ties
    s = ((b + 0x7FFFF + ((b >> 20) & 1)) & ~0xFFFFF).view(torch.float32)  # 4 significant bits, nearest even
    s = torch.where(amax < 2.0 ** 123, torch.where(amax < 2.0 ** -120, 0.0, s), math.nan)
    n = torch.round(g / s[..., None]).clamp(-7, 7)
    n = torch.where((s > 0)[..., None], n, 0.0)
    return n.flatten(-2), s


def _values(n, s):
    """What the codes stand for, fp32 [..., 128] (exact in bf16)."""
    return (n.unflatten(-1, (4, GROUP)) * s[..., None]).flatten(-2)


def _pack(x, place):
    """Rows x [pages, Hkv, 16, 128] -> blocks [pages, Hkv, 1152] uint8."""
    n, s = _quantise(x)
    word, bit = place
    order = torch.argsort((word * 32 + bit).flatten())  # (token, dim) by word, then by code
    c = (n.to(torch.int32) + 8).flatten(-2).index_select(-1, order).unflatten(-1, (256, 8))
    w = (c << (4 * torch.arange(8, device=x.device, dtype=torch.int32))).sum(-1).to(torch.int32)
    return torch.cat([w.view(torch.uint8), s.to(torch.bfloat16).contiguous().view(torch.uint8).flatten(-2)], -1)


def _unpack(blocks, place):
    """Blocks [..., 1152] uint8 -> rows [..., 16, 128] fp32."""
    word, bit = place
    w = blocks[..., :1024].view(torch.int32).index_select(-1, word.flatten()).unflatten(-1, (PAGE, D))
    s = blocks[..., 1024:].view(torch.bfloat16).unflatten(-1, (PAGE, 4))
    n = ((w >> bit.to(torch.int32)) & 15) - 8
    return _values(n.float(), s.float())


# ------------------------------------------------------------------ inputs ----
def _pages(lens, gen, device):
    """Pages handed out by a random permutation: block table [n, width] (-1 past a sequence's last page) and their number."""
    need = [-(-n // PAGE) for n in lens]
    perm = torch.randperm(sum(need), generator=gen, device=device).to(torch.int32)
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=device)
    at = torch.arange(max(need), device=device)
    live = at < torch.tensor(need, device=device)[:, None]
    table = torch.where(live, perm[torch.where(live, first[:, None] + at, 0)], -1)
    return table.to(torch.int32).contiguous(), sum(need)


def prepare(c, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=device)  # noqa: E731
    st = dict(c)
    if c["op"] == "report":
        # rows of different sharpness; a few tokens of every other row stand out
        x = normal(c["rows"], c["vocab"]) * (1 + 3 * torch.rand(c["rows"], 1, generator=gen, device=device))
        hot = torch.randint(c["vocab"], (c["rows"], 4), generator=gen, device=device)
        x.scatter_add_(1, hot, 10.0 * (torch.arange(c["rows"], device=device) % 2).float()[:, None].expand(-1, 4).contiguous())
        st["logits"] = x.to(torch.bfloat16)
        pick = torch.randint(c["vocab"], (c["rows"],), generator=gen, device=device)
        st["targets"] = torch.where(torch.arange(c["rows"], device=device) % 2 == 1, hot[:, 0], pick).to(torch.int32)
        return st
    Hq, Hkv = c["Hq"], c["Hkv"]
    mixed = lambda v: [v[i] for i in torch.randperm(len(v), generator=torch.Generator().manual_seed(seed)).tolist()]  # noqa: E731
    if c["op"] in ("decode", "step"):
        lens = mixed(_lens(c["B"], c["lo"], c["hi"]))
        new = [1] * c["B"]
    else:
        new = mixed(_lens(c["S"], c["lo"], c["hi"]))
        lens = [n + c.get("past", 0) for n in new]
    i32 = dict(dtype=torch.int32, device=device)
    st["lens"], st["max_len"], st["max_new"] = torch.tensor(lens, **i32), max(lens), max(new)
    st["table"], pages = _pages(lens, gen, device)
    kplace, vplace = st["places"] = _places(device)
    # keys have channels of their own size, as trained models' have; values do not
    channel = torch.exp(0.5 * normal(Hkv, 1, D))
    if c["op"] == "write":
        st["k_cache"] = torch.zeros(pages, Hkv, RECORD, dtype=torch.uint8, device=device)
        st["v_cache"] = torch.zeros_like(st["k_cache"])
    else:
        st["k_cache"] = _pack((normal(pages, Hkv, PAGE, D) * channel).to(torch.bfloat16), kplace)
        st["v_cache"] = _pack(normal(pages, Hkv, PAGE, D).to(torch.bfloat16), vplace)
    if c["op"] in ("decode", "step"):
        chunks = -(-st["max_len"] // 256)
        size = 262144 + c["B"] * Hq * chunks * (D + 2) * 4 if chunks > 1 else 0
        st["ws"] = torch.zeros(size, dtype=torch.uint8, device=device) if size else None
    if c["op"] == "decode":
        st["q"] = normal(c["B"], Hq, D).to(torch.bfloat16)
        return st
    # the new tokens: the last new[i] of each sequence
    T = sum(new)
    seq = torch.repeat_interleave(torch.arange(len(new), device=device), torch.tensor(new, device=device))
    st["indptr"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], **i32)
    row = torch.arange(T, device=device) - st["indptr"].long()[seq]
    pos = st["lens"].long()[seq] - torch.tensor(new, device=device)[seq] + row
    st["seq"], st["row"] = seq, row
    st["slots"] = (st["table"].long()[seq, pos // PAGE] * PAGE + pos % PAGE).to(torch.int32)
    qkv = normal(T, Hq + 2 * Hkv, D)
    qkv[:, Hq:Hq + Hkv] *= channel[:, 0]
    st["qkv"] = qkv.to(torch.bfloat16).view(T, -1)
    if c["op"] in ("write", "prompt"):
        st["k_out"] = torch.zeros(pages, Hkv, PAGE, D, dtype=torch.bfloat16, device=device)
        st["v_out"] = torch.zeros_like(st["k_out"])
    if c["op"] == "write":
        return st
    st["positions"] = pos.to(torch.int32)
    f = THETA ** (-torch.arange(D // 2, dtype=torch.float64, device=device) / (D // 2))
    ang = torch.arange(st["max_len"], dtype=torch.float64, device=device)[:, None] * f
    st["rope"] = torch.cat([torch.cos(ang), torch.sin(ang)], 1).float()
    st["q_w"] = (1 + 0.1 * normal(D)).to(torch.bfloat16)
    st["k_w"] = (1 + 0.1 * normal(D)).to(torch.bfloat16)
    if c["op"] == "prompt":
        st["pws"] = torch.empty(T * Hq * D * 4, dtype=torch.uint8, device=device) if st["max_len"] > 256 else None
    return st


# ------------------------------------------------------------- plain forms ----
def _norm_rope(x, w, cos, sin):
    """Per-head RMSNorm to bf16, rotate-half RoPE to bf16: x [T, heads, 128]."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    x = x.to(torch.bfloat16).float()
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)


def _new_rows(st):
    """q, k, v of the new tokens, bf16 [T, heads, 128]."""
    Hq, Hkv = st["Hq"], st["Hkv"]
    x = st["qkv"].unflatten(-1, (-1, D))
    rope = st["rope"][st["positions"].long()]
    cos, sin = rope[:, None, :64], rope[:, None, 64:]
    return (_norm_rope(x[:, :Hq], st["q_w"], cos, sin), _norm_rope(x[:, Hq:Hq + Hkv], st["k_w"], cos, sin),
            x[:, Hq + Hkv:])


def _rows(blocks, table, place):
    """The cached rows of every sequence, fp32 [n, Hkv, width * 16, 128] (rows past its end are some page's)."""
    return _unpack(blocks[table.long().clamp(min=0)], place).transpose(1, 2).flatten(2, 3)


def _set_rows(rows, st, x):
    """The new tokens' rows in their places."""
    pos = st["positions"].long()
    rows[st["seq"], :, pos] = _values(*_quantise(x))
    return rows


def _softmax_rows(q, k, v, seen):
    """q [n, Hkv, rows, 128], k, v [n, Hkv, tokens, 128]; seen: which tokens a row sees."""
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    x = torch.where(seen, x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return torch.matmul(p, v) / p.sum(-1, keepdim=True)


def _plain_decode(st, q, k, v):
    n, Hq, Hkv = q.shape[0], st["Hq"], st["Hkv"]
    seen = torch.arange(k.shape[2], device=k.device) < st["lens"][:, None, None, None]
    v = torch.where(seen.transpose(-1, -2), v, 0.0)
    return _softmax_rows(q.float().unflatten(1, (Hkv, Hq // Hkv)), k, v, seen).reshape(n, Hq, D).to(torch.bfloat16)


def _plain_prompt(st, q, k, v):
    Hq, Hkv, n, most = st["Hq"], st["Hkv"], st["table"].shape[0], st["max_new"]
    qp = torch.zeros(n, most, Hq, D, device=q.device)
    qp[st["seq"], st["row"]] = q.float()
    qp = qp.view(n, most, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).flatten(2, 3)  # rows: (head of the group, token)
    new = st["indptr"][1:] - st["indptr"][:-1]
    upto = (st["lens"] - new)[:, None] + torch.arange(most, device=q.device)
    seen = (torch.arange(k.shape[2], device=k.device) <= upto[..., None])[:, None, None]
    seen = seen.expand(-1, -1, Hq // Hkv, -1, -1).flatten(2, 3)
    out = _softmax_rows(qp, k, v, seen).unflatten(2, (Hq // Hkv, most)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return out[st["seq"], st["row"]].to(torch.bfloat16)


def _plain_report(st):
    x = st["logits"].float()
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1)
    lse = m[:, 0] + torch.log(total)
    entropy = torch.log(total) - (e * (x - m)).sum(-1) / total
    best, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    best, ids = best[:, :st["top"]], ids[:, :st["top"]]
    return {"logprob": x.gather(1, st["targets"].long()[:, None])[:, 0] - lse, "lse": lse, "entropy": entropy,
            "top_ids": ids.to(torch.int32), "top_logprobs": best - lse[:, None]}


def _split(st):
    """k and v of the new tokens where they lie, in the projection's rows."""
    Hq, Hkv = st["Hq"], st["Hkv"]
    x = st["qkv"].unflatten(-1, (-1, D))
    return x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def run(st):
    op = st["op"]
    if own:
        return _run_own(st)
    if op == "report":
        return _plain_report(st)
    if op == "write":
        page, off = st["slots"].long() // PAGE, st["slots"].long() % PAGE
        for out, x in zip((st["k_out"], st["v_out"]), _split(st)):
            out[page, :, off] = _values(*_quantise(x)).to(torch.bfloat16)
        return {"k": st["k_out"], "v": st["v_out"]}
    kplace, vplace = st["places"]
    k, v = _rows(st["k_cache"], st["table"], kplace), _rows(st["v_cache"], st["table"], vplace)
    if op == "decode":
        return {"out": _plain_decode(st, st["q"], k, v)}
    q, new_k, new_v = _new_rows(st)
    k, v = _set_rows(k, st, new_k), _set_rows(v, st, new_v)
    return {"q": q, "out": (_plain_decode if op == "step" else _plain_prompt)(st, q, k, v)}


def _run_own(st):
    import invariant_bi_rmsnorm_gb300 as bi
    op = st["op"]
    if op == "report":
        return dict(zip(("logprob", "lse", "entropy", "top_ids", "top_logprobs"),
                        bi.logprobs_top(st["logits"], st["targets"], st["top"])))
    kc, vc, table, lens, most = st["k_cache"], st["v_cache"], st["table"], st["lens"], st["max_len"]
    if op == "write":
        k, v = _split(st)
        bi.kv4_append(k, v, st["slots"], kc, vc)
        bi.kv4_read(kc, vc, table, lens, most, st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if op == "decode":
        return {"out": bi.decode_attention_kv4(st["q"], kc, vc, table, lens, most, workspace=st["ws"])}
    q = bi.qk_norm_rope_append_kv4(st["qkv"], st["Hq"], st["Hkv"], st["positions"], st["slots"], st["rope"],
                                   st["q_w"], st["k_w"], kc, vc, EPS)
    if op == "step":
        return {"q": q, "out": bi.decode_attention_kv4(q, kc, vc, table, lens, most, workspace=st["ws"])}
    bi.kv4_read(kc, vc, table, lens, most, st["k_out"], st["v_out"])
    return {"q": q, "out": bi.prefill_attention(q, st["k_out"], st["v_out"], table, lens, st["indptr"],
                                                st["max_new"], most, workspace=st["pws"])}


# ---------------------------------------------------- the definition, in 64 bits ----
def _read64(blocks, is_v):
    """Blocks [n, Hkv, 1152] -> [Hkv, n * 16, 128], from the bytes by the format's formula."""
    b = blocks.to(torch.int64)
    r, d = torch.arange(PAGE, device=b.device)[:, None], torch.arange(D, device=b.device)
    if is_v:
        code = 4 * ((d // 32) % 2) + (d % 32) // 8
        byte = 512 * (r // 8) + 64 * (d % 8) + 16 * ((r % 8) // 2) + 8 * (r % 2) + 4 * (d // 64) + code // 2
    else:
        code = (d % 32) // 8 + 4 * (d % 2)
        byte = 64 * r + 16 * ((d % 8) // 2) + 4 * (d // 32) + code // 2
    n = torch.where(code % 2 == 1, b[..., byte] // 16, b[..., byte] % 16) - 8
    sb = b[..., 1024:].reshape(*b.shape[:2], PAGE, 4, 2)
    s = ((sb[..., 0] + (sb[..., 1] << 8)) << 16).to(torch.int32).view(torch.float32).double()
    x = n.double() * s[..., d // GROUP]
    return x.permute(1, 0, 2, 3).reshape(b.shape[1], -1, D)


def _four64(x):
    """What rows x [..., 128] are held as in 4 bits, in 64 bits: the scale from exact quotients and powers of two."""
    g = x.double().reshape(*x.shape[:-1], 4, GROUP)
    amax = g.abs().amax(-1)
    m, e = torch.frexp(amax / torch.full_like(amax, 7.0))
    s = (torch.round(m * 16) * ((e.long() + 1019) << 52).view(torch.float64))[..., None]  # times 2^(e - 4), from its bits
    n = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, 1.0)), 0.0).clamp(-7, 7)
    return (n * s).reshape(x.shape)


def _rotated64(x, w, pos):
    """bf16-rounded norm, then rotation by angles from 64 bits (rounded to the table's fp32), bf16-rounded."""
    x = x.double()
    x = (x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS) * w.double()).to(torch.bfloat16).double()
    f = torch.pow(torch.tensor(THETA, dtype=torch.float64, device=x.device),
                  -torch.arange(64, dtype=torch.float64, device=x.device) / 64)
    ang = pos.double()[:, None, None] * f
    c, s = ang.cos().float().double(), ang.sin().float().double()
    return torch.cat([x[..., :64] * c - x[..., 64:] * s, x[..., 64:] * c + x[..., :64] * s], -1).to(torch.bfloat16)


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "report":
        x = st["logits"].double()
        lse = torch.logsumexp(x, -1)
        lp = x - lse[:, None]
        entropy = -(lp.exp() * lp).sum(-1)
        b = st["logits"].view(torch.int16).to(torch.int64)
        order = torch.where(b < 0, -(b & 0x7FFF), b)  # orders bf16 values as whole numbers
        key = (order << 20) - torch.arange(c["vocab"], device=x.device)
        ids = torch.topk(key, c["top"], dim=-1).indices
        return {"logprob": lp.gather(1, st["targets"].long()[:, None])[:, 0], "lse": lse, "entropy": entropy,
                "top_ids": ids.to(torch.int32), "top_logprobs": lp.gather(1, ids)}
    Hq, Hkv = c["Hq"], c["Hkv"]
    if c["op"] == "write":
        page, off = st["slots"].long() // PAGE, st["slots"].long() % PAGE
        outs = []
        for x in _split(st):
            o = torch.zeros(st["k_out"].shape, dtype=torch.float64, device=x.device)
            o[page, :, off] = _four64(x)
            outs.append(o)
        return {"k": outs[0], "v": outs[1]}
    if sum(st["lens"].tolist()) * Hkv > 10_000_000:
        return None  # too long in 64 bits
    if c["op"] == "decode":
        q, first = st["q"], torch.arange(c["B"] + 1).tolist()
    else:
        x = st["qkv"].unflatten(-1, (-1, D))
        q = _rotated64(x[:, :Hq], st["q_w"], st["positions"])
        new_k, new_v = _four64(_rotated64(x[:, Hq:Hq + Hkv], st["k_w"], st["positions"])), _four64(x[:, Hq + Hkv:])
        first = st["indptr"].tolist()
    outs = []
    for i, L in enumerate(st["lens"].tolist()):
        a, b = first[i], first[i + 1]
        at = st["table"][i, :-(-L // PAGE)].long()
        k, v = (_read64(st[m][at], m == "v_cache")[:, :L] for m in ("k_cache", "v_cache"))
        if c["op"] != "decode":
            k[:, L - (b - a):], v[:, L - (b - a):] = new_k[a:b].transpose(0, 1), new_v[a:b].transpose(0, 1)
        k, v = (x.repeat_interleave(Hq // Hkv, 0) for x in (k, v))
        s = torch.einsum("rhd,htd->hrt", q[a:b].double(), k) * D ** -0.5
        ahead = torch.arange(L, device=q.device) > torch.arange(L - (b - a), L, device=q.device)[:, None]
        p = torch.softmax(s.masked_fill(ahead, -math.inf), -1)
        outs.append(torch.einsum("hrt,htd->rhd", p, v))
    out = torch.cat(outs)
    return {"out": out} if c["op"] == "decode" else {"q": q.double(), "out": out}
