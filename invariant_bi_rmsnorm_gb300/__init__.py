"""Batch-invariant forward kernels for LLM inference on GB300 (sm_103a).

Thin Python binding over libbi.so (C ABI: include/bi.h).  Each function only
checks and marshals its torch arguments (device pointers, sizes, leading
dimensions, the current CUDA stream) and calls the library; every step of the
computation runs in the library's CUDA kernels.  There is no CPU fallback:
tensors must live on a CUDA device, and a missing library raises.

    rmsnorm(x, w, eps)                    y = x * rsqrt(mean(x^2) + eps) * w, per row
    add_rmsnorm(x, residual, w, eps)      residual += x, then rmsnorm(residual)
    gemm(x, W)                            y = x @ W.T  (W in nn.Linear [N, K] layout)
    gemm_swiglu(x, interleave_gate_up(W)) silu(x @ W_gate.T) * (x @ W_up.T), fused
    decode_attention(q, k_cache, v_cache, block_table, seq_lens, max_seq_len)
                                          paged decode attention, 256-token splits
    prefill_attention(...)                causal attention for many rows per sequence,
                                          bit-identical per row to decode_attention
    qk_norm_rope_append(...), silu_mul(gate_up), logprobs(logits, targets)
    kv4_cache(num_pages, Hkv)             a pair of empty 4-bit caches, and what uses them:
    kv4_append(k, v, slots, ...), qk_norm_rope_append_kv4(...)
                                          quantise new tokens' K/V into their slots
    kv4_read(...)                         read sequences back into a bf16 cache (prefill's)
    decode_attention_kv4(...)             decode attention over the 4-bit cache
    logprobs_top(logits, targets, k)      log-probability, lse, entropy, k best tokens

Every output row's bits depend only on that row's own inputs (batch
invariance); see include/bi.h for the exact contract of each call.
"""
from __future__ import annotations

import math

import torch

from . import _lib
from ._lib import (DECODE_CHUNK, DECODE_COUNTER_BYTES, KV4_BLOCK_BYTES, MAX_TOP_LOGPROBS,
                   PAGE_SIZE)

__all__ = ["BiError", "rmsnorm", "gemm", "gemm_swiglu", "interleave_gate_up",
           "decode_attention", "decode_attention_fixed_splits",
           "prefill_attention", "prefill_attention_workspace_size", "add_rmsnorm",
           "qk_norm_rope_append", "silu_mul", "logprobs",
           "decode_attention_workspace_size", "selftest_wait_timeout",
           "decode_num_chunks", "decode_chunk_len", "get_device_error", "abi_version",
           "status_string", "PAGE_SIZE", "DECODE_CHUNK", "kv4_cache", "kv4_append",
           "qk_norm_rope_append_kv4", "kv4_read", "decode_attention_kv4", "logprobs_top",
           "KV4_BLOCK_BYTES", "MAX_TOP_LOGPROBS"]


def _stream_of(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# The handle of a device's current stream.  Building a torch.cuda.Stream object
# for it takes 3 us; the function that gives the handle alone exists in CUDA
# builds of torch only.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _current_device() -> int:
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2  # no device: no tensor is there


class BiError(RuntimeError):
    """A libbi.so call returned a status other than BI_OK."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def status_string(status: int) -> str:
    return _lib.load().bi_status_string(int(status)).decode()


def abi_version() -> int:
    return int(_lib.load().bi_abi_version())


def _check(status: int, where: str) -> None:
    if status != _lib.BI_OK:
        raise BiError(status, where)


def _stream(stream) -> int:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())  # which raises where there is no device
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _cuda_bf16(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")


def _row_major_2d(t: torch.Tensor, name: str) -> int:
    """Leading dimension (elements) of a 2-D tensor with unit inner stride."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return int(t.stride(0)) if t.shape[0] > 1 else int(t.shape[1])


def get_device_error(stream=None) -> None:
    """Synchronise `stream` and raise BiError if a kernel recorded a
    device-side problem (a barrier wait past its limit, or an out-of-range
    seq_lens / block_table entry).  Clears the record."""
    _check(_lib.load().bi_get_device_error(_stream(stream)), "bi_get_device_error")


# ------------------------------------------------------------- RMSNorm ------
def rmsnorm(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """Batch-invariant RMSNorm over the last dimension of x [rows, hidden]."""
    _cuda_bf16(x, "x")
    _cuda_bf16(w, "w")
    if x.dim() != 2 or w.dim() != 1 or w.shape[0] != x.shape[1] or not w.is_contiguous():
        raise ValueError("rmsnorm: x [rows, hidden] and contiguous w [hidden] expected")
    rows, hidden = x.shape
    if out is None:
        out = torch.empty((rows, hidden), dtype=torch.bfloat16, device=x.device)
    _cuda_bf16(out, "out")
    if tuple(out.shape) != (rows, hidden):
        raise ValueError("rmsnorm: out has the wrong shape")
    ld_x = _row_major_2d(x, "x")
    ld_y = _row_major_2d(out, "out")
    _check(_lib.load().bi_rmsnorm(x.data_ptr(), w.data_ptr(), out.data_ptr(), rows, hidden,
                                  ld_x, ld_y, float(eps), _stream(stream)), "bi_rmsnorm")
    return out


def add_rmsnorm(x: torch.Tensor, residual: torch.Tensor, w: torch.Tensor, eps: float = 1e-6,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """residual += x (bf16, in place), then RMSNorm(residual) * w -> out."""
    for t, n in ((x, "x"), (residual, "residual"), (w, "w")):
        _cuda_bf16(t, n)
    if x.shape != residual.shape or x.dim() != 2 or w.dim() != 1 or w.shape[0] != x.shape[1]:
        raise ValueError("add_rmsnorm: x, residual [rows, hidden] and w [hidden] expected")
    rows, hidden = x.shape
    if out is None:
        out = torch.empty((rows, hidden), dtype=torch.bfloat16, device=x.device)
    _cuda_bf16(out, "out")
    _check(_lib.load().bi_add_rmsnorm(x.data_ptr(), residual.data_ptr(), w.data_ptr(),
                                      out.data_ptr(), rows, hidden, _row_major_2d(x, "x"),
                                      _row_major_2d(residual, "residual"),
                                      _row_major_2d(out, "out"), float(eps), _stream(stream)),
           "bi_add_rmsnorm")
    return out


def qk_norm_rope_append(qkv: torch.Tensor, Hq: int, Hkv: int, positions: torch.Tensor,
                        slots: torch.Tensor, rope: torch.Tensor, q_norm_w, k_norm_w,
                        k_cache: torch.Tensor, v_cache: torch.Tensor, eps: float = 1e-6,
                        q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Per-head q/k RMSNorm + RoPE; q -> q_out [T, Hq, 128]; k, v -> cache slots."""
    _cuda_bf16(qkv, "qkv")
    T = qkv.shape[0]
    D = 128
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=qkv.device)
    for t, n in ((positions, "positions"), (slots, "slots")):
        if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous() or t.shape[0] != T:
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor of length T")
    if not rope.is_cuda or rope.dtype != torch.float32 or not rope.is_contiguous():
        raise ValueError("rope must be a contiguous float32 CUDA tensor")
    num_pages, Hkv2, page, D2 = k_cache.shape
    if Hkv2 != Hkv or D2 != D:
        raise ValueError("qk_norm_rope_append: cache shape mismatch")
    _check(_lib.load().bi_qk_norm_rope_append(
        qkv.data_ptr(), _row_major_2d(qkv, "qkv"), T, Hq, Hkv, D, positions.data_ptr(),
        slots.data_ptr(), rope.data_ptr(), rope.shape[0],
        q_norm_w.data_ptr() if q_norm_w is not None else None,
        k_norm_w.data_ptr() if k_norm_w is not None else None, float(eps), q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), num_pages, page, _stream(stream)),
        "bi_qk_norm_rope_append")
    return q_out


def silu_mul(gate_up: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """SwiGLU: out = silu(gate_up[:, :F]) * gate_up[:, F:]."""
    _cuda_bf16(gate_up, "gate_up")
    T, F2 = gate_up.shape
    F = F2 // 2
    if out is None:
        out = torch.empty((T, F), dtype=torch.bfloat16, device=gate_up.device)
    _check(_lib.load().bi_silu_mul(gate_up.data_ptr(), _row_major_2d(gate_up, "gate_up"), T, F,
                                   out.data_ptr(), _row_major_2d(out, "out"), _stream(stream)),
           "bi_silu_mul")
    return out


def logprobs(logits: torch.Tensor, targets: torch.Tensor | None = None, stream=None):
    """(logprob of targets [rows] fp32 or None, lse [rows] fp32) of bf16 logits
    [rows, vocab], batch-invariant per row."""
    _cuda_bf16(logits, "logits")
    rows, vocab = logits.shape
    lse = torch.empty(rows, dtype=torch.float32, device=logits.device)
    lp = None
    if targets is not None:
        if not targets.is_cuda or targets.dtype != torch.int32 or not targets.is_contiguous():
            raise ValueError("targets must be a contiguous int32 CUDA tensor")
        lp = torch.empty(rows, dtype=torch.float32, device=logits.device)
    _check(_lib.load().bi_logprobs(logits.data_ptr(), rows, vocab, _row_major_2d(logits, "logits"),
                                   targets.data_ptr() if targets is not None else None,
                                   lp.data_ptr() if lp is not None else None, lse.data_ptr(),
                                   _stream(stream)), "bi_logprobs")
    return lp, lse


# ---------------------------------------------------------------- GEMM ------
def gemm(x: torch.Tensor, W: torch.Tensor, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Batch-invariant y = x @ W.T with x [M, K] and W [N, K] (nn.Linear layout)."""
    _cuda_bf16(x, "x")
    _cuda_bf16(W, "W")
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1]:
        raise ValueError("gemm: x [M, K] and W [N, K] expected")
    M, K = x.shape
    N = W.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _cuda_bf16(out, "out")
    if tuple(out.shape) != (M, N):
        raise ValueError("gemm: out has the wrong shape")
    _check(_lib.load().bi_gemm(x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K,
                               _row_major_2d(x, "x"), _row_major_2d(W, "W"),
                               _row_major_2d(out, "out"), _stream(stream)), "bi_gemm")
    return out


def interleave_gate_up(W_gate_up: torch.Tensor) -> torch.Tensor:
    """[2F, K] weight with the gate rows first and the up rows after them ->
    the [2F, K] layout bi_gemm_swiglu reads: groups of 8 gate rows, each
    followed by the 8 matching up rows."""
    F2, K = W_gate_up.shape
    if F2 % 16:
        raise ValueError("interleave_gate_up: 2F must be a multiple of 16")
    F = F2 // 2
    g = W_gate_up[:F].reshape(F // 8, 8, K)
    u = W_gate_up[F:].reshape(F // 8, 8, K)
    return torch.cat([g, u], dim=1).reshape(F2, K).contiguous()


def gemm_swiglu(x: torch.Tensor, W_gu: torch.Tensor, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Batch-invariant h = silu(x @ W_gate.T) * (x @ W_up.T), bit-identical to
    silu_mul(gemm(x, W_gate_up)); W_gu is interleave_gate_up(W_gate_up)."""
    _cuda_bf16(x, "x")
    _cuda_bf16(W_gu, "W_gu")
    if x.dim() != 2 or W_gu.dim() != 2 or x.shape[1] != W_gu.shape[1]:
        raise ValueError("gemm_swiglu: x [M, K] and W_gu [2F, K] expected")
    M, K = x.shape
    if W_gu.shape[0] % 16:
        raise ValueError("gemm_swiglu: W_gu must have 2F rows, F a multiple of 8")
    F = W_gu.shape[0] // 2
    if out is None:
        out = torch.empty((M, F), dtype=torch.bfloat16, device=x.device)
    _cuda_bf16(out, "out")
    if tuple(out.shape) != (M, F):
        raise ValueError("gemm_swiglu: out has the wrong shape")
    _check(_lib.load().bi_gemm_swiglu(x.data_ptr(), W_gu.data_ptr(), out.data_ptr(), M, F, K,
                                      _row_major_2d(x, "x"), _row_major_2d(W_gu, "W_gu"),
                                      _row_major_2d(out, "out"), _stream(stream)),
           "bi_gemm_swiglu")
    return out


# ----------------------------------------------------------- attention ------
def decode_attention_workspace_size(B: int, Hq: int, D: int, max_seq_len: int) -> int:
    return int(_lib.load().bi_decode_attention_workspace_size(B, Hq, D, max_seq_len))


def decode_num_chunks(seq_len: int) -> int:
    return int(_lib.load().bi_decode_num_chunks(seq_len))


def decode_chunk_len(seq_len: int, c: int) -> int:
    return int(_lib.load().bi_decode_chunk_len(seq_len, c))


def selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Launch the device timeout self-test (a bounded wait that must run out);
    read its outcome with get_device_error()."""
    _check(_lib.load().bi_selftest_wait_timeout(int(limit_us), _stream(stream)),
           "bi_selftest_wait_timeout")


def _attention_args(q, k_cache, v_cache, block_table, seq_lens):
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _cuda_bf16(t, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens")):
        if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    if q.dim() != 3 or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("decode_attention: q [B,Hq,D] and caches [P,Hkv,page,D] expected")
    B, Hq, D = q.shape
    num_pages, Hkv, page, D2 = k_cache.shape
    if D2 != D or block_table.dim() != 2 or block_table.shape[0] != B or tuple(seq_lens.shape) != (B,):
        raise ValueError("decode_attention: inconsistent shapes")
    return B, Hq, D, num_pages, Hkv, page


def decode_attention_fixed_splits(q, k_cache, v_cache, block_table, seq_lens, max_seq_len: int,
                                  num_splits: int, scale: float | None = None, out=None,
                                  workspace=None, stream=None) -> torch.Tensor:
    """Fixed split-COUNT attention: NOT batch- or growth-invariant.  The
    comparison variant (negative control and cost reference) only."""
    B, Hq, D, num_pages, Hkv, page = _attention_args(q, k_cache, v_cache, block_table, seq_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    need = decode_attention_workspace_size(B, Hq, D, int(num_splits) * DECODE_CHUNK)
    if workspace is None and need > 0:
        # the leading arrival counters must start at zero (every call leaves
        # them zero, so a caller-kept workspace is cleared only once)
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.load().bi_decode_attention_fixed_splits(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
        block_table.shape[1], seq_lens.data_ptr(), B, Hq, Hkv, D, page, num_pages,
        int(max_seq_len), float(scale), int(num_splits), out.data_ptr(), ws_ptr, ws_bytes,
        _stream(stream)), "bi_decode_attention_fixed_splits")
    return out


def prefill_attention_workspace_size(T: int, Hq: int, D: int, max_seq_len: int) -> int:
    return int(_lib.load().bi_prefill_attention_workspace_size(T, Hq, D, max_seq_len))


def prefill_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_table: torch.Tensor, seq_lens: torch.Tensor, q_indptr: torch.Tensor,
                      max_q_len: int, max_seq_len: int, scale: float | None = None,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Causal attention for the last n_i tokens of each sequence at once.

    q [T, Hq, D]; q_indptr [S + 1] int32 (sequence i owns q rows
    q_indptr[i] .. q_indptr[i+1]-1); seq_lens [S] int32 (cached tokens,
    including the query rows); block_table [S, max_pages_per_seq] int32.
    Bit-identical per row to decode_attention with the row's own length."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _cuda_bf16(t, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens"), (q_indptr, "q_indptr")):
        if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    if q.dim() != 3 or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("prefill_attention: q [T,Hq,D] and caches [P,Hkv,page,D] expected")
    T, Hq, D = q.shape
    num_pages, Hkv, page, D2 = k_cache.shape
    S = seq_lens.shape[0]
    if (D2 != D or block_table.dim() != 2 or block_table.shape[0] != S
            or tuple(q_indptr.shape) != (S + 1,)):
        raise ValueError("prefill_attention: inconsistent shapes")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
    _cuda_bf16(out, "out")
    if tuple(out.shape) != (T, Hq, D) or not out.is_contiguous():
        raise ValueError("prefill_attention: out must be a contiguous [T, Hq, D] tensor")
    need = prefill_attention_workspace_size(T, Hq, D, int(max_seq_len))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.load().bi_prefill_attention(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
        block_table.shape[1], seq_lens.data_ptr(), q_indptr.data_ptr(), S, T, Hq, Hkv, D, page,
        num_pages, int(max_q_len), int(max_seq_len), float(scale), out.data_ptr(), ws_ptr,
        ws_bytes, _stream(stream)), "bi_prefill_attention")
    return out


def decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                     scale: float | None = None, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Batch-invariant paged decode attention.

    q [B, Hq, D]; k_cache, v_cache [num_pages, Hkv, 16, D]; block_table
    [B, max_pages_per_seq] int32; seq_lens [B] int32 (1 .. max_seq_len).
    `max_seq_len` is a host-side bound on seq_lens that sizes the launch (it
    is not read from the device, so no synchronisation happens)."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _cuda_bf16(t, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens")):
        if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    if q.dim() != 3 or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("decode_attention: q [B,Hq,D] and caches [P,Hkv,page,D] expected")
    B, Hq, D = q.shape
    num_pages, Hkv, page, D2 = k_cache.shape
    if D2 != D or block_table.dim() != 2 or block_table.shape[0] != B or tuple(seq_lens.shape) != (B,):
        raise ValueError("decode_attention: inconsistent shapes")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    _cuda_bf16(out, "out")
    if tuple(out.shape) != (B, Hq, D) or not out.is_contiguous():
        raise ValueError("decode_attention: out must be a contiguous [B, Hq, D] tensor")
    need = decode_attention_workspace_size(B, Hq, D, max_seq_len)
    if workspace is None and need > 0:
        # the leading arrival counters must start at zero (every call leaves
        # them zero, so a caller-kept workspace is cleared only once)
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.load().bi_decode_attention(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
        block_table.shape[1], seq_lens.data_ptr(), B, Hq, Hkv, D, page, num_pages,
        int(max_seq_len), float(scale), out.data_ptr(), ws_ptr, ws_bytes, _stream(stream)),
        "bi_decode_attention")
    return out


# --------------------------------------------------------- 4-bit KV cache ----
# A decode step makes these calls once a layer, so each tests all it has to in
# one condition and sorts out what was wrong only when something was.
_BF16, _I32, _U8, _F32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32


def _refuse(where: str, *wanted):
    """Raise for the first of (tensor, name, dtype, shape) that is not a
    contiguous tensor of that type and shape (None: any) on the current CUDA
    device."""
    for t, name, dtype, shape in wanted:
        if t is None:
            continue
        kind = str(dtype).split(".")[-1]
        if not t.is_cuda:
            raise ValueError(f"{where}: {name} must be a CUDA tensor (no CPU path exists)")
        if t.dtype != dtype:
            raise ValueError(f"{where}: {name} must be {kind}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")
        if shape is not None and (t.dim() != len(shape)
                                  or any(w is not None and w != n for w, n in zip(shape, t.shape))):
            want = ", ".join("any" if w is None else str(w) for w in shape)
            raise ValueError(f"{where}: {name} must have shape [{want}], got {tuple(t.shape)}")
    for t, name, _, _ in wanted:
        if t is not None and t.get_device() != _current_device():
            raise ValueError(f"{where}: {name} must be on the current CUDA device ({_current_device()})")
    raise ValueError(f"{where}: arguments do not fit together")


def _made(stream, make, *args, **kw) -> torch.Tensor:
    """make(...) on the stream that is to use the tensor first, so that what
    fills it comes before, and its memory is not handed out again too soon."""
    if stream is None:
        return make(*args, **kw)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def kv4_cache(num_pages: int, Hkv: int, device="cuda") -> tuple[torch.Tensor, torch.Tensor]:
    """A pair of empty 4-bit K and V caches, uint8 [num_pages, Hkv, 1152]: pages
    of 16 tokens, heads of 128 dims (include/bi.h gives the layout)."""
    k = torch.zeros((num_pages, Hkv, KV4_BLOCK_BYTES), dtype=torch.uint8, device=device)
    return k, torch.zeros_like(k)


def _side_by_side(t: torch.Tensor) -> bool:
    """Whether t [T, Hkv, 128] has the values of a token in one run."""
    if t.dim() != 3 or t.shape[2] != 128:
        return False
    st = t.stride()
    return t.numel() == 0 or (st[2] == 1 and (t.shape[1] == 1 or st[1] == 128))


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
               v_cache: torch.Tensor, stream=None) -> None:
    """Quantise k, v [T, Hkv, 128] (any token stride: views of a qkv projection
    will do) to 4 bits in the slots (page * 16 + offset, int32 [T]) of the caches."""
    dev = _current_device()
    shape, cs = k.shape, k_cache.shape
    if not (k.dtype is v.dtype is _BF16 and _side_by_side(k) and _side_by_side(v) and v.shape == shape
            and slots.dtype is _I32 and slots.shape == shape[:1] and slots.is_contiguous()
            and k_cache.dtype is v_cache.dtype is _U8 and len(cs) == 3 and cs[1] == shape[1]
            and cs[2] == KV4_BLOCK_BYTES and v_cache.shape == cs and k_cache.is_contiguous()
            and v_cache.is_contiguous()
            and dev == k.get_device() == v.get_device() == slots.get_device()
            == k_cache.get_device() == v_cache.get_device()):
        for t, n in ((k, "k"), (v, "v")):
            _cuda_bf16(t, n)
            if not _side_by_side(t):
                raise ValueError(f"kv4_append: {n} must be [T, Hkv, 128], the heads of a token side by side")
        if v.shape != shape:
            raise ValueError("kv4_append: k and v must have the same shape")
        cache = (None, shape[1], KV4_BLOCK_BYTES)
        _refuse("kv4_append", (k_cache, "k_cache", _U8, cache), (v_cache, "v_cache", _U8, cache),
                (slots, "slots", _I32, shape[:1]))
    T, Hkv, _ = shape
    _check(_lib.load().bi_kv4_append(
        k.data_ptr(), k.stride(0) if T > 1 else Hkv * 128, v.data_ptr(),
        v.stride(0) if T > 1 else Hkv * 128, T, Hkv, 128, slots.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), cs[0], PAGE_SIZE, _raw_stream(dev) if stream is None else _stream(stream)),
        "bi_kv4_append")


def qk_norm_rope_append_kv4(qkv: torch.Tensor, Hq: int, Hkv: int, positions: torch.Tensor,
                            slots: torch.Tensor, rope: torch.Tensor, q_norm_w, k_norm_w,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, eps: float = 1e-6,
                            q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qk_norm_rope_append into 4-bit caches: q -> q_out [T, Hq, 128]; the k and
    v rows, quantised -> their slots."""
    dev = _current_device()
    if q_out is None:
        q_out = _made(stream, torch.empty, (qkv.shape[0], Hq, 128), dtype=_BF16, device=qkv.device)
    shape, cs, rs = qkv.shape, k_cache.shape, rope.shape
    if not (len(shape) == 2 and qkv.dtype is _BF16 and shape[1] >= (Hq + 2 * Hkv) * 128
            and qkv.stride(1) == 1 and positions.dtype is slots.dtype is _I32
            and positions.shape == slots.shape == shape[:1] and positions.is_contiguous()
            and slots.is_contiguous() and rope.dtype is _F32 and len(rs) == 2 and rs[1] == 128
            and rope.is_contiguous() and k_cache.dtype is v_cache.dtype is _U8 and len(cs) == 3
            and cs[1] == Hkv and cs[2] == KV4_BLOCK_BYTES and v_cache.shape == cs
            and k_cache.is_contiguous() and v_cache.is_contiguous() and q_out.dtype is _BF16
            and q_out.shape == (shape[0], Hq, 128) and q_out.is_contiguous()
            and dev == qkv.get_device() == positions.get_device() == slots.get_device()
            == rope.get_device() == k_cache.get_device() == v_cache.get_device() == q_out.get_device()):
        where = "qk_norm_rope_append_kv4"
        _cuda_bf16(qkv, "qkv")
        if qkv.dim() != 2 or shape[1] < (Hq + 2 * Hkv) * 128 or qkv.stride(1) != 1:
            raise ValueError(f"{where}: qkv [T, (Hq + 2 Hkv) * 128] with whole rows expected")
        cache = (None, Hkv, KV4_BLOCK_BYTES)
        _refuse(where, (k_cache, "k_cache", _U8, cache), (v_cache, "v_cache", _U8, cache),
                (positions, "positions", _I32, shape[:1]), (slots, "slots", _I32, shape[:1]),
                (rope, "rope", _F32, (None, 128)), (q_out, "q_out", _BF16, (shape[0], Hq, 128)))
    for t, n in ((q_norm_w, "q_norm_w"), (k_norm_w, "k_norm_w")):
        if t is not None and not (t.dtype is _BF16 and t.shape == (128,) and t.is_contiguous()
                                  and t.get_device() == dev):
            _refuse("qk_norm_rope_append_kv4", (t, n, _BF16, (128,)))
    T = shape[0]
    _check(_lib.load().bi_qk_norm_rope_append_kv4(
        qkv.data_ptr(), qkv.stride(0) if T > 1 else shape[1], T, Hq, Hkv, 128, positions.data_ptr(),
        slots.data_ptr(), rope.data_ptr(), rs[0], None if q_norm_w is None else q_norm_w.data_ptr(),
        None if k_norm_w is None else k_norm_w.data_ptr(), eps, q_out.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), cs[0], PAGE_SIZE, _raw_stream(dev) if stream is None else _stream(stream)),
        "bi_qk_norm_rope_append_kv4")
    return q_out


def kv4_read(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
             seq_lens: torch.Tensor, max_seq_len: int, k_out: torch.Tensor, v_out: torch.Tensor,
             stream=None) -> None:
    """Read the tokens of sequences back from 4-bit caches into bf16 caches
    k_out, v_out [num_pages, Hkv, 16, 128] of the same page numbering (other
    rows stay as they are): the caches prefill_attention takes, with the same
    block_table [S, max_pages_per_seq] and seq_lens [S]."""
    dev = _current_device()
    cs, bs, ls = k_cache.shape, block_table.shape, seq_lens.shape
    if not (k_cache.dtype is v_cache.dtype is _U8 and len(cs) == 3 and cs[2] == KV4_BLOCK_BYTES
            and v_cache.shape == cs and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_table.dtype is seq_lens.dtype is _I32 and len(bs) == 2 and len(ls) == 1
            and ls[0] == bs[0] and block_table.is_contiguous() and seq_lens.is_contiguous()
            and k_out.dtype is v_out.dtype is _BF16
            and k_out.shape == v_out.shape == (cs[0], cs[1], PAGE_SIZE, 128)
            and k_out.is_contiguous() and v_out.is_contiguous()
            and dev == k_cache.get_device() == v_cache.get_device() == block_table.get_device()
            == seq_lens.get_device() == k_out.get_device() == v_out.get_device()):
        cache = (None, None, KV4_BLOCK_BYTES)
        _refuse("kv4_read", (k_cache, "k_cache", _U8, cache), (v_cache, "v_cache", _U8, cs),
                (block_table, "block_table", _I32, (None, None)), (seq_lens, "seq_lens", _I32, bs[:1]),
                *((t, n, _BF16, (cs[0], cs[1], PAGE_SIZE, 128)) for t, n in ((k_out, "k_out"), (v_out, "v_out"))))
    _check(_lib.load().bi_kv4_read(
        k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), bs[1], seq_lens.data_ptr(),
        bs[0], cs[1], 128, PAGE_SIZE, cs[0], int(max_seq_len), k_out.data_ptr(), v_out.data_ptr(),
        _raw_stream(dev) if stream is None else _stream(stream)), "bi_kv4_read")


def decode_attention_kv4(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                         scale: float | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """decode_attention over 4-bit caches [num_pages, Hkv, 1152]: the bits of
    decode_attention over what kv4_read gives of them.  Other arguments, and
    the workspace, as decode_attention."""
    dev = _current_device()
    if out is None:
        out = _made(stream, torch.empty_like, q)
    qs, cs, bs = q.shape, k_cache.shape, block_table.shape
    if not (q.dtype is out.dtype is _BF16 and len(qs) == 3 and out.shape == qs and q.is_contiguous()
            and out.is_contiguous() and k_cache.dtype is v_cache.dtype is _U8 and len(cs) == 3
            and cs[2] == KV4_BLOCK_BYTES and v_cache.shape == cs and k_cache.is_contiguous()
            and v_cache.is_contiguous() and block_table.dtype is seq_lens.dtype is _I32
            and len(bs) == 2 and bs[0] == qs[0] and seq_lens.shape == qs[:1]
            and block_table.is_contiguous() and seq_lens.is_contiguous()
            and dev == q.get_device() == out.get_device() == k_cache.get_device()
            == v_cache.get_device() == block_table.get_device() == seq_lens.get_device()):
        where = "decode_attention_kv4"
        _refuse(where, (q, "q", _BF16, (None, None, None)),
                (k_cache, "k_cache", _U8, (None, None, KV4_BLOCK_BYTES)), (v_cache, "v_cache", _U8, cs),
                (block_table, "block_table", _I32, (qs[0], None)), (seq_lens, "seq_lens", _I32, qs[:1]),
                (out, "out", _BF16, qs))
    B, Hq, D = qs
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if workspace is None:
        need = decode_attention_workspace_size(B, Hq, D, int(max_seq_len))
        if need > 0:
            # the leading arrival counters must start at zero (every call leaves
            # them zero, so a caller-kept workspace is cleared only once)
            workspace = _made(stream, torch.zeros, need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse("decode_attention_kv4", (workspace, "workspace", workspace.dtype, None))
    ws = workspace is not None
    _check(_lib.load().bi_decode_attention_kv4(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), bs[1],
        seq_lens.data_ptr(), B, Hq, cs[1], D, PAGE_SIZE, cs[0], int(max_seq_len), scale, out.data_ptr(),
        workspace.data_ptr() if ws else None, workspace.nbytes if ws else 0,
        _raw_stream(dev) if stream is None else _stream(stream)), "bi_decode_attention_kv4")
    return out


# ---------------------------------------------------- per-token log-probs ----
def logprobs_top(logits: torch.Tensor, targets: torch.Tensor | None, k: int, stream=None):
    """(logprob of targets [rows] or None, lse [rows], entropy [rows], top_ids
    [rows, k] int32, top_logprobs [rows, k]) of bf16 logits [rows, vocab]: the
    bits of logprobs(logits, targets) where logits are -inf or within +-1024, the
    softmax's entropy in nats, and the k (1 .. 32) largest logits' tokens, largest first, equal ones by ascending id."""
    dev = _current_device()
    shape = logits.shape
    if not (logits.dtype is _BF16 and len(shape) == 2 and logits.stride(1) == 1
            and logits.get_device() == dev):
        _cuda_bf16(logits, "logits")
        _row_major_2d(logits, "logits")
        if logits.get_device() != dev:
            _refuse("logprobs_top", (logits.contiguous(), "logits", _BF16, None))
    rows, vocab = shape
    k = int(k)
    if k < 1:
        raise ValueError("logprobs_top: k must be at least 1")
    if targets is not None and not (targets.dtype is _I32 and targets.shape == shape[:1]
                                    and targets.is_contiguous() and targets.get_device() == dev):
        _refuse("logprobs_top", (targets, "targets", _I32, shape[:1]))
    on = logits.device
    lse = _made(stream, torch.empty, rows, dtype=_F32, device=on)
    entropy = _made(stream, torch.empty_like, lse)
    lp = _made(stream, torch.empty_like, lse) if targets is not None else None
    top = _made(stream, torch.empty, (rows, k), dtype=_F32, device=on)
    ids = _made(stream, torch.empty, (rows, k), dtype=_I32, device=on)
    _check(_lib.load().bi_logprobs_top(
        logits.data_ptr(), rows, vocab, logits.stride(0) if rows > 1 else vocab,
        None if targets is None else targets.data_ptr(), None if lp is None else lp.data_ptr(),
        lse.data_ptr(), entropy.data_ptr(), k, ids.data_ptr(), top.data_ptr(),
        _raw_stream(dev) if stream is None else _stream(stream)), "bi_logprobs_top")
    return lp, lse, entropy, ids, top
