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
        return torch.cuda.current_stream().cuda_stream
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
def _cuda_i32(t: torch.Tensor, name: str, shape: tuple) -> None:
    if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _one_device(where: str, *tensors) -> None:
    """Every tensor on the current device, whose stream and error word the call uses."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: every tensor must be on the current CUDA device ({dev})")


def _kv4_caches(k_cache: torch.Tensor, v_cache: torch.Tensor, where: str) -> tuple[int, int]:
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError(f"{where}: {n} must be a contiguous uint8 CUDA tensor")
    shape = k_cache.shape
    if len(shape) != 3 or shape[2] != KV4_BLOCK_BYTES or v_cache.shape != shape:
        raise ValueError(f"{where}: 4-bit caches [num_pages, Hkv, {KV4_BLOCK_BYTES}] expected")
    return shape[0], shape[1]


def kv4_cache(num_pages: int, Hkv: int, device="cuda") -> tuple[torch.Tensor, torch.Tensor]:
    """A pair of empty 4-bit K and V caches, uint8 [num_pages, Hkv, 1152]: pages
    of 16 tokens, heads of 128 dims (include/bi.h gives the layout)."""
    k = torch.zeros((num_pages, Hkv, KV4_BLOCK_BYTES), dtype=torch.uint8, device=device)
    return k, torch.zeros_like(k)


def _kv4_rows(t: torch.Tensor, name: str) -> int:
    """Token stride (elements) of k or v [T, Hkv, 128] with whole heads side by side."""
    _cuda_bf16(t, name)
    if t.dim() != 3 or t.shape[2] != 128:
        raise ValueError(f"{name} must be [T, Hkv, 128]")
    T, Hkv, _ = t.shape
    if t.numel() and (t.stride(2) != 1 or (Hkv > 1 and t.stride(1) != 128)):
        raise ValueError(f"{name}: the heads of a token must lie side by side")
    return int(t.stride(0)) if T > 1 else Hkv * 128


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
               v_cache: torch.Tensor, stream=None) -> None:
    """Quantise k, v [T, Hkv, 128] (any token stride: views of a qkv projection
    will do) to 4 bits in the slots (page * 16 + offset, int32 [T]) of the caches."""
    num_pages, Hkv = _kv4_caches(k_cache, v_cache, "kv4_append")
    ld_k, ld_v = _kv4_rows(k, "k"), _kv4_rows(v, "v")
    T = k.shape[0]
    if k.shape != v.shape or k.shape[1] != Hkv:
        raise ValueError("kv4_append: k and v [T, Hkv, 128] of the caches' Hkv expected")
    _cuda_i32(slots, "slots", (T,))
    _one_device("kv4_append", k, v, slots, k_cache, v_cache)
    _check(_lib.load().bi_kv4_append(
        k.data_ptr(), ld_k, v.data_ptr(), ld_v, T, Hkv, 128, slots.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), num_pages, PAGE_SIZE, _stream(stream)), "bi_kv4_append")


def qk_norm_rope_append_kv4(qkv: torch.Tensor, Hq: int, Hkv: int, positions: torch.Tensor,
                            slots: torch.Tensor, rope: torch.Tensor, q_norm_w, k_norm_w,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, eps: float = 1e-6,
                            q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qk_norm_rope_append into 4-bit caches: q -> q_out [T, Hq, 128]; the k and
    v rows, quantised -> their slots."""
    num_pages, Hkv2 = _kv4_caches(k_cache, v_cache, "qk_norm_rope_append_kv4")
    _cuda_bf16(qkv, "qkv")
    ld = _row_major_2d(qkv, "qkv")
    T = qkv.shape[0]
    if Hkv2 != Hkv or qkv.shape[1] < (Hq + 2 * Hkv) * 128:
        raise ValueError("qk_norm_rope_append_kv4: qkv [T, (Hq + 2 Hkv) * 128] and caches of Hkv "
                         "heads expected")
    _cuda_i32(positions, "positions", (T,))
    _cuda_i32(slots, "slots", (T,))
    if (not rope.is_cuda or rope.dtype != torch.float32 or not rope.is_contiguous()
            or rope.dim() != 2 or rope.shape[1] != 128):
        raise ValueError("rope must be a contiguous float32 CUDA tensor [max_pos, 128]")
    for t, n in ((q_norm_w, "q_norm_w"), (k_norm_w, "k_norm_w")):
        if t is not None:
            _cuda_bf16(t, n)
            if t.shape != (128,) or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous [128] tensor")
    if q_out is None:
        q_out = torch.empty((T, Hq, 128), dtype=torch.bfloat16, device=qkv.device)
    else:
        _cuda_bf16(q_out, "q_out")
        if q_out.shape != (T, Hq, 128) or not q_out.is_contiguous():
            raise ValueError("q_out must be a contiguous [T, Hq, 128] tensor")
    _one_device("qk_norm_rope_append_kv4", qkv, positions, slots, rope, q_norm_w, k_norm_w,
                k_cache, v_cache, q_out)
    _check(_lib.load().bi_qk_norm_rope_append_kv4(
        qkv.data_ptr(), ld, T, Hq, Hkv, 128, positions.data_ptr(), slots.data_ptr(),
        rope.data_ptr(), rope.shape[0], q_norm_w.data_ptr() if q_norm_w is not None else None,
        k_norm_w.data_ptr() if k_norm_w is not None else None, eps, q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), num_pages, PAGE_SIZE, _stream(stream)),
        "bi_qk_norm_rope_append_kv4")
    return q_out


def kv4_read(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
             seq_lens: torch.Tensor, max_seq_len: int, k_out: torch.Tensor, v_out: torch.Tensor,
             stream=None) -> None:
    """Read the tokens of sequences back from 4-bit caches into bf16 caches
    k_out, v_out [num_pages, Hkv, 16, 128] of the same page numbering (other
    rows stay as they are): the caches prefill_attention takes, with the same
    block_table [S, max_pages_per_seq] and seq_lens [S]."""
    num_pages, Hkv = _kv4_caches(k_cache, v_cache, "kv4_read")
    shape = (num_pages, Hkv, PAGE_SIZE, 128)
    for t, n in ((k_out, "k_out"), (v_out, "v_out")):
        _cuda_bf16(t, n)
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"kv4_read: {n} must be a contiguous {shape} tensor")
    if block_table.dim() != 2:
        raise ValueError("kv4_read: block_table [S, max_pages_per_seq] expected")
    S, width = block_table.shape
    _cuda_i32(block_table, "block_table", (S, width))
    _cuda_i32(seq_lens, "seq_lens", (S,))
    _one_device("kv4_read", k_cache, v_cache, block_table, seq_lens, k_out, v_out)
    _check(_lib.load().bi_kv4_read(
        k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), width, seq_lens.data_ptr(),
        S, Hkv, 128, PAGE_SIZE, num_pages, int(max_seq_len), k_out.data_ptr(), v_out.data_ptr(),
        _stream(stream)), "bi_kv4_read")


def decode_attention_kv4(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                         scale: float | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """decode_attention over 4-bit caches [num_pages, Hkv, 1152]: the bits of
    decode_attention over what kv4_read gives of them.  Other arguments, and
    the workspace, as decode_attention."""
    num_pages, Hkv = _kv4_caches(k_cache, v_cache, "decode_attention_kv4")
    _cuda_bf16(q, "q")
    if q.dim() != 3 or not q.is_contiguous() or block_table.dim() != 2:
        raise ValueError("decode_attention_kv4: contiguous q [B, Hq, D] and block_table "
                         "[B, max_pages_per_seq] expected")
    B, Hq, D = q.shape
    width = block_table.shape[1]
    _cuda_i32(block_table, "block_table", (B, width))
    _cuda_i32(seq_lens, "seq_lens", (B,))
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda_bf16(out, "out")
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError("decode_attention_kv4: out must be a contiguous [B, Hq, D] tensor")
    if workspace is None:
        need = decode_attention_workspace_size(B, Hq, D, max_seq_len)
        if need > 0:
            # the leading arrival counters must start at zero (every call leaves
            # them zero, so a caller-kept workspace is cleared only once)
            workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("decode_attention_kv4: workspace must be a contiguous CUDA tensor")
    _one_device("decode_attention_kv4", q, k_cache, v_cache, block_table, seq_lens, out, workspace)
    _check(_lib.load().bi_decode_attention_kv4(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), width,
        seq_lens.data_ptr(), B, Hq, Hkv, D, PAGE_SIZE, num_pages, int(max_seq_len), scale,
        out.data_ptr(), workspace.data_ptr() if workspace is not None else None,
        workspace.nbytes if workspace is not None else 0, _stream(stream)),
        "bi_decode_attention_kv4")
    return out


# ---------------------------------------------------- per-token log-probs ----
def logprobs_top(logits: torch.Tensor, targets: torch.Tensor | None, k: int, stream=None):
    """(logprob of targets [rows] or None, lse [rows], entropy [rows], top_ids
    [rows, k] int32, top_logprobs [rows, k]) of bf16 logits [rows, vocab]: the
    bits of logprobs(logits, targets), the softmax's entropy in nats, and the k
    (1 .. 32) largest logits' tokens, largest first, equal ones by ascending id."""
    _cuda_bf16(logits, "logits")
    ld = _row_major_2d(logits, "logits")
    rows, vocab = logits.shape
    k = int(k)
    if k < 1:
        raise ValueError("logprobs_top: k must be at least 1")
    if targets is not None:
        _cuda_i32(targets, "targets", (rows,))
    _one_device("logprobs_top", logits, targets)
    dev = logits.device
    f = torch.empty((3, rows), dtype=torch.float32, device=dev)
    lp, lse, entropy = f.unbind(0)
    ids = torch.empty((rows, k), dtype=torch.int32, device=dev)
    top = torch.empty((rows, k), dtype=torch.float32, device=dev)
    _check(_lib.load().bi_logprobs_top(
        logits.data_ptr(), rows, vocab, ld, targets.data_ptr() if targets is not None else None,
        lp.data_ptr() if targets is not None else None, lse.data_ptr(), entropy.data_ptr(), k,
        ids.data_ptr(), top.data_ptr(), _stream(stream)), "bi_logprobs_top")
    return (lp if targets is not None else None), lse, entropy, ids, top
