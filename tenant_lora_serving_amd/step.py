"""Python binding of libstep.so (the C ABI in include/step.h): the operators a
serving step runs around the routed LoRA delta.

    rms_norm        norm with the residual's addition and an 8-bit copy
    lora_linear     the shared projection with every row's adapter added
    token_logprobs  log probabilities, ranks, entropies, top alternatives

Argument marshalling only, as in `lora`: every function checks types, devices
and shapes, passes raw device pointers and the current HIP stream to the
library, and raises LoraError on a non-zero status.  There is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

from .lora import LoraError, _c_f, _c_i32, _c_i64, _c_p, _c_sz, _dev, _stream

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libstep.so")
MAX_TOP = 32

EXPORTED = ["step_rms_norm", "step_lora_linear_workspace_bytes", "step_lora_linear",
            "step_token_logprobs_workspace_bytes", "step_token_logprobs", "step_status_string"]

_lib = None


def lib():
    """Load libstep.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m tenant_lora_serving_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.step_rms_norm.restype = ctypes.c_int
        L.step_rms_norm.argtypes = [_c_p, _c_i64, _c_p, _c_i64, _c_p, _c_i32, _c_i32, _c_f, _c_p, _c_p, _c_p,
                                    _c_p, _c_p]
        L.step_lora_linear_workspace_bytes.restype = _c_sz
        L.step_lora_linear_workspace_bytes.argtypes = [_c_i32] * 5
        L.step_lora_linear.restype = ctypes.c_int
        L.step_lora_linear.argtypes = [_c_p, _c_i64, _c_i32, _c_i32, _c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p,
                                       _c_p, _c_i32, _c_i32, _c_p, _c_i32, _c_p, _c_p, _c_i64, _c_p, _c_sz, _c_p]
        L.step_token_logprobs_workspace_bytes.restype = _c_sz
        L.step_token_logprobs_workspace_bytes.argtypes = [_c_i32] * 3
        L.step_token_logprobs.restype = ctypes.c_int
        L.step_token_logprobs.argtypes = [_c_p, _c_i64, _c_i32, _c_i32, _c_i32, _c_p, _c_i32, _c_p, _c_p, _c_p,
                                          _c_p, _c_p, _c_p, _c_sz, _c_p]
        L.step_status_string.restype = ctypes.c_char_p
        L.step_status_string.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise LoraError(fn, status, lib().step_status_string(status).decode())


def _rows(t: torch.Tensor, name: str, *dtypes) -> tuple:
    """A 2-D tensor of rows with unit column stride: (pointer, row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    # (the stride of a single row, or of none, means nothing)
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 16) * 16


def _same(name: str, got, want):
    if tuple(got) != tuple(want):
        raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(got)}")


# ---------------------------------------------------------------- norm
class NormResult(NamedTuple):
    y: Optional[torch.Tensor]          # [n, h] bf16, with bf16=True
    residual: Optional[torch.Tensor]   # [n, h] bf16: x + residual, where a residual was given
    q: Optional[torch.Tensor]          # [n, h] float8_e4m3fn, with quant=True
    q_scale: Optional[torch.Tensor]    # [n] float32: y = q * q_scale[:, None] up to q's rounding


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, *, residual: Optional[torch.Tensor] = None,
             bf16: bool = True, quant: bool = False, residual_out: Optional[torch.Tensor] = None,
             stream=None) -> NormResult:
    """s = x + residual; y = s / sqrt(mean(s^2) + eps) * weight per row, from
    the unrounded s.  bf16: return y; quant: return its e4m3 copy with one
    scale a row.  residual_out: where to put the rounded s (it may be
    `residual` itself, which is then updated in place)."""
    xp, ldx = _rows(x, "x", torch.bfloat16)
    n, h = x.shape
    wp = _dev(weight, "weight", torch.bfloat16)
    _same("weight", weight.shape, (h,))
    dev = x.device
    rp, ldr, sp = None, 0, None
    if residual is not None:
        rp, ldr = _rows(residual, "residual", torch.bfloat16)
        _same("residual", residual.shape, (n, h))
        if residual_out is None:
            residual_out = torch.empty((n, h), dtype=torch.bfloat16, device=dev)
        else:
            _same("residual_out", residual_out.shape, (n, h))
        sp = _dev(residual_out, "residual_out", torch.bfloat16)
        if sp == rp:
            ldr = h if n <= 1 else ldr
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    y = torch.empty((n, h), dtype=torch.bfloat16, device=dev) if bf16 else None
    q = torch.empty((n, h), dtype=torch.float8_e4m3fn, device=dev) if quant else None
    q_scale = torch.empty((n,), dtype=torch.float32, device=dev) if quant else None
    st = lib().step_rms_norm(xp, ldx, rp, ldr, wp, n, h, eps, sp, y.data_ptr() if bf16 else None,
                             q.data_ptr() if quant else None, q_scale.data_ptr() if quant else None, _stream(stream))
    if st:
        _check("step_rms_norm", st)
    return NormResult(y, residual_out, q, q_scale)


# ---------------------------------------------------------------- projection
def linear_workspace(n: int, k: int, out: int, num_slices: int, max_rank: int, device="cuda") -> torch.Tensor:
    b = int(lib().step_lora_linear_workspace_bytes(n, k, out, num_slices, max_rank))
    return torch.zeros(max(b, 16), dtype=torch.uint8, device=device)


def lora_linear(x: torch.Tensor, w: torch.Tensor, a_pool: torch.Tensor, b_pool: torch.Tensor, scale: torch.Tensor,
                slice_sizes, slot: torch.Tensor, *, xq: Optional[torch.Tensor] = None,
                x_scale: Optional[torch.Tensor] = None, w_scale: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[i] = x[i] @ w^T + scale[s] * (x[i] @ A_s^T) @ B_s^T for s = slot[i]
    (no second term for a slot outside [0, num_slots)), in bf16.
    w [N, k] bf16; or, with xq [n, k] (float8_e4m3fn), x_scale [n] and w_scale
    [N], w in float8_e4m3fn and the first term from the 8-bit rows.
    a_pool [S, L, R, k], b_pool [S, N, R], slice_sizes L widths that add up to N."""
    if a_pool.dim() != 4 or b_pool.dim() != 3 or w.dim() != 2:
        raise ValueError("a_pool must be [S, L, R, k], b_pool [S, N, R] and w [N, k]")
    S, L, R, k = a_pool.shape
    N = w.shape[0]
    n = x.shape[0]
    xp, ldx = _rows(x, "x", torch.bfloat16)
    _same("x", x.shape, (n, k))
    _same("w", w.shape, (N, k))
    _same("b_pool", b_pool.shape, (S, N, R))
    _same("scale", scale.shape, (S,))
    _same("slot", slot.shape, (n,))
    if len(slice_sizes) != L or sum(slice_sizes) != N:
        raise ValueError("slice sizes do not match the pools")
    xqp, ldxq, xsp, wsp, w_type = None, 0, None, None, torch.bfloat16
    if xq is not None:
        if x_scale is None or w_scale is None:
            raise ValueError("xq needs x_scale and w_scale")
        xqp, ldxq = _rows(xq, "xq", torch.float8_e4m3fn)
        _same("xq", xq.shape, (n, k))
        _same("x_scale", x_scale.shape, (n,))
        _same("w_scale", w_scale.shape, (N,))
        xsp, wsp = _dev(x_scale, "x_scale", torch.float32), _dev(w_scale, "w_scale", torch.float32)
        w_type = torch.float8_e4m3fn
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale belong to the 8-bit form, which needs xq")
    if out is None:
        out = torch.empty((n, N), dtype=torch.bfloat16, device=x.device)
    else:
        _same("out", out.shape, (n, N))
    yp, ldy = _rows(out, "out", torch.bfloat16)
    if ws is None:
        ws = linear_workspace(n, k, N, L, R, x.device)
    st = lib().step_lora_linear(xp, ldx, n, k, xqp, ldxq, xsp, _dev(w, "w", w_type), wsp,
                                _dev(a_pool, "a_pool", torch.bfloat16), _dev(b_pool, "b_pool", torch.bfloat16),
                                _dev(scale, "scale", torch.float32), S, L, (_c_i32 * L)(*slice_sizes), R,
                                _dev(slot, "slot", torch.int32), yp, ldy, _dev(ws, "ws", torch.uint8), ws.numel(),
                                _stream(stream))
    if st:
        _check("step_lora_linear", st)
    return out


# ---------------------------------------------------------------- log probabilities
class LogprobResult(NamedTuple):
    logprob: torch.Tensor                  # [n] float32
    rank: torch.Tensor                     # [n] int32: 1 + the number of larger logits; 0 without a token
    entropy: torch.Tensor                  # [n] float32, in nats
    top_ids: Optional[torch.Tensor]        # [n, top] int32, -1 past the last unmasked logit
    top_logprobs: Optional[torch.Tensor]   # [n, top] float32


def logprobs_workspace(n: int, v: int, top: int = 0, device="cuda") -> torch.Tensor:
    b = int(lib().step_token_logprobs_workspace_bytes(n, v, top))
    return torch.zeros(max(b, 16), dtype=torch.uint8, device=device)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, *, ws: Optional[torch.Tensor] = None,
                   stream=None) -> LogprobResult:
    """Per row of logits ([n, v], bf16 or float32): the log probability and the
    rank of tokens[i] (int32; negative: none asked for), the entropy, and the
    `top` most likely tokens with their log probabilities."""
    lp, ld = _rows(logits, "logits", torch.bfloat16, torch.float32)
    n, v = logits.shape
    _same("tokens", tokens.shape, (n,))
    dev = logits.device
    # one block for the five outputs: fewer allocations in a decode step
    flat = torch.empty((n * (3 + 2 * top),), dtype=torch.float32, device=dev)
    logprob, rank, entropy = flat[:n], flat[n:2 * n].view(torch.int32), flat[2 * n:3 * n]
    ids = best = None
    if top > 0:
        ids = flat[3 * n:(3 + top) * n].view(torch.int32).view(n, top)
        best = flat[(3 + top) * n:].view(n, top)
    if ws is None:
        ws = logprobs_workspace(n, v, top, dev)
    base = flat.data_ptr()
    st = lib().step_token_logprobs(lp, ld, 1 if logits.dtype == torch.float32 else 0, n, v,
                                   _dev(tokens, "tokens", torch.int32), top, base, base + 4 * n, base + 8 * n,
                                   base + 12 * n if top > 0 else None, base + (12 + 4 * top) * n if top > 0 else None,
                                   _dev(ws, "ws", torch.uint8), ws.numel(), _stream(stream))
    if st:
        _check("step_token_logprobs", st)
    return LogprobResult(logprob, rank, entropy, ids, best)
