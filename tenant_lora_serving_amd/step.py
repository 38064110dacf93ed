"""Python binding of libstep.so (the C ABI in include/step.h): the operators a
serving step runs around the routed LoRA delta.

    rms_norm        norm with the residual's addition and an 8-bit copy
    lora_linear     the shared projection with every row's adapter added
    kv_append       new keys and values into the paged cache, turned by position
    paged_attention attention over that cache, shared prefixes read once
    token_logprobs  log probabilities, ranks, entropies, top alternatives

Argument marshalling only, as in `lora`: every function checks types, devices
and shapes, passes raw device pointers and the current HIP stream to the
library, and raises LoraError on a non-zero status.  There is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch

from .lora import LoraError, _c_f, _c_i32, _c_i64, _c_p, _c_sz, _dev

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libstep.so")
MAX_TOP = 32

EXPORTED = ["step_rms_norm", "step_lora_linear_workspace_bytes", "step_lora_linear",
            "step_token_logprobs_workspace_bytes", "step_token_logprobs", "step_kv_append",
            "step_paged_attention_workspace_bytes", "step_paged_attention", "step_status_string"]

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
        L.step_kv_append.restype = ctypes.c_int
        L.step_kv_append.argtypes = [_c_p, _c_i64, _c_p, _c_i64, _c_p, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p,
                                     _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32,
                                     _c_p, _c_p, _c_p, _c_i64, _c_p]
        L.step_paged_attention_workspace_bytes.restype = _c_sz
        L.step_paged_attention_workspace_bytes.argtypes = [_c_i32] * 5
        L.step_paged_attention.restype = ctypes.c_int
        L.step_paged_attention.argtypes = [_c_p, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_i64,
                                           _c_i64, _c_i64, _c_i32, _c_i32, _c_p, _c_p, _c_p, _c_i64, _c_i32, _c_p, _c_p,
                                           _c_i32, _c_i32, _c_f, _c_i32, _c_p, _c_i64, _c_i32, _c_p, _c_p, _c_p, _c_i64,
                                           _c_p, _c_p, _c_sz, _c_p]
        L.step_status_string.restype = ctypes.c_char_p
        L.step_status_string.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise LoraError(fn, status, lib().step_status_string(status).decode())


def _fits(fn: str, *sizes):
    """Every size of the call is a 32-bit one (ctypes would hand over the low half of others)."""
    if max(sizes) > 0x7fffffff:
        _check(fn, -2)


_raw_stream = torch._C._cuda_getCurrentRawStream   # what torch.cuda.current_stream() wraps, at a fortieth of its time


def _on(stream, fn, args, kw):
    """The call on another stream: what it allocates belongs to that stream."""
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


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


def _arg(t: torch.Tensor, name: str, dtype, shape, dev: int):
    """A contiguous tensor of this type and shape on device `dev`: its pointer."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev \
            and t.is_contiguous():
        return t.data_ptr()
    _dev(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on another device")


def _same(name: str, got, want):
    if tuple(got) != tuple(want):
        raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(got)}")


def _device(x: torch.Tensor, *rest) -> int:
    """The device of the call: the current one, which holds every tensor."""
    dev = x.get_device()
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on device {dev}, which is not the current one")
    return dev


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
    if stream is not None:
        return _on(stream, rms_norm, (x, weight, eps), dict(residual=residual, bf16=bf16, quant=quant,
                                                            residual_out=residual_out))
    xp, ldx = _rows(x, "x", torch.bfloat16)
    n, h = x.shape
    _fits("step_rms_norm", n, h)
    dev = _device(x, residual)
    wp = _arg(weight, "weight", torch.bfloat16, (h,), dev)
    rp, ldr, sp = None, 0, None
    if residual is not None:
        rp, ldr = _rows(residual, "residual", torch.bfloat16)
        _same("residual", residual.shape, (n, h))
        if residual_out is None:
            residual_out = torch.empty_like(x)
        sp = _arg(residual_out, "residual_out", torch.bfloat16, (n, h), dev)
        if sp == rp:
            ldr = h if n <= 1 else ldr
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    y = torch.empty_like(x) if bf16 else None
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn) if quant else None
    q_scale = x.new_empty(n, dtype=torch.float32) if quant else None
    st = lib().step_rms_norm(xp, ldx, rp, ldr, wp, n, h, eps, sp, y.data_ptr() if bf16 else None,
                             q.data_ptr() if quant else None, q_scale.data_ptr() if quant else None, _raw_stream(dev))
    if st:
        _check("step_rms_norm", st)
    return NormResult(y, residual_out, q, q_scale)


# ---------------------------------------------------------------- projection
def linear_workspace(n: int, k: int, out: int, num_slices: int, max_rank: int, device="cuda") -> torch.Tensor:
    """A workspace for calls of at most these sizes."""
    _fits("step_lora_linear_workspace_bytes", n, k, out, num_slices, max_rank)
    b = int(lib().step_lora_linear_workspace_bytes(n, k, out, num_slices, max_rank))
    return torch.zeros(max(b, 16), dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=256)
def _slice_array(sizes: tuple) -> tuple:
    """The widths as the library takes them, and their sum."""
    return (_c_i32 * len(sizes))(*sizes), sum(sizes)


def lora_linear(x: torch.Tensor, w: torch.Tensor, a_pool: torch.Tensor, b_pool: torch.Tensor, scale: torch.Tensor,
                slice_sizes, slot: torch.Tensor, *, xq: Optional[torch.Tensor] = None,
                x_scale: Optional[torch.Tensor] = None, w_scale: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[i] = x[i] @ w^T + scale[s] * (x[i] @ A_s^T) @ B_s^T for s = slot[i]
    (no second term for a slot outside [0, num_slots)), in bf16.
    w [N, k] bf16; or, with xq [n, k] (float8_e4m3fn), x_scale [n] and w_scale
    [N], w in float8_e4m3fn and the first term from the 8-bit rows.
    a_pool [S, L, R, k], b_pool [S, N, R], slice_sizes L widths that add up to N."""
    if stream is not None:
        return _on(stream, lora_linear, (x, w, a_pool, b_pool, scale, slice_sizes, slot),
                   dict(xq=xq, x_scale=x_scale, w_scale=w_scale, out=out, ws=ws))
    if a_pool.dim() != 4 or b_pool.dim() != 3 or w.dim() != 2:
        raise ValueError("a_pool must be [S, L, R, k], b_pool [S, N, R] and w [N, k]")
    S, L, R, k = a_pool.shape
    N = w.shape[0]
    n = x.shape[0]
    xp, ldx = _rows(x, "x", torch.bfloat16)
    if x.shape[1] != k:
        _same("x", x.shape, (n, k))
    _fits("step_lora_linear", n, k, N, S, L, R)
    dev = _device(x, xq, out, ws)
    sizes, total = _slice_array(tuple(slice_sizes))
    if len(sizes) != L or total != N:
        raise ValueError("slice sizes do not match the pools")
    xqp, ldxq, xsp, wsp, w_type = None, 0, None, None, torch.bfloat16
    if xq is not None:
        if x_scale is None or w_scale is None:
            raise ValueError("xq needs x_scale and w_scale")
        xqp, ldxq = _rows(xq, "xq", torch.float8_e4m3fn)
        _same("xq", xq.shape, (n, k))
        xsp = _arg(x_scale, "x_scale", torch.float32, (n,), dev)
        wsp = _arg(w_scale, "w_scale", torch.float32, (N,), dev)
        w_type = torch.float8_e4m3fn
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale belong to the 8-bit form, which needs xq")
    if out is None:
        out = x.new_empty((n, N))
        yp, ldy = out.data_ptr(), N
    else:
        _same("out", out.shape, (n, N))
        yp, ldy = _rows(out, "out", torch.bfloat16)
    if ws is None:
        ws = linear_workspace(n, k, N, L, R, x.device)
    st = lib().step_lora_linear(xp, ldx, n, k, xqp, ldxq, xsp, _arg(w, "w", w_type, (N, k), dev), wsp,
                                _arg(a_pool, "a_pool", torch.bfloat16, (S, L, R, k), dev),
                                _arg(b_pool, "b_pool", torch.bfloat16, (S, N, R), dev),
                                _arg(scale, "scale", torch.float32, (S,), dev), S, L, sizes, R,
                                _arg(slot, "slot", torch.int32, (n,), dev), yp, ldy, _dev(ws, "ws", torch.uint8),
                                ws.numel(), _raw_stream(dev))
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
    """A workspace for calls of at most n rows, v logits a row and `top` alternatives."""
    _fits("step_token_logprobs_workspace_bytes", n, v, top)
    b = int(lib().step_token_logprobs_workspace_bytes(n, v, top))
    return torch.zeros(max(b, 16), dtype=torch.uint8, device=device)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, *, ws: Optional[torch.Tensor] = None,
                   stream=None) -> LogprobResult:
    """Per row of logits ([n, v], bf16 or float32): the log probability and the
    rank of tokens[i] (int32; negative: none asked for), the entropy, and the
    `top` most likely tokens with their log probabilities."""
    if stream is not None:
        return _on(stream, token_logprobs, (logits, tokens, top), dict(ws=ws))
    lp, ld = _rows(logits, "logits", torch.bfloat16, torch.float32)
    n, v = logits.shape
    _fits("step_token_logprobs", n, v, top)
    dev = _device(logits, ws)
    tp = _arg(tokens, "tokens", torch.int32, (n,), dev)
    logprob, rank = torch.empty_like(tokens, dtype=torch.float32), torch.empty_like(tokens)
    entropy = torch.empty_like(logprob)
    ids = best = ip = bp = None
    if top > 0:
        ids, best = tokens.new_empty((n, top)), tokens.new_empty((n, top), dtype=torch.float32)
        ip, bp = ids.data_ptr(), best.data_ptr()
    if ws is None:
        ws = logprobs_workspace(n, v, top, logits.device)
    st = lib().step_token_logprobs(lp, ld, 1 if logits.dtype == torch.float32 else 0, n, v, tp, top,
                                   logprob.data_ptr(), rank.data_ptr(), entropy.data_ptr(), ip, bp,
                                   _dev(ws, "ws", torch.uint8), ws.numel(), _raw_stream(dev))
    if st:
        _check("step_token_logprobs", st)
    return LogprobResult(logprob, rank, entropy, ids, best)


# ---------------------------------------------------------------- the paged cache
def _heads(t: torch.Tensor, name: str) -> tuple:
    """A bf16 tensor [rows, heads, dim] whose rows are contiguous: (pointer, row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, dim]")
    n, heads, dim = t.shape
    row, head, unit = t.stride()
    if (unit != 1 and dim > 1) or (head != dim and heads > 1):
        raise ValueError(f"{name} must hold the heads of a row side by side")
    return t.data_ptr(), row if n > 1 else heads * dim


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale, v_scale, kv: int, dim: int, dev: int) -> tuple:
    """The cache as the library takes it: two pointers, three strides, pages and their tokens, two scales."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        if t.dim() != 4 or t.shape[2] != kv or t.shape[3] != dim:
            raise ValueError(f"{name} must be [pages, page, {kv}, {dim}]")
    if k_cache.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or v_cache.dtype is not k_cache.dtype:
        raise TypeError("k_cache and v_cache must both be bfloat16 or both float8_e4m3fn")
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    pages, page = k_cache.shape[:2]
    _fits("the cache", pages, page)
    ps, ts, hs, unit = k_cache.stride()
    if unit != 1:
        raise ValueError("k_cache and v_cache must have contiguous heads")
    ksp = vsp = None
    if k_cache.dtype is torch.float8_e4m3fn:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        ksp = _arg(k_scale, "k_scale", torch.float32, (kv,), dev)
        vsp = _arg(v_scale, "v_scale", torch.float32, (kv,), dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to an 8-bit cache")
    return k_cache.data_ptr(), v_cache.data_ptr(), ps, ts, hs, pages, page, ksp, vsp


def rotation_table(positions: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """kv_append's rotation for positions 0 .. positions: [positions, rot] float32, row t the
    cosines and then the sines of t base^(-2 i / rot) for i < rot / 2, from angles in 64 bits."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    angles = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * base ** (-i / rot)
    return torch.cat([angles.cos(), angles.sin()], dim=1).float()


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, place: torch.Tensor, *,
              q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
              rotation: Optional[torch.Tensor] = None, neighbours: bool = False, k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
              stream=None) -> Optional[torch.Tensor]:
    """k, v [n, kv_heads, dim] bf16 into the cache ([pages, page, kv_heads, dim], bf16 or
    float8_e4m3fn with a scale a head), token t to place[t] = page number * page + place in the
    page (int32; a place outside the cache: not stored).  With rotation ([R, rot] float32, see
    rotation_table) and positions [n] int32, the first rot columns of every head of k and q are
    turned by the position's angles, in pairs of columns (i, i + rot / 2), or (2 i, 2 i + 1)
    with neighbours.  Returns the turned q [n, heads, dim], in q_out if given (it may be q)."""
    if stream is not None:
        return _on(stream, kv_append, (k, v, k_cache, v_cache, place),
                   dict(q=q, positions=positions, rotation=rotation, neighbours=neighbours, k_scale=k_scale,
                        v_scale=v_scale, q_out=q_out))
    kp, ldk = _heads(k, "k")
    vp, ldv = _heads(v, "v")
    n, kv, dim = k.shape
    _same("v", v.shape, k.shape)
    dev = _device(k, v, k_cache, v_cache, q, q_out)
    qp, ldq, op, ldo, heads = None, 0, None, 0, kv
    if q is not None:
        qp, ldq = _heads(q, "q")
        heads = q.shape[1]
        _same("q", q.shape, (n, heads, dim))
        if q_out is None:
            q_out = q.new_empty((n, heads, dim))
        op, ldo = _heads(q_out, "q_out")
        _same("q_out", q_out.shape, q.shape)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _fits("step_kv_append", n, heads, kv, dim)
    pp = rp = None
    rows = rot = 0
    if rotation is not None:
        if positions is None:
            raise ValueError("rotation needs positions")
        rp = _dev(rotation, "rotation", torch.float32)
        if rotation.dim() != 2:
            raise ValueError("rotation must be [positions, rot]")
        if rotation.get_device() != dev:
            raise ValueError("rotation is on another device")
        rows, rot = rotation.shape
        _fits("step_kv_append", rows, rot)
        pp = _arg(positions, "positions", torch.int32, (n,), dev)
    elif positions is not None:
        raise ValueError("positions need a rotation")
    kc, vc, ps, ts, hs, pages, page, ksp, vsp = _cache(k_cache, v_cache, k_scale, v_scale, kv, dim, dev)
    st = lib().step_kv_append(qp, ldq, kp, ldk, vp, ldv, n, heads, kv, dim, pp, rp, rows, rot, 1 if neighbours else 0,
                              _arg(place, "place", torch.int32, (n,), dev), kc, vc, ps, ts, hs, pages, page, ksp, vsp,
                              op, ldo, _raw_stream(dev))
    if st:
        _check("step_kv_append", st)
    return q_out


class Prefixes(NamedTuple):
    """Keys that requests share: prefix p, lens[p] keys on the pages pages[p], is that of the
    requests starts[p] .. starts[p + 1] of the batch."""
    pages: torch.Tensor    # [P, columns] int32
    lens: torch.Tensor     # [P] int32
    starts: torch.Tensor   # [P + 1] int32, ascending


class AttentionResult(NamedTuple):
    out: torch.Tensor             # [n, heads, dim] bf16
    lse: Optional[torch.Tensor]   # [n, heads] float32, with lse=True


_ZEROED = 4096   # STEP_ATTENTION_ZEROED


def attention_workspace(n: int, heads: int, kv_heads: int, dim: int, prefixes: bool = False,
                        device="cuda") -> torch.Tensor:
    """A workspace for calls of at most n rows of these heads, with shared prefixes if asked for."""
    _fits("step_paged_attention_workspace_bytes", n, heads, kv_heads, dim)
    b = int(lib().step_paged_attention_workspace_bytes(n, heads, kv_heads, dim, 1 if prefixes else 0))
    ws = torch.empty(max(b, 16), dtype=torch.uint8, device=device)
    ws[:_ZEROED].zero_()
    return ws


def _table(t: torch.Tensor, name: str, rows: int, dev: int) -> tuple:
    """A table of page numbers: (pointer, row stride, columns)."""
    p, ld = _rows(t, name, torch.int32)
    if t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got {t.shape[0]}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    cols = t.shape[1]
    _fits("step_paged_attention", cols)
    return p, ld, cols   # (rows that overlap, as an expanded table's do, are refused by the library)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor,
                    lens: torch.Tensor, *, starts: Optional[torch.Tensor] = None, max_rows: Optional[int] = None,
                    scale: Optional[float] = None, causal: bool = True, prefix: Optional[Prefixes] = None,
                    k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None, lse: bool = False,
                    out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None) -> AttentionResult:
    """Attention of the rows q [n, heads, dim] bf16 over the paged cache.  Request b reads lens[b]
    keys (int32) on the pages pages[b] (int32 page numbers; rows of the table do not overlap) for
    its row b or, with starts ([requests + 1] int32, ascending), its rows starts[b] ..
    starts[b + 1], at most max_rows of them (which only decides how the work is cut).  causal: a
    request's rows are its last tokens and see no later key.  prefix: keys that groups of
    requests share and see before their own.  scale: dim ** -0.5 by default.  A row without keys
    is 0.  Rows of no request stay as they are in `out`, and are not written in a new result."""
    if stream is not None:
        return _on(stream, paged_attention, (q, k_cache, v_cache, pages, lens),
                   dict(starts=starts, max_rows=max_rows, scale=scale, causal=causal, prefix=prefix, k_scale=k_scale,
                        v_scale=v_scale, lse=lse, out=out, ws=ws))
    qp, ldq = _heads(q, "q")
    n, heads, dim = q.shape
    dev = _device(q, k_cache, v_cache, out, ws)
    kv = k_cache.shape[2] if k_cache.dim() == 4 else 0
    _fits("step_paged_attention", n, heads, dim)
    kc, vc, ps, ts, hs, num_pages, page, ksp, vsp = _cache(k_cache, v_cache, k_scale, v_scale, kv, dim, dev)
    requests = lens.shape[0] if lens.dim() == 1 else -1
    lp = _arg(lens, "lens", torch.int32, (max(requests, 0),), dev)
    tp, ldt, cols = _table(pages, "pages", requests, dev)
    sp = None
    if starts is not None:
        sp = _arg(starts, "starts", torch.int32, (requests + 1,), dev)
        if max_rows is None:
            max_rows = max(n, 1)
        _fits("step_paged_attention", max_rows)
    elif requests != n:
        raise ValueError(f"lens must have a length for each of the {n} rows, or starts be given")
    P, ptp, ldp, pcols, plp, psp = 0, None, 0, 0, None, None
    if prefix is not None:
        P = prefix.lens.shape[0] if prefix.lens.dim() == 1 else -1
        plp = _arg(prefix.lens, "prefix.lens", torch.int32, (max(P, 0),), dev)
        ptp, ldp, pcols = _table(prefix.pages, "prefix.pages", P, dev)
        psp = _arg(prefix.starts, "prefix.starts", torch.int32, (P + 1,), dev)
    if out is None:
        out = q.new_empty((n, heads, dim))
    else:
        _same("out", out.shape, q.shape)
    op, ldo = _heads(out, "out")
    sums = q.new_empty((n, heads), dtype=torch.float32) if lse else None
    if ws is None and heads and kv and heads % kv == 0:
        ws = attention_workspace(n, heads, kv, dim, P > 0, q.device)
    st = lib().step_paged_attention(qp, ldq, n, requests, heads, kv, dim, kc, vc, ps, ts, hs, num_pages, page, ksp, vsp,
                                    tp, ldt, cols, lp, sp, max_rows or 1, 1 if causal else 0,
                                    dim ** -0.5 if scale is None else scale, P, ptp, ldp, pcols, plp, psp, op, ldo,
                                    sums.data_ptr() if lse else None,
                                    _dev(ws, "ws", torch.uint8) if ws is not None else None,
                                    ws.numel() if ws is not None else 0, _raw_stream(dev))
    if st:
        _check("step_paged_attention", st)
    return AttentionResult(out, sums)
