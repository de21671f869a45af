"""The attention half of a decoder layer on torch tensors (C ABI: include/maple_attn.h).

    int8_linear        rows quantised to int8 times int8 weights (projections, output head)
    qk_norm_rope       norm and rotation of query and key heads, appended to the 4-bit cache in the same pass
    kv_read            the values that the cache holds at given slots
    prompt_attention   causal attention over packed prompts
    cached_attention   attention of one new token per sequence over the cache

Each function checks its tensors, allocates outputs and scratch with torch on
the tensors' device and launches on that device's current stream; none
synchronises, and all may be captured into a CUDA graph.  A tensor of the wrong
type, shape, stride or device raises ValueError, an error of the library
MapleError.  What only the kernels can see (a page number outside the cache) is
reported in `flags`, an int32 tensor of one element that the caller zeroes and
reads (MAPLE_FLAG_* bits).  No gradients: these are serving operators, and a call
with a tensor that requires one is refused unless gradients are off.

Cache: uint8 [num_pages][kv_heads][page bytes], made by kv_pages(); a token's
slot is page * page_size + row.
"""
from __future__ import annotations

import ctypes as C
import struct

import torch

from . import MapleError, lib

MAPLE_BF16, MAPLE_FP16, MAPLE_FP32 = 0, 1, 2

_HEAD_TYPES = {torch.bfloat16: MAPLE_BF16, torch.float16: MAPLE_FP16}
_OUT_TYPES = {torch.bfloat16: MAPLE_BF16, torch.float32: MAPLE_FP32}

# the argument structs of include/maple_attn.h, field for field
_LINEAR = struct.Struct("=7Qq Q 4q 2i")
_ROPE = struct.Struct("=12Q 5q 7i f")
_READ = struct.Struct("=5Q 2q 4i")
_PROMPT = struct.Struct("=8Q 5q 7i f")
_CACHED = struct.Struct("=6Q q Q 3q 8i f 4x")

_fn = None
_calls = {}     # the entry points by name
_PAGE_SIZES = (16, 32, 64)
_CONTIGUOUS = torch.contiguous_format


def _lib():
    global _fn
    if _fn is None:
        L = lib()
        P, I32, I64 = C.c_void_p, C.c_int32, C.c_int64
        for name in ("linear", "qk_norm_rope", "kv_read", "prompt", "cached"):
            f = getattr(L, "maple_attn_" + name)
            f.argtypes, f.restype = [C.c_char_p, P], C.c_int
            _calls[name] = f
        L.maple_attn_page_bytes.argtypes, L.maple_attn_page_bytes.restype = [I32, I32], I64
        L.maple_attn_linear_workspace.argtypes, L.maple_attn_linear_workspace.restype = [I64] * 3 + [I32], I64
        L.maple_attn_cached_workspace.argtypes, L.maple_attn_cached_workspace.restype = [I32] * 7, I64
        _fn = L
    return _fn


# The device and stream that torch has current, without building the Python objects around them: these functions are
# called once per operator and token.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(name: str, form: struct.Struct, fields: tuple, dev: int) -> None:
    """Launch with the argument struct's fields on the device's current stream, with that device current."""
    if _fn is None:
        _lib()
    try:
        args = form.pack(*fields)
    except (struct.error, OverflowError) as e:      # (sizes beyond 32 bits, a scale beyond fp32, what is no number)
        raise ValueError(f"an argument does not fit its field: {e}") from None
    stream = _raw_stream(dev)
    if dev == _current_device():
        rc = _calls[name](args, stream)
    else:
        with torch.cuda.device(dev):
            rc = _calls[name](args, stream)
    if rc:
        raise MapleError(rc, "maple_attn_" + name)


def _size(n: int, what: str) -> int:
    if n < 0:
        raise MapleError(n, what)
    return n


def _device(first, *others) -> int:
    """The CUDA device index that all tensors (None aside) are on."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")
    return dev


def _refuse_gradient() -> None:
    """For a call with a tensor that requires a gradient."""
    if torch.is_grad_enabled():
        raise ValueError("no gradients are computed here: detach the tensors that require one, or call under torch.no_grad()")


def _flags(t) -> int:
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.numel() != 1:
        raise ValueError("flags must be one int32")
    return t.data_ptr()


def _vector(t, dtype, n: int, what: str) -> int:
    """Address of a contiguous vector of n values (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.numel() != n or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(what)
    return t.data_ptr()


def _heads(t, dtype, what: str):
    """A [tokens][heads][head_dim] tensor whose heads are contiguous within a token; returns its shape and token stride."""
    if t.dim() != 3 or t.dtype is not dtype:
        raise ValueError(what)
    n, h, d = t.shape
    step, head, one = t.stride()
    if one != 1 or (head != d and h != 1):
        raise ValueError(what)
    return n, h, d, (step if n > 1 else h * d)


def _overlap(out, t) -> bool:
    """Whether the contiguous tensor `out` reaches into the memory from the first to the last element of t."""
    if t is None or not out.numel() or not t.numel():
        return False
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    a, b = out.data_ptr(), t.data_ptr()
    return a < b + (last + 1) * t.element_size() and b < a + out.numel() * out.element_size()


def kv_pages(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> torch.Tensor:
    """A zeroed cache of `num_pages` pages of `page_size` tokens (16, 32 or 64) with head_dim 64 or 128."""
    b = _size(_lib().maple_attn_page_bytes(head_dim, page_size), "maple_attn_page_bytes")
    return torch.zeros(num_pages, kv_heads, b, dtype=torch.uint8, device=device)


def _pages(pages, head_dim: int, page_size: int | None):
    """(num_pages, kv_heads, page_size) of a cache tensor."""
    if pages.dtype is not torch.uint8 or pages.dim() != 3 or not pages.is_contiguous():
        raise ValueError("pages must be a contiguous uint8 [num_pages][kv_heads][page bytes]")
    P, Hkv, size = pages.shape
    n = 4 * size // (5 * head_dim) if head_dim else 0
    if 4 * size != 5 * head_dim * n or n not in _PAGE_SIZES or page_size not in (None, n):
        raise ValueError("the pages do not fit this head_dim" + ("" if page_size is None else " and page_size"))
    return P, Hkv, n


def int8_linear(x: torch.Tensor, weight: torch.Tensor, alpha: torch.Tensor, bias: torch.Tensor | None = None,
                resid: torch.Tensor | None = None, normalise: bool = False, out_dtype: torch.dtype = torch.float32,
                out: torch.Tensor | None = None, flags: torch.Tensor | None = None) -> torch.Tensor:
    """y = (q_x weight^T) * (s_x alpha) (+ bias) (+ resid), q_x and s_x the int8 absmax codes and scales of x's rows.

    x bf16 [T][K] (rows may be strided), or the fp32 residual stream with `normalise` (its RMS-normed rows, rounded to
    bf16, are quantised).  weight int8 [N][K], alpha fp32 [N], bias fp32 [N], resid fp32 [T][N].  `out`, where given, sets
    the output's type; it may be resid and overlaps nothing else that is read.  A row of x with a NaN or an infinity gives a
    row of NaN.
    """
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [T][K] and weight [N][K]")
    T, K = x.shape
    N, Kw = weight.shape
    if K != Kw:
        raise ValueError("x must be [T][K] and weight [N][K]")
    step, one = x.stride()
    if (x.requires_grad or (alpha is not None and alpha.requires_grad) or (bias is not None and bias.requires_grad) or
            (resid is not None and resid.requires_grad) or (out is not None and out.requires_grad)):
        _refuse_gradient()
    dev = _device(x, weight, alpha, bias, resid, out, flags)
    if x.dtype is not (torch.float32 if normalise else torch.bfloat16):
        raise ValueError("x must be bf16, or fp32 with normalise")
    if one != 1 and K != 1:
        raise ValueError("the rows of x must be contiguous")
    if weight.dtype is not torch.int8 or not weight.is_contiguous():
        raise ValueError("weight must be contiguous int8")
    if resid is not None and (resid.dtype is not torch.float32 or resid.shape != (T, N) or not resid.is_contiguous()):
        raise ValueError("resid must be contiguous fp32 [T][N]")
    if out is None:
        out = x.new_empty((T, N), dtype=out_dtype)
    elif out.shape != (T, N) or not out.is_contiguous():
        raise ValueError("out must be contiguous [T][N]")
    elif _overlap(out, x):
        raise ValueError("x must not be out or overlap it")
    elif resid is not None and _overlap(out, resid) and (out.dtype is not torch.float32 or out.data_ptr() != resid.data_ptr()):
        raise ValueError("resid must be out or not overlap it")
    elif _overlap(out, weight) or _overlap(out, alpha) or _overlap(out, bias):
        raise ValueError("out must not overlap weight, alpha or bias")
    ydt = _OUT_TYPES.get(out.dtype)
    if ydt is None:
        raise ValueError("the output must be bf16 or fp32")
    n = _size((_fn or _lib()).maple_attn_linear_workspace(T, K, N, 1 if normalise else 0), "maple_attn_linear")
    ws = x.new_empty(n, dtype=torch.uint8) if n else None
    _call("linear", _LINEAR, (
        x.data_ptr(), weight.data_ptr(), _vector(alpha, torch.float32, N, "alpha must be fp32 [N]"),
        _vector(bias, torch.float32, N, "bias must be fp32 [N]"), 0 if resid is None else resid.data_ptr(), out.data_ptr(),
        0 if ws is None else ws.data_ptr(), n, _flags(flags), step if T > 1 else K, T, K, N, ydt, 1 if normalise else 0), dev)
    return out


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, v: torch.Tensor | None = None, pages: torch.Tensor | None = None,
                 slots: torch.Tensor | None = None, flags: torch.Tensor | None = None, page_size: int | None = None):
    """(q', k'): every head normed (RMS, weights fp32 [head_dim] or 1) and rotated by its position.

    q [T][heads][d], k [T][kv_heads][d], bf16 or fp16 (views of one projection are taken as they are); positions int64
    [T]; inv_freq float64 [rotary_dim/2] in radians per position.  With `pages`, `v` and `slots` (int64 [T], < 0: do not
    store, distinct otherwise) the rotated keys and the values are also written to the cache (page_size: see kv_read).
    """
    dt = q.dtype
    if dt not in _HEAD_TYPES:
        raise ValueError("q must be bf16 or fp16")
    T, H, d, qs = _heads(q, dt, "q must be [T][heads][d], a token's heads contiguous")
    Tk, Hkv, dk, ks = _heads(k, dt, "k must be [T][kv_heads][d] of q's type, a token's heads contiguous")
    if Tk != T or dk != d:
        raise ValueError("k must hold the same tokens and head_dim as q")
    vs = n = P = vp = pp = 0
    if pages is not None:
        if v is None or slots is None:
            raise ValueError("pages, v and slots go together")
        vs = _heads(v, dt, "v must be [T][kv_heads][d] of q's type, a token's heads contiguous")[3]
        P, Hc, n = _pages(pages, d, page_size)
        if v.shape != k.shape or Hc != Hkv:
            raise ValueError("v must have the shape of k, and the cache its heads")
        vp, pp = v.data_ptr(), pages.data_ptr()
    elif v is not None or slots is not None:
        raise ValueError("pages, v and slots go together")
    if (q.requires_grad or k.requires_grad or (v is not None and v.requires_grad) or inv_freq.requires_grad or
            (q_weight is not None and q_weight.requires_grad) or (k_weight is not None and k_weight.requires_grad)):
        _refuse_gradient()
    dev = _device(q, k, positions, inv_freq, q_weight, k_weight, v, pages, slots, flags)
    qo = torch.empty_like(q, memory_format=_CONTIGUOUS)
    ko = torch.empty_like(k, memory_format=_CONTIGUOUS)
    rot = inv_freq.shape[0]
    _call("qk_norm_rope", _ROPE, (
        q.data_ptr(), k.data_ptr(), vp, qo.data_ptr(), ko.data_ptr(),
        _vector(q_weight, torch.float32, d, "q_weight must be fp32 [head_dim]"),
        _vector(k_weight, torch.float32, d, "k_weight must be fp32 [head_dim]"),
        _vector(positions, torch.int64, T, "positions must be int64 [T]"),
        _vector(inv_freq, torch.float64, rot, "inv_freq must be float64 [rotary_dim/2]"), pp,
        _vector(slots, torch.int64, T, "slots must be int64 [T]"), _flags(flags), qs, ks, vs, T, P, H, Hkv, d, 2 * rot, n,
        _HEAD_TYPES[dt], 1 if interleaved else 0, eps), dev)
    return qo, ko


def kv_read(pages: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype: torch.dtype = torch.bfloat16,
            flags: torch.Tensor | None = None, page_size: int | None = None):
    """(k, v) [n][kv_heads][head_dim]: the values that the cache holds at `slots` (int64 [n]; < 0 reads as zeros).

    The bytes of a page and head_dim give its tokens, but not the other way round: 64 tokens of 64 channels are as many
    bytes as 32 of 128.  With page_size a cache made for another head_dim or page size is refused; without it one of as
    many bytes is taken for what head_dim says.
    """
    if dtype not in _HEAD_TYPES:
        raise ValueError("dtype must be bf16 or fp16")
    P, Hkv, page_size = _pages(pages, head_dim, page_size)
    dev = _device(pages, slots, flags)
    n = slots.numel()
    k = pages.new_empty((n, Hkv, head_dim), dtype=dtype)
    v = torch.empty_like(k)
    _call("kv_read", _READ, (pages.data_ptr(), _vector(slots, torch.int64, n, "slots must be int64 [n]"), k.data_ptr(),
                              v.data_ptr(), _flags(flags), n, P, Hkv, head_dim, page_size, _HEAD_TYPES[dtype]), dev)
    return k, v


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                     max_q: int, scale: float | None = None, window: int = 0, return_lse: bool = False,
                     out: torch.Tensor | None = None, flags: torch.Tensor | None = None):
    """Causal attention over packed sequences: out [Tq][heads][d] (and lse fp32 [Tq][heads]).

    q [Tq][heads][d], k and v [Tk][kv_heads][d], bf16 or fp16; cu_q, cu_k int32 [B+1], the rows where sequences begin;
    max_q at least the longest sequence's query rows.  A sequence's queries are its last positions.  scale defaults to
    d^-1/2; window > 0 lets a query see that many positions, its own included.  Rows outside every sequence are not
    written (`out` keeps them); `out` must not overlap q, k or v.
    """
    dt = q.dtype
    if dt not in _HEAD_TYPES:
        raise ValueError("q must be bf16 or fp16")
    Tq, H, d, qs = _heads(q, dt, "q must be [Tq][heads][d], a token's heads contiguous")
    Tk, Hkv, dk, ks = _heads(k, dt, "k must be [Tk][kv_heads][d] of q's type, a token's heads contiguous")
    vs = _heads(v, dt, "v must be [Tk][kv_heads][d] of q's type, a token's heads contiguous")[3]
    if k.shape != v.shape or dk != d:
        raise ValueError("k and v must have one shape and q's head_dim")
    if q.requires_grad or k.requires_grad or v.requires_grad or (out is not None and out.requires_grad):
        _refuse_gradient()
    dev = _device(q, k, v, cu_q, cu_k, out, flags)
    B = cu_q.numel() - 1
    if B < 0:
        raise ValueError("cu_q must be int32 [B+1]")
    if out is None:
        out = torch.empty_like(q, memory_format=_CONTIGUOUS)
    elif out.dtype is not dt or out.shape != (Tq, H, d) or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's type and shape")
    elif _overlap(out, q) or _overlap(out, k) or _overlap(out, v):
        raise ValueError("out must not be q, k or v or overlap them")
    lse = q.new_empty((Tq, H), dtype=torch.float32) if return_lse else None
    _call("prompt", _PROMPT, (
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
        _vector(cu_q, torch.int32, B + 1, "cu_q must be int32 [B+1]"), _vector(cu_k, torch.int32, B + 1, "cu_k must be int32 [B+1]"),
        _flags(flags), qs, ks, vs, Tq, Tk, B, max_q, H, Hkv, d, window, _HEAD_TYPES[dt], d ** -0.5 if scale is None else scale),
        dev)
    return (out, lse) if return_lse else out


def cached_attention(q: torch.Tensor, pages: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                     scale: float | None = None, window: int = 0, flags: torch.Tensor | None = None,
                     page_size: int | None = None) -> torch.Tensor:
    """Attention of one new token per sequence over its cached tokens: out [B][heads][d].

    q [B][heads][d] bf16 or fp16; block_table int32 [B][max_pages]; lens int32 [B], the cached tokens of each sequence
    (the new one among them).  scale and window as in prompt_attention, page_size as in kv_read; an empty sequence gives a
    row of zeros.
    """
    dt = q.dtype
    if dt not in _HEAD_TYPES:
        raise ValueError("q must be bf16 or fp16")
    B, H, d, qs = _heads(q, dt, "q must be [B][heads][d], a token's heads contiguous")
    P, Hkv, n = _pages(pages, d, page_size)
    if q.requires_grad:
        _refuse_gradient()
    dev = _device(q, pages, block_table, lens, flags)
    if block_table.dtype is not torch.int32 or block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B][max_pages]")
    rows, mp = block_table.shape
    step, one = block_table.stride()
    if rows != B or (one != 1 and mp > 1):
        raise ValueError("block_table must be int32 [B][max_pages]")
    out = torch.empty_like(q, memory_format=_CONTIGUOUS)
    w = _size((_fn or _lib()).maple_attn_cached_workspace(B, mp, H, Hkv, d, n, window), "maple_attn_cached")
    ws = q.new_empty(w, dtype=torch.uint8) if w else None
    _call("cached", _CACHED, (
        q.data_ptr(), out.data_ptr(), pages.data_ptr(), block_table.data_ptr(), _vector(lens, torch.int32, B, "lens must be int32 [B]"),
        0 if ws is None else ws.data_ptr(), w, _flags(flags), qs, step if B > 1 else mp, P, B, mp, H, Hkv, d, n, window,
        _HEAD_TYPES[dt], d ** -0.5 if scale is None else scale), dev)
    return out
