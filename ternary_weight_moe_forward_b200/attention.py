"""The attention half of a decoder layer on torch tensors (C ABI: include/maple_attn.h).

    int8_linear        rows quantised to int8 times int8 weights (projections, output head)
    qk_norm_rope       norm and rotation of query and key heads, appended to the 4-bit cache in the same pass
    kv_read            the values that the cache holds at given slots
    prompt_attention   causal attention over packed prompts
    cached_attention   attention of one new token per sequence over the cache

Each function checks its tensors, allocates outputs and scratch with torch on
the tensors' device and launches on that device's current stream (or `stream`);
none synchronises, and all may be captured into a CUDA graph.  A tensor of the
wrong type, shape, stride or device raises ValueError, an error of the library
MapleError.  What only the kernels can see (a page number outside the cache) is
reported in `flags`, an int32 tensor of one element that the caller zeroes and
reads (MAPLE_FLAG_* bits).  No gradients: these are serving operators.

Cache: uint8 [num_pages][kv_heads][page bytes], made by kv_pages(); a token's
slot is page * page_size + row.
"""
from __future__ import annotations

import ctypes as C
import struct

import torch

from . import MAPLE_OK, MapleError, lib

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


def _lib():
    global _fn
    if _fn is None:
        L = lib()
        P, I32, I64 = C.c_void_p, C.c_int32, C.c_int64
        for name in ("linear", "qk_norm_rope", "kv_read", "prompt", "cached"):
            f = getattr(L, "maple_attn_" + name)
            f.argtypes, f.restype = [C.c_char_p, P], C.c_int
        L.maple_attn_page_bytes.argtypes, L.maple_attn_page_bytes.restype = [I32, I32], I64
        L.maple_attn_linear_workspace.argtypes, L.maple_attn_linear_workspace.restype = [I64] * 3, I64
        L.maple_attn_cached_workspace.argtypes, L.maple_attn_cached_workspace.restype = [I32] * 7, I64
        _fn = L
    return _fn


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _p(t) -> int:
    return 0 if t is None else t.data_ptr()


def _call(name: str, args: bytes, device, stream) -> None:
    """Launch on `stream` or the device's current one, with that device current."""
    fn = getattr(_lib(), "maple_attn_" + name)
    here = torch.cuda.current_device()
    if device.index != here:
        with torch.cuda.device(device):
            rc = fn(args, torch.cuda.current_stream().cuda_stream if stream is None else stream)
    else:
        rc = fn(args, torch.cuda.current_stream().cuda_stream if stream is None else stream)
    if rc != MAPLE_OK:
        raise MapleError(rc, "maple_attn_" + name)


def _size(n: int, what: str) -> int:
    if n < 0:
        raise MapleError(n, what)
    return n


def _same_device(device, *tensors) -> None:
    _need(device.type == "cuda", "the tensors must be on a CUDA device")
    for t in tensors:
        _need(t is None or t.device == device, f"all tensors must be on {device}")


def _check_flags(flags) -> None:
    _need(flags is None or (flags.dtype is torch.int32 and flags.numel() == 1), "flags must be one int32")


def _heads(t, name: str, dtype=None):
    """A [tokens][heads][head_dim] tensor whose heads are contiguous within a token; returns its token stride."""
    _need(t.dim() == 3, f"{name} must be [tokens][heads][head_dim]")
    n, h, d = t.shape
    s = t.stride()
    _need(s[2] == 1 and (h == 1 or s[1] == d), f"{name}: a token's heads must be contiguous")
    _need(dtype is None or t.dtype is dtype, f"{name} must be {dtype}")
    return s[0] if n > 1 else h * d


def kv_pages(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> torch.Tensor:
    """A zeroed cache of `num_pages` pages of `page_size` tokens (16, 32 or 64) with head_dim 64 or 128."""
    b = _size(_lib().maple_attn_page_bytes(head_dim, page_size), "maple_attn_page_bytes")
    return torch.zeros(num_pages, kv_heads, b, dtype=torch.uint8, device=device)


def _page_size(pages, kv_heads: int, head_dim: int) -> int:
    _need(pages.dtype is torch.uint8 and pages.dim() == 3 and pages.is_contiguous(),
          "pages must be a contiguous uint8 [num_pages][kv_heads][page bytes]")
    _need(pages.shape[1] == kv_heads, f"the cache holds {pages.shape[1]} key/value heads, not {kv_heads}")
    n, rest = divmod(pages.shape[2] * 4, 5 * head_dim)
    _need(rest == 0 and n in (16, 32, 64), f"pages of {pages.shape[2]} bytes do not fit head_dim {head_dim}")
    return n


def int8_linear(x: torch.Tensor, weight: torch.Tensor, alpha: torch.Tensor, bias: torch.Tensor | None = None,
                resid: torch.Tensor | None = None, normalise: bool = False, out_dtype: torch.dtype = torch.float32,
                out: torch.Tensor | None = None, flags: torch.Tensor | None = None, stream: int | None = None) -> torch.Tensor:
    """y = (q_x weight^T) * (s_x alpha) (+ bias) (+ resid), q_x and s_x the int8 absmax codes and scales of x's rows.

    x bf16 [T][K] (rows may be strided), or the fp32 residual stream with `normalise` (its RMS-normed rows, rounded to
    bf16, are quantised).  weight int8 [N][K], alpha fp32 [N], bias fp32 [N], resid fp32 [T][N] (may be `out`).
    """
    _need(x.dim() == 2 and weight.dim() == 2 and x.shape[1] == weight.shape[1], "x must be [T][K] and weight [N][K]")
    T, K = x.shape
    N = weight.shape[0]
    dev = x.device
    _same_device(dev, weight, alpha, bias, resid, out, flags)
    _need(x.dtype is (torch.float32 if normalise else torch.bfloat16), "x must be bf16, or fp32 with normalise")
    _need(x.stride(1) == 1 or K == 1, "the rows of x must be contiguous")
    _need(weight.dtype is torch.int8 and weight.is_contiguous(), "weight must be contiguous int8")
    for v, name in ((alpha, "alpha"), (bias, "bias")):
        _need(v is None or (v.dtype is torch.float32 and v.shape == (N,) and v.is_contiguous()), f"{name} must be fp32 [N]")
    _need(resid is None or (resid.dtype is torch.float32 and resid.shape == (T, N) and resid.is_contiguous()),
          "resid must be contiguous fp32 [T][N]")
    if out is None:
        _need(out_dtype in _OUT_TYPES, "out_dtype must be bf16 or fp32")
        out = torch.empty((T, N), dtype=out_dtype, device=dev)
    else:
        _need(out.dtype in _OUT_TYPES and out.shape == (T, N) and out.is_contiguous(), "out must be contiguous bf16 or fp32 [T][N]")
    _check_flags(flags)
    n = _size(_lib().maple_attn_linear_workspace(T, K, N), "maple_attn_linear")
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _call("linear", _LINEAR.pack(_p(x), _p(weight), _p(alpha), _p(bias), _p(resid), _p(out), _p(ws), n, _p(flags),
                                 x.stride(0) if T > 1 else K, T, K, N, _OUT_TYPES[out.dtype], int(normalise)), dev, stream)
    return out


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, v: torch.Tensor | None = None, pages: torch.Tensor | None = None,
                 slots: torch.Tensor | None = None, flags: torch.Tensor | None = None, stream: int | None = None):
    """(q', k'): every head normed (RMS, weights fp32 [head_dim] or 1) and rotated by its position.

    q [T][heads][d], k [T][kv_heads][d], bf16 or fp16 (views of one projection are taken as they are); positions int64
    [T]; inv_freq float64 [rotary_dim/2] in radians per position.  With `pages`, `v` and `slots` (int64 [T], < 0: do not
    store, distinct otherwise) the rotated keys and the values are also written to the cache.
    """
    dt = q.dtype
    _need(dt in _HEAD_TYPES, "q must be bf16 or fp16")
    qs, ks = _heads(q, "q"), _heads(k, "k", dt)
    T, H, d = q.shape
    Hkv = k.shape[1]
    dev = q.device
    _same_device(dev, k, positions, inv_freq, q_weight, k_weight, v, pages, slots, flags)
    _need(k.shape == (T, Hkv, d), "k must hold the same tokens and head_dim as q")
    _need(positions.dtype is torch.int64 and positions.shape == (T,) and positions.is_contiguous(), "positions must be int64 [T]")
    _need(inv_freq.dtype is torch.float64 and inv_freq.dim() == 1 and inv_freq.is_contiguous(), "inv_freq must be float64 [rotary_dim/2]")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        _need(w is None or (w.dtype is torch.float32 and w.shape == (d,) and w.is_contiguous()), f"{name} must be fp32 [head_dim]")
    _need((pages is None) == (v is None) == (slots is None), "pages, v and slots go together")
    vs = n = P = 0
    if pages is not None:
        vs = _heads(v, "v", dt)
        _need(v.shape == k.shape, "v must have the shape of k")
        _need(slots.dtype is torch.int64 and slots.shape == (T,) and slots.is_contiguous(), "slots must be int64 [T]")
        n, P = _page_size(pages, Hkv, d), pages.shape[0]
    _check_flags(flags)
    qo = torch.empty((T, H, d), dtype=dt, device=dev)
    ko = torch.empty((T, Hkv, d), dtype=dt, device=dev)
    _call("qk_norm_rope", _ROPE.pack(_p(q), _p(k), _p(v), _p(qo), _p(ko), _p(q_weight), _p(k_weight), _p(positions),
                                     _p(inv_freq), _p(pages), _p(slots), _p(flags), qs, ks, vs, T, P, H, Hkv, d,
                                     2 * inv_freq.shape[0], n, _HEAD_TYPES[dt], int(interleaved), eps), dev, stream)
    return qo, ko


def kv_read(pages: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype: torch.dtype = torch.bfloat16,
            flags: torch.Tensor | None = None, stream: int | None = None):
    """(k, v) [n][kv_heads][head_dim]: the values that the cache holds at `slots` (int64 [n]; < 0 reads as zeros)."""
    _need(dtype in _HEAD_TYPES, "dtype must be bf16 or fp16")
    _need(pages.dim() == 3, "pages must be [num_pages][kv_heads][page bytes]")
    P, Hkv = pages.shape[:2]
    page_size = _page_size(pages, Hkv, head_dim)
    dev = pages.device
    _same_device(dev, slots, flags)
    _need(slots.dtype is torch.int64 and slots.dim() == 1 and slots.is_contiguous(), "slots must be int64 [n]")
    _check_flags(flags)
    n = slots.shape[0]
    k = torch.empty((n, Hkv, head_dim), dtype=dtype, device=dev)
    v = torch.empty((n, Hkv, head_dim), dtype=dtype, device=dev)
    _call("kv_read", _READ.pack(_p(pages), _p(slots), _p(k), _p(v), _p(flags), n, P, Hkv, head_dim, page_size,
                                _HEAD_TYPES[dtype]), dev, stream)
    return k, v


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                     max_q: int, scale: float | None = None, window: int = 0, return_lse: bool = False,
                     out: torch.Tensor | None = None, flags: torch.Tensor | None = None, stream: int | None = None):
    """Causal attention over packed sequences: out [Tq][heads][d] (and lse fp32 [Tq][heads]).

    q [Tq][heads][d], k and v [Tk][kv_heads][d], bf16 or fp16; cu_q, cu_k int32 [B+1], the rows where sequences begin;
    max_q at least the longest sequence's query rows.  A sequence's queries are its last positions.  scale defaults to
    d^-1/2; window > 0 lets a query see that many positions, its own included.  Rows outside every sequence are not
    written (`out` keeps them).
    """
    dt = q.dtype
    _need(dt in _HEAD_TYPES, "q must be bf16 or fp16")
    qs, ks, vs = _heads(q, "q"), _heads(k, "k", dt), _heads(v, "v", dt)
    Tq, H, d = q.shape
    Tk, Hkv = k.shape[:2]
    dev = q.device
    _same_device(dev, k, v, cu_q, cu_k, out, flags)
    _need(k.shape == v.shape and k.shape[2] == d, "k and v must have one shape and q's head_dim")
    B = cu_q.shape[0] - 1
    for c, name in ((cu_q, "cu_q"), (cu_k, "cu_k")):
        _need(c.dtype is torch.int32 and c.dim() == 1 and c.shape[0] == B + 1 >= 1 and c.is_contiguous(), f"{name} must be int32 [B+1]")
    _check_flags(flags)
    if out is None:
        out = torch.empty((Tq, H, d), dtype=dt, device=dev)
    else:
        _need(out.dtype is dt and out.shape == (Tq, H, d) and out.is_contiguous(), "out must be contiguous, of q's type and shape")
    lse = torch.empty((Tq, H), dtype=torch.float32, device=dev) if return_lse else None
    _call("prompt", _PROMPT.pack(_p(q), _p(k), _p(v), _p(out), _p(lse), _p(cu_q), _p(cu_k), _p(flags), qs, ks, vs, Tq, Tk,
                                 B, max_q, H, Hkv, d, window, _HEAD_TYPES[dt], d ** -0.5 if scale is None else scale), dev, stream)
    return (out, lse) if return_lse else out


def cached_attention(q: torch.Tensor, pages: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                     scale: float | None = None, window: int = 0, flags: torch.Tensor | None = None,
                     stream: int | None = None) -> torch.Tensor:
    """Attention of one new token per sequence over its cached tokens: out [B][heads][d].

    q [B][heads][d] bf16 or fp16; block_table int32 [B][max_pages]; lens int32 [B], the cached tokens of each sequence
    (the new one among them).  scale and window as in prompt_attention; an empty sequence gives a row of zeros.
    """
    dt = q.dtype
    _need(dt in _HEAD_TYPES, "q must be bf16 or fp16")
    qs = _heads(q, "q")
    B, H, d = q.shape
    dev = q.device
    _same_device(dev, pages, block_table, lens, flags)
    _need(pages.dim() == 3, "pages must be [num_pages][kv_heads][page bytes]")
    P, Hkv = pages.shape[:2]
    n = _page_size(pages, Hkv, d)
    _need(block_table.dtype is torch.int32 and block_table.dim() == 2 and block_table.shape[0] == B and
          (block_table.stride(1) == 1 or block_table.shape[1] <= 1), "block_table must be int32 [B][max_pages]")
    _need(lens.dtype is torch.int32 and lens.shape == (B,) and lens.is_contiguous(), "lens must be int32 [B]")
    _check_flags(flags)
    mp = block_table.shape[1]
    out = torch.empty((B, H, d), dtype=dt, device=dev)
    w = _size(_lib().maple_attn_cached_workspace(B, mp, H, Hkv, d, n, window), "maple_attn_cached")
    ws = torch.empty(w, dtype=torch.uint8, device=dev) if w else None
    _call("cached", _CACHED.pack(_p(q), _p(out), _p(pages), _p(block_table), _p(lens), _p(ws), w, _p(flags), qs,
                                 block_table.stride(0) if B > 1 else mp, P, B, mp, H, Hkv, d, n, window, _HEAD_TYPES[dt],
                                 d ** -0.5 if scale is None else scale), dev, stream)
    return out
