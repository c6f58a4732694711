"""Python API of the paged key/value cache around the verify step, over torch tensors.

The calls mirror include/spec_kv.h, which holds their definitions and the cache's layout; shapes,
dtypes and strides are read from the tensors, which lie on the current device, outputs are allocated
unless ``out`` supplies them.
A round is ``block_tables`` -> (projections) -> ``qk_norm_rope`` -> ``kv4_append`` ->
``kv4_attention`` -> (the rest of the layer, the head) -> ``verify`` / ``verify_hidden``, whose
``accept_len`` goes into the next round's ``block_tables``. ``kv8_append`` and ``kv8_attention`` take
the places of the 4-bit pair over a cache in 8 bits; ``prompt_attention`` is a prompt's own attention,
from its keys and values as they are, or as the cache holds them.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._lib import SV_DTYPE_BF16, SV_DTYPE_F32
from .api import _stream_handle

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_several: Optional[bool] = None  # the process sees more than one device


def _stream(stream, at: Optional[int]) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(at or 0)
    return _stream_handle(stream)


def _device(t: torch.Tensor, name: str) -> Optional[int]:
    """Index of the tensor's device, which must be the current one: the library launches there, whatever
    device its arguments are on. Every tensor of a call is then held to it. None where the process sees
    one device, which any CUDA tensor is on."""
    global _several
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if _several is None:
        _several = torch.cuda.device_count() > 1
    if not _several:
        return None
    at = t.get_device()
    if at != _current_device():
        raise ValueError(f"{name} is on CUDA device {at}, the current one is {_current_device()}")
    return at


def _dev(t: torch.Tensor, dtype, shape, name: str, at: Optional[int]) -> int:
    """Address of a contiguous CUDA tensor of this dtype and shape, on device ``at``."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and (at is None or t.get_device() == at) \
            and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be a contiguous CUDA tensor, on the device of the others")


def _vec(t: torch.Tensor, dtype, n: int, name: str, at: Optional[int]) -> int:
    """Address of a contiguous CUDA tensor of this dtype that holds n values. These calls take some
    microseconds in all, so what is checked of each of a dozen tensors counts."""
    if t.dtype is dtype and t.numel() == n and t.is_cuda and (at is None or t.get_device() == at) \
            and t.is_contiguous():
        return t.data_ptr()
    return _dev(t, dtype, t.shape if t.numel() == n else (n,), name, at)


def _rows(t: torch.Tensor, name: str, at: Optional[int]):
    """(address, token stride) of [T, H, D] whose heads lie side by side."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, D], got {tuple(t.shape)}")
    T, H, D = t.shape
    s = t.stride()
    if not t.is_cuda or (at is not None and t.get_device() != at) \
            or (s[2] != 1 and D > 1) or (s[1] != D and H > 1):
        raise ValueError(f"{name} must be a CUDA tensor whose heads are contiguous in a token, on the "
                         "device of the others")
    return t.data_ptr(), s[0] if T > 1 else H * D


def _float_code(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return SV_DTYPE_BF16
    if t.dtype == torch.float32:
        return SV_DTYPE_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def block_tables(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                 held: torch.Tensor, ring: torch.Tensor, counters: torch.Tensor, *,
                 page_size: int, max_tokens: int, accept_len: Optional[torch.Tensor] = None,
                 out: Optional[dict] = None, stream=None) -> dict:
    """Pages, slots and positions of the next round from the sequences' lengths
    (``spec_block_tables``). ``block_table`` [B, max_blocks] and ``ring`` are updated in place;
    ``counters`` is int64 [2], the rest int32. Returns {"ctx_lens", "held", "counters",
    "cu_new", "kv_lens", "status", "slots", "positions", "seq_ids"}, buffers other than the
    inputs: two sets in turn serve a loop."""
    i32, i64 = torch.int32, torch.int64
    at, B = _device(ctx_lens, "ctx_lens"), ctx_lens.shape[0]
    if block_table.dim() != 2 or ring.dim() != 1:
        raise ValueError("block_table must be [B, max_blocks] and ring [pages]")
    most, ring_size = block_table.shape[1], ring.shape[0]
    if out is None:
        dev = ctx_lens.device

        def new(n, t=i32):
            return torch.empty(n, dtype=t, device=dev)
        out = {"ctx_lens": new(B), "held": new(B), "counters": new(2, i64), "cu_new": new(B + 1),
               "kv_lens": new(B), "status": new(B), "slots": new(max_tokens, i64),
               "positions": new(max_tokens), "seq_ids": new(max_tokens)}
    st = _lib.load().spec_block_tables(
        B, page_size, most, max_tokens, _vec(ctx_lens, i32, B, "ctx_lens", at),
        0 if accept_len is None else _vec(accept_len, i32, B, "accept_len", at),
        _vec(new_lens, i32, B, "new_lens", at), _vec(block_table, i32, B * most, "block_table", at),
        _vec(held, i32, B, "held", at), _vec(ring, i32, ring_size, "ring", at),
        ring_size, _vec(counters, i64, 2, "counters", at),
        _vec(out["ctx_lens"], i32, B, "out ctx_lens", at),
        _vec(out["held"], i32, B, "out held", at), _vec(out["counters"], i64, 2, "out counters", at),
        _vec(out["kv_lens"], i32, B, "out kv_lens", at), _vec(out["status"], i32, B, "out status", at),
        _vec(out["cu_new"], i32, B + 1, "out cu_new", at),
        _vec(out["slots"], i64, max_tokens, "out slots", at),
        _vec(out["positions"], i32, max_tokens, "out positions", at),
        _vec(out["seq_ids"], i32, max_tokens, "out seq_ids", at), _stream(stream, at))
    _lib._check(st, "spec_block_tables")
    return out


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
                 inv_freq: torch.Tensor, *, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, out: Optional[dict] = None, stream=None) -> dict:
    """Norm of every query and key head and the rotation by position, in one pass
    (``spec_qk_norm_rope``). ``q`` [T, Hq, D] and ``k`` [T, Hkv, D] (or None) bf16 or f32, heads
    contiguous in a token; ``positions`` [T] int32; ``inv_freq`` [rot / 2] float64. Returns
    {"q", "k"}; ``out={"q": q, "k": k}`` works in place."""
    T, hq, D = q.shape
    code, at = _float_code(q, "q"), _device(q, "q")
    hk = 0 if k is None else k.shape[1]
    if k is not None and (k.dtype != q.dtype or k.shape[0] != T or k.shape[2] != D):
        raise ValueError("k must be [T, Hkv, D] of q's dtype")
    if out is None:
        out = {"q": torch.empty((T, hq, D), dtype=q.dtype, device=q.device)}
        if k is not None:
            out["k"] = torch.empty((T, hk, D), dtype=q.dtype, device=q.device)
    for n, h in (("q", hq), ("k", hk)):
        if h and (out[n].dtype != q.dtype or out[n].shape != (T, h, D)):
            raise ValueError(f"out {n} must be {(T, h, D)} of q's dtype")
    half = inv_freq.numel()
    qp, qs = _rows(q, "q", at)
    oq, oqs = _rows(out["q"], "out q", at)
    kp, ks = _rows(k, "k", at) if k is not None else (0, 0)
    ok, oks = _rows(out["k"], "out k", at) if k is not None else (0, 0)
    st = _lib.load().spec_qk_norm_rope(
        T, hq, hk, D, 2 * half, bool(interleaved), code, qp, qs, kp, ks,
        0 if q_weight is None else _vec(q_weight, q.dtype, D, "q_weight", at),
        0 if k_weight is None else _vec(k_weight, q.dtype, D, "k_weight", at),
        _vec(positions, torch.int32, T, "positions", at),
        _vec(inv_freq, torch.float64, half, "inv_freq", at), eps, oq, oqs, ok, oks,
        _stream(stream, at))
    _lib._check(st, "spec_qk_norm_rope")
    return out


def kv4_page_bytes(page_size: int, D: int) -> int:
    """Bytes of one page of one head; 0 where the sizes are not supported."""
    return int(_lib.load().spec_kv4_page_bytes(int(page_size), int(D)))


def kv4_cache(num_pages: int, heads: int, D: int, page_size: int, device="cuda") -> torch.Tensor:
    """An empty cache: uint8 [num_pages, heads, kv4_page_bytes(page_size, D)]."""
    nbytes = kv4_page_bytes(page_size, D)
    if not nbytes:
        raise ValueError("page_size must be 16, 32, 64 or 128 and D 64 or 128")
    return torch.zeros(num_pages, heads, nbytes, dtype=torch.uint8, device=device)


def _cache(cache: torch.Tensor, heads: int, D: int, page_size: int, at: Optional[int],
           token_bytes: Optional[int] = None) -> int:
    if cache.dim() != 3 or cache.shape[1] != heads or \
            cache.shape[2] != page_size * (token_bytes or D + D // 8):
        raise ValueError(f"cache {tuple(cache.shape)} is not [pages, {heads}, page bytes] for "
                         f"page_size {page_size}, D {D}")
    return _dev(cache, torch.uint8, cache.shape, "cache", at)


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, *,
               page_size: int, k_scale: float = 1.0, v_scale: float = 1.0,
               out: Optional[dict] = None, values: bool = False, stream=None) -> dict:
    """Write the keys and values of T tokens into the cache at ``slots`` (``spec_kv4_append``).
    ``k``, ``v`` [T, Hkv, D] bf16 or f32; ``slots`` [T] int64, -1 for a token that is not
    written. Returns {}, or with ``values`` (or ``out``) {"k", "v"}: bf16, what the cache now
    stands for."""
    T, H, D = k.shape
    at = _device(k, "k")
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must share shape and dtype")
    if out is None:
        out = {n: torch.empty((T, H, D), dtype=torch.bfloat16, device=k.device)
               for n in ("k", "v")} if values else {}
    kp, ks = _rows(k, "k", at)
    vp, vs = _rows(v, "v", at)
    st = _lib.load().spec_kv4_append(
        T, H, D, page_size, cache.shape[0], _float_code(k, "k"), kp, ks, vp, vs,
        _vec(slots, torch.int64, T, "slots", at), k_scale, v_scale,
        _cache(cache, H, D, page_size, at),
        _dev(out["k"], torch.bfloat16, (T, H, D), "out k", at) if out else 0,
        _dev(out["v"], torch.bfloat16, (T, H, D), "out v", at) if out else 0, _stream(stream, at))
    _lib._check(st, "spec_kv4_append")
    return out


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                  kv_lens: torch.Tensor, cu_new: torch.Tensor, *, page_size: int,
                  scale: Optional[float] = None, k_scale: float = 1.0, v_scale: float = 1.0,
                  max_new: int = 1, out: Optional[dict] = None, stream=None) -> dict:
    """Causal attention of the new tokens over the cache (``spec_kv4_attention``). ``q``
    [T, Hq, D] bf16; ``block_table`` [B, max_blocks], ``kv_lens`` [B], ``cu_new`` [B + 1] int32;
    ``max_new`` is the largest number of new tokens of a sequence, as far as known (speed only).
    ``scale`` defaults to 1 / sqrt(D). Returns {"out" [T, Hq, D] bf16, "lse" [T, Hq] f32}; rows
    of no sequence are left as they are."""
    T, hq, D = q.shape
    if q.dtype != torch.bfloat16:
        raise TypeError(f"q must be bfloat16, got {q.dtype}")
    at, B = _device(q, "q"), kv_lens.shape[0]
    if block_table.dim() != 2 or cache.dim() != 3:
        raise ValueError("block_table must be [B, max_blocks] and cache [pages, Hkv, page bytes]")
    H = cache.shape[1]
    if out is None:
        out = {"out": torch.empty((T, hq, D), dtype=torch.bfloat16, device=q.device),
               "lse": torch.empty((T, hq), dtype=torch.float32, device=q.device)}
    qp, qs = _rows(q, "q", at)
    lse = out.get("lse")
    st = _lib.load().spec_kv4_attention(
        B, T, hq, H, D, page_size, cache.shape[0], block_table.shape[1], qp, qs,
        _cache(cache, H, D, page_size, at),
        _dev(block_table, torch.int32, (B, block_table.shape[1]), "block_table", at),
        _vec(kv_lens, torch.int32, B, "kv_lens", at), _vec(cu_new, torch.int32, B + 1, "cu_new", at),
        D ** -0.5 if scale is None else scale, k_scale, v_scale, max_new,
        _dev(out["out"], torch.bfloat16, (T, hq, D), "out", at),
        0 if lse is None else _dev(lse, torch.float32, (T, hq), "lse", at), _stream(stream, at))
    _lib._check(st, "spec_kv4_attention")
    return out


def kv8_page_bytes(page_size: int, D: int) -> int:
    """Bytes of one page of one head of the 8-bit cache; 0 where the sizes are not supported."""
    return int(_lib.load().spec_kv8_page_bytes(int(page_size), int(D)))


def kv8_cache(num_pages: int, heads: int, D: int, page_size: int, device="cuda") -> torch.Tensor:
    """An empty 8-bit cache: uint8 [num_pages, heads, kv8_page_bytes(page_size, D)]."""
    nbytes = kv8_page_bytes(page_size, D)
    if not nbytes:
        raise ValueError("page_size must be 16, 32, 64 or 128 and D 64 or 128")
    return torch.zeros(num_pages, heads, nbytes, dtype=torch.uint8, device=device)


def kv8_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, *,
               page_size: int, out: Optional[dict] = None, values: bool = False,
               stream=None) -> dict:
    """Write the keys and values of T tokens into the 8-bit cache at ``slots`` (``spec_kv8_append``).
    ``k``, ``v`` [T, Hkv, D] bf16 or f32; ``slots`` [T] int64, -1 for a token that is not written;
    tokens of one block of 16 lie together, as ``block_tables`` gives them. Returns {}, or with
    ``values`` (or ``out``) {"k", "v"}: bf16, what the cache now stands for."""
    T, H, D = k.shape
    at = _device(k, "k")
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must share shape and dtype")
    if out is None:
        out = {n: torch.empty((T, H, D), dtype=torch.bfloat16, device=k.device)
               for n in ("k", "v")} if values else {}
    kp, ks = _rows(k, "k", at)
    vp, vs = _rows(v, "v", at)
    st = _lib.load().spec_kv8_append(
        T, H, D, page_size, cache.shape[0], _float_code(k, "k"), kp, ks, vp, vs,
        _vec(slots, torch.int64, T, "slots", at), _cache(cache, H, D, page_size, at, 2 * D + 1),
        _dev(out["k"], torch.bfloat16, (T, H, D), "out k", at) if out else 0,
        _dev(out["v"], torch.bfloat16, (T, H, D), "out v", at) if out else 0, _stream(stream, at))
    _lib._check(st, "spec_kv8_append")
    return out


def kv8_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                  kv_lens: torch.Tensor, cu_new: torch.Tensor, *, page_size: int,
                  scale: Optional[float] = None, max_new: int = 1, out: Optional[dict] = None,
                  stream=None) -> dict:
    """Causal attention of the new tokens over the 8-bit cache (``spec_kv8_attention``); arguments
    and results as in ``kv4_attention``, without tensor scales."""
    T, hq, D = q.shape
    if q.dtype != torch.bfloat16:
        raise TypeError(f"q must be bfloat16, got {q.dtype}")
    at, B = _device(q, "q"), kv_lens.shape[0]
    if block_table.dim() != 2 or cache.dim() != 3:
        raise ValueError("block_table must be [B, max_blocks] and cache [pages, Hkv, page bytes]")
    H = cache.shape[1]
    if out is None:
        out = {"out": torch.empty((T, hq, D), dtype=torch.bfloat16, device=q.device),
               "lse": torch.empty((T, hq), dtype=torch.float32, device=q.device)}
    qp, qs = _rows(q, "q", at)
    lse = out.get("lse")
    st = _lib.load().spec_kv8_attention(
        B, T, hq, H, D, page_size, cache.shape[0], block_table.shape[1], qp, qs,
        _cache(cache, H, D, page_size, at, 2 * D + 1),
        _dev(block_table, torch.int32, (B, block_table.shape[1]), "block_table", at),
        _vec(kv_lens, torch.int32, B, "kv_lens", at), _vec(cu_new, torch.int32, B + 1, "cu_new", at),
        D ** -0.5 if scale is None else scale, max_new,
        _dev(out["out"], torch.bfloat16, (T, hq, D), "out", at),
        0 if lse is None else _dev(lse, torch.float32, (T, hq), "lse", at), _stream(stream, at))
    _lib._check(st, "spec_kv8_attention")
    return out


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, *,
                     scale: Optional[float] = None, out: Optional[dict] = None,
                     stream=None) -> dict:
    """Causal attention over whole prompts, packed (``spec_prompt_attention``). ``q`` [T, Hq, D],
    ``k``, ``v`` [T, Hkv, D] bf16, heads contiguous in a token; ``cu`` [B + 1] int32, where each
    sequence's rows begin. ``scale`` defaults to 1 / sqrt(D). Returns {"out" [T, Hq, D] bf16,
    "lse" [T, Hq] f32}; rows of no sequence are left as they are."""
    T, hq, D = q.shape
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError(f"q, k and v must be bfloat16, got {q.dtype}, {k.dtype}, {v.dtype}")
    at = _device(q, "q")
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or v.shape != k.shape:
        raise ValueError(f"k and v must be [{T}, Hkv, {D}], got {tuple(k.shape)}, {tuple(v.shape)}")
    if out is None:
        out = {"out": torch.empty((T, hq, D), dtype=torch.bfloat16, device=q.device),
               "lse": torch.empty((T, hq), dtype=torch.float32, device=q.device)}
    qp, qs = _rows(q, "q", at)
    kp, ks = _rows(k, "k", at)
    vp, vs = _rows(v, "v", at)
    lse = out.get("lse")
    st = _lib.load().spec_prompt_attention(
        cu.numel() - 1, T, hq, k.shape[1], D, qp, qs, kp, ks, vp, vs,
        _vec(cu, torch.int32, cu.numel(), "cu", at), D ** -0.5 if scale is None else scale,
        _dev(out["out"], torch.bfloat16, (T, hq, D), "out", at),
        0 if lse is None else _dev(lse, torch.float32, (T, hq), "lse", at), _stream(stream, at))
    _lib._check(st, "spec_prompt_attention")
    return out
