"""Python binding of grinqh_qk_rope: norms of queries and keys, rotation by
position, and the cache's write in one pass (include/grinqh.h)."""

from __future__ import annotations

import ctypes

try:
    import torch
except ImportError:
    torch = None

from .attention import KVCache, _empty, _float_code, _plain, _rows, _run, _tensor
from .grinqh import GRINQH_BF16, RopeArgs

if torch is not None:
    from .attention import _CODES
    _I32, _I64, _F64 = torch.int32, torch.int64, torch.float64


def _check_rope(q, k, positions, freqs, q_weight, k_weight, cache, v, slots, q_out, k_out) -> None:
    """Goes through the conditions one by one to say which fails."""
    device = _tensor(q, "q")
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q and k must be [tokens][heads][head_dim]")
    n, heads, dim = q.shape
    kv_heads = k.shape[1]
    _rows(q, "q", heads, dim, device)
    _rows(k, "k", kv_heads, dim, device)
    _float_code(q.dtype, "q")
    if k.shape[0] != n or k.dtype != q.dtype:
        raise ValueError("q and k must hold the same tokens in one type")
    _plain(positions, "positions", _I32, device, n)
    if positions.numel() != n:
        raise ValueError("positions must name every token's")
    _plain(freqs, "freqs", _F64, device, 0)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _float_code(w.dtype if isinstance(w, torch.Tensor) else None, name)
            _plain(w, name, w.dtype, device, dim)
            if w.numel() != dim:
                raise ValueError(f"{name} must be [{dim}]")
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("q_weight and k_weight must have one dtype")
    for name, t, h in (("q_out", q_out, heads), ("k_out", k_out, kv_heads)):
        if t is None:
            continue
        _rows(t, name, h, dim, device)
        if t.shape[0] != n or t.dtype != q.dtype:
            raise ValueError(f"{name} must hold the same tokens in the same type")
    if q_out is None or (k_out is None and cache is None):
        raise ValueError("q_out and, without a cache, k_out are needed")
    if cache is not None:
        if not isinstance(cache, KVCache) or cache.device != device or cache.n_kv_heads != kv_heads or cache.head_dim != dim:
            raise ValueError("the cache must have the keys' heads, head_dim and device")
        _rows(v, "v", kv_heads, dim, device)
        if v.shape[0] != n or v.dtype != q.dtype:
            raise ValueError("v must hold the same tokens in the same type")
        _plain(slots, "slots", _I64, device, n)
        if slots.numel() != n:
            raise ValueError("slots must name every token's")
    elif v is not None or slots is not None:
        raise ValueError("v and slots go with a cache")


def grinqh_qk_rope(q, k, positions, freqs, q_out, k_out, q_weight=None, k_weight=None, eps: float = 1e-6,
                   neighbours: bool = False, cache: KVCache = None, v=None, slots=None, stream=None) -> None:
    """q, k (and v): bf16 or fp32 [tokens][heads][head_dim], token rows contiguous;
    positions: int32 [tokens]; freqs: float64 [rope_dim / 2]; q_out, k_out: as q and
    k, or q and k themselves (k_out may be None with a cache); weights: bf16 or fp32
    [head_dim] or None; slots: int64 [tokens]."""
    try:
        (n, heads, dim), (n_k, kv_heads, kd) = q.shape, k.shape
        device = q.device
        index = device.index
        (qs, q1, q2), (ks, k1, k2), (os, o1, o2) = q.stride(), k.stride(), q_out.stride()
        width, kv_width = heads * dim, kv_heads * dim
        fits = (n_k == n and kd == dim and q2 == k2 == o2 == 1 and (q1 == o1 == dim or heads == 1) and (k1 == dim or kv_heads == 1)
                and (n < 2 or (qs >= width and ks >= kv_width and os >= width)) and q.dtype is k.dtype is q_out.dtype
                and q.dtype in _CODES and q_out.shape == q.shape and positions.dtype is _I32 and positions.is_contiguous()
                and positions.numel() == n and freqs.dtype is _F64 and freqs.is_contiguous() and q.is_cuda
                and k.get_device() == q_out.get_device() == positions.get_device() == freqs.get_device() == index)
        kos = vs = kv_width
        if fits and k_out is not None:
            kos, o1, o2 = k_out.stride()
            fits = (o2 == 1 and (o1 == dim or kv_heads == 1) and (n < 2 or kos >= kv_width) and k_out.shape == k.shape
                    and k_out.dtype is q.dtype and k_out.get_device() == index)
        weight_code = GRINQH_BF16
        for w in (q_weight, k_weight):
            if w is not None:
                fits = (fits and w.dtype in _CODES and w.is_contiguous() and w.numel() == dim and w.get_device() == index
                        and (q_weight is None or w.dtype is q_weight.dtype))
                weight_code = _CODES.get(w.dtype)
        if cache is None:
            fits = fits and k_out is not None and v is None and slots is None
        else:
            vs, v1, v2 = v.stride()
            fits = (fits and isinstance(cache, KVCache) and cache.device == device and cache.n_kv_heads == kv_heads
                    and cache.head_dim == dim and v2 == 1 and (v1 == dim or kv_heads == 1) and (n < 2 or vs >= kv_width)
                    and v.shape == k.shape and v.dtype is q.dtype and v.get_device() == index and slots.dtype is _I64
                    and slots.is_contiguous() and slots.numel() == n and slots.get_device() == index)
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        _check_rope(q, k, positions, freqs, q_weight, k_weight, cache, v, slots, q_out, k_out)
        raise ValueError("the operands do not fit one another")
    if n < 2:                                    # one token: its distance to the next is never used
        qs = os = width
        ks = kos = vs = kv_width
    a = RopeArgs(q.data_ptr(), k.data_ptr(), None if v is None else v.data_ptr(), qs, ks, vs, n, heads, kv_heads, dim,
                 _CODES[q.dtype], None if q_weight is None else q_weight.data_ptr(),
                 None if k_weight is None else k_weight.data_ptr(), weight_code, eps, positions.data_ptr(),
                 freqs.data_ptr(), min(2 * freqs.numel(), 1 << 30), bool(neighbours), q_out.data_ptr(),
                 None if k_out is None else k_out.data_ptr(), os, kos)
    if cache is not None:
        (a.cache, a.pools), a.slots = cache._pointers, slots.data_ptr()
    _run("grinqh_qk_rope", device, stream, ctypes.byref(a))


def qk_rope(q, k, positions, freqs, q_weight=None, k_weight=None, eps: float = 1e-6, neighbours: bool = False,
            cache: KVCache = None, v=None, slots=None, keys: bool = True, stream=None):
    """(q, k) normed for each head (where there are weights) and rotated by their
    positions, contiguous (allocates them).  freqs: float64 [rope_dim / 2], radians per
    position; pairs are (p, p + rope_dim / 2), or with neighbours (2p, 2p + 1).  With a
    cache, keys and values (v) also go into their slots; keys=False then leaves
    the rotated keys to the cache alone (k is None in the result)."""
    if stream is None and isinstance(q, torch.Tensor) and isinstance(k, torch.Tensor) and q.is_cuda and k.is_cuda:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)       # the shorter way there
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format) if keys else None
    else:
        device = _tensor(q, "q")
        _tensor(k, "k", device)
        q_out = _empty(q.shape, q.dtype, device, stream)
        k_out = _empty(k.shape, k.dtype, device, stream) if keys else None
    grinqh_qk_rope(q, k, positions, freqs, q_out, k_out, q_weight, k_weight, eps, neighbours, cache, v, slots, stream)
    return q_out, k_out
