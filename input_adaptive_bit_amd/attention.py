"""Python binding of the key-value cache and the attention calls of
libgrinqh.so (include/grinqh.h).

As in grinqh.py, the functions with the C names take caller-allocated tensors;
the short names (kv_write, kv_read, decode_attention, prefill_attention)
allocate their outputs and call the same entry points.  A call runs on the
device of its tensors, on `stream` or that device's current stream; what it
allocates belongs to that stream.  Argument marshalling only: there is no CPU
fallback.
"""

from __future__ import annotations

import contextlib
import ctypes

from .grinqh import (GRINQH_BF16, GRINQH_EINVAL, GRINQH_F32, GrinqhError, KVLayout, KVPools, PrefillAttentionArgs,
                     _check, load)


# ------------------------------------------------------------------ host ----

def grinqh_kv_layout_init(n_kv_heads: int, head_dim: int, page_size: int, n_pages: int, bits: int) -> KVLayout:
    L = KVLayout()
    _check(load().grinqh_kv_layout_init(int(n_kv_heads), int(head_dim), int(page_size), int(n_pages), int(bits),
                                        ctypes.byref(L)), "grinqh_kv_layout_init")
    return L


def grinqh_kv_code_bytes(L: KVLayout) -> int:
    return int(load().grinqh_kv_code_bytes(ctypes.byref(L)))


def grinqh_kv_grid_bytes(L: KVLayout) -> int:
    return int(load().grinqh_kv_grid_bytes(ctypes.byref(L)))


def grinqh_debug_kv_row(L: KVLayout, slot: int, head: int) -> int:
    return int(load().grinqh_debug_kv_row(ctypes.byref(L), int(slot), int(head)))


def grinqh_attention_workspace_bytes(L: KVLayout, n_q_heads: int, batch: int, max_len: int) -> int:
    return int(load().grinqh_attention_workspace_bytes(ctypes.byref(L), int(n_q_heads), int(batch), int(max_len)))


# ---------------------------------------------------------------- checks ----

def _tensor(t, name, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t.device


def _plain(t, name, dtype, device, numel):
    """A contiguous tensor of one type with at least numel elements."""
    _tensor(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} is too small ({t.numel()} < {numel} elements)")


def _float_code(dtype, name) -> int:
    import torch
    if dtype == torch.bfloat16:
        return GRINQH_BF16
    if dtype == torch.float32:
        return GRINQH_F32
    raise TypeError(f"{name} must be bfloat16 or float32, not {dtype}")


def _rows(t, name, heads, dim, device):
    """Token stride in elements of [tokens][heads][dim] whose token rows are
    each contiguous (the tokens may lie further apart)."""
    _tensor(t, name, device)
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must be [tokens][{heads}][{dim}], not {list(t.shape)}")
    st, sh, sd = t.stride()
    if sd != 1 or (heads > 1 and sh != dim):
        raise ValueError(f"a token's rows of {name} must be contiguous (strides {t.stride()})")
    if t.shape[0] < 2:
        return heads * dim                   # one token: its distance to the next is never used
    if st < heads * dim:
        raise ValueError(f"the tokens of {name} must not overlap (strides {t.stride()})")
    return st


@contextlib.contextmanager
def _on(device):
    import torch
    if torch.cuda.current_device() == device.index:
        yield
    else:
        with torch.cuda.device(device):
            yield


def _stream_of(device, stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if hasattr(stream, "cuda_stream"):
        if getattr(stream, "device", device) != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, device, stream):
    """An output that belongs to the call's stream."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# ------------------------------------------------------------------ cache ---

class KVCache:
    """One layer's paged cache: the layout and the tensors that hold its rows.

    k_codes, v_codes: uint8 [n_pages][n_kv_heads][page_size][row_bytes];
    k_grid, v_grid: float16 [n_pages][n_kv_heads][page_size][2], not used (and
    may be None) at 16 bits.
    """

    def __init__(self, layout: KVLayout, k_codes, v_codes, k_grid=None, v_grid=None):
        import torch
        n, g = grinqh_kv_code_bytes(layout), grinqh_kv_grid_bytes(layout) // 2
        if n == 0:
            raise GrinqhError(GRINQH_EINVAL, "KVCache")
        self.device = _tensor(k_codes, "k_codes")
        _plain(k_codes, "k_codes", torch.uint8, self.device, n)
        _plain(v_codes, "v_codes", torch.uint8, self.device, n)
        if g:
            _plain(k_grid, "k_grid", torch.float16, self.device, g)
            _plain(v_grid, "v_grid", torch.float16, self.device, g)
        self.layout, self.k_codes, self.v_codes, self.k_grid, self.v_grid = layout, k_codes, v_codes, k_grid, v_grid
        self._pools = KVPools(k_codes.data_ptr(), v_codes.data_ptr(), k_grid.data_ptr() if g else None,
                              v_grid.data_ptr() if g else None)


def new_kv_cache(n_kv_heads: int, head_dim: int, page_size: int, n_pages: int, bits: int, device=None) -> KVCache:
    """A cache of zeros on `device`."""
    import torch
    L = grinqh_kv_layout_init(n_kv_heads, head_dim, page_size, n_pages, bits)
    device = device or "cuda"
    rows = (n_pages, n_kv_heads, page_size)
    codes = [torch.zeros(*rows, L.row_bytes, dtype=torch.uint8, device=device) for _ in range(2)]
    grid = [torch.zeros(*rows, 2, dtype=torch.float16, device=device) if bits < 16 else None for _ in range(2)]
    return KVCache(L, *codes, *grid)


def new_attention_workspace(L: KVLayout, n_q_heads: int, batch: int, max_len: int, device=None):
    """A zero-filled workspace tensor for grinqh_decode_attention on `device`."""
    import torch
    n = grinqh_attention_workspace_bytes(L, n_q_heads, batch, max_len)
    if n == 0:
        raise GrinqhError(GRINQH_EINVAL, "grinqh_attention_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def grinqh_kv_write(cache: KVCache, k, v, slots, stream=None) -> None:
    """k, v: bf16 or fp32 [tokens][n_kv_heads][head_dim], token rows contiguous;
    slots: int64 [tokens]."""
    import torch
    L, device = cache.layout, cache.device
    k_stride = _rows(k, "k", L.n_kv_heads, L.head_dim, device)
    v_stride = _rows(v, "v", L.n_kv_heads, L.head_dim, device)
    n = k.shape[0]
    if v.shape[0] != n or slots.numel() != n:
        raise ValueError("k, v and slots must name the same number of tokens")
    if v.dtype != k.dtype:
        raise TypeError("k and v must have one dtype")
    _plain(slots, "slots", torch.int64, device, n)
    with _on(device):
        _check(load().grinqh_kv_write(ctypes.byref(L), ctypes.byref(cache._pools), k.data_ptr(), v.data_ptr(),
                                      _float_code(k.dtype, "k"), k_stride, v_stride, n, slots.data_ptr(),
                                      _stream_of(device, stream)), "grinqh_kv_write")


def grinqh_kv_read(cache: KVCache, slots, k, v, stream=None) -> None:
    """k, v: bf16 or fp32 [tokens][n_kv_heads][head_dim], contiguous, overwritten."""
    import torch
    L, device = cache.layout, cache.device
    n = slots.numel()
    _plain(slots, "slots", torch.int64, device, n)
    for name, t in (("k", k), ("v", v)):
        _plain(t, name, k.dtype, device, n * L.n_kv_heads * L.head_dim)
    with _on(device):
        _check(load().grinqh_kv_read(ctypes.byref(L), ctypes.byref(cache._pools), slots.data_ptr(), n, k.data_ptr(),
                                     v.data_ptr(), _float_code(k.dtype, "k"), _stream_of(device, stream)),
               "grinqh_kv_read")


def kv_write(cache: KVCache, k, v, slots, stream=None) -> None:
    """Write new tokens' keys and values into their slots (grinqh_kv_write)."""
    grinqh_kv_write(cache, k, v, slots, stream)


def kv_read(cache: KVCache, slots, out_dtype=None, stream=None):
    """(k, v) of the slots, [tokens][n_kv_heads][head_dim] (allocates them)."""
    import torch
    L = cache.layout
    shape = (slots.numel(), L.n_kv_heads, L.head_dim)
    k, v = (_empty(shape, out_dtype or torch.bfloat16, cache.device, stream) for _ in range(2))
    grinqh_kv_read(cache, slots, k, v, stream)
    return k, v


# -------------------------------------------------------------- attention ---

def grinqh_decode_attention(cache: KVCache, q, page_table, seq_lens, max_len: int, out, workspace, scale=None,
                            lse=None, stream=None) -> None:
    """q: bf16 or fp32 [batch][n_q_heads][head_dim], token rows contiguous;
    page_table: int32 [batch][max_pages]; seq_lens: int32 [batch]; out: bf16 or
    fp32, contiguous; lse: fp32 [batch][n_q_heads] or None; scale: default
    head_dim ** -0.5."""
    import torch
    L, device = cache.layout, cache.device
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [batch][n_q_heads][head_dim] tensor")
    batch, heads = q.shape[0], q.shape[1]
    q_stride = _rows(q, "q", heads, L.head_dim, device)
    _tensor(page_table, "page_table", device)
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError("page_table must be int32 [batch][max_pages]")
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("the rows of page_table must be contiguous")
    max_pages = page_table.shape[1]
    table_stride = page_table.stride(0) if batch > 1 else max_pages
    _plain(seq_lens, "seq_lens", torch.int32, device, batch)
    _tensor(out, "out", device)
    _plain(out, "out", out.dtype, device, batch * heads * L.head_dim)
    if lse is not None:
        _plain(lse, "lse", torch.float32, device, batch * heads)
    _tensor(workspace, "workspace", device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    with _on(device):
        _check(load().grinqh_decode_attention(
            ctypes.byref(L), ctypes.byref(cache._pools), q.data_ptr(), _float_code(q.dtype, "q"), q_stride, heads,
            page_table.data_ptr(), table_stride, max_pages, seq_lens.data_ptr(), batch, max_len,
            L.head_dim ** -0.5 if scale is None else scale, out.data_ptr(), _float_code(out.dtype, "out"),
            None if lse is None else lse.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_of(device, stream)), "grinqh_decode_attention")


def decode_attention(cache: KVCache, q, page_table, seq_lens, max_len=None, scale=None, out_dtype=None,
                     return_lse: bool = False, workspace=None, stream=None):
    """Attention of one new token of every sequence over its cached tokens:
    out [batch][n_q_heads][head_dim], and lse if asked for (allocates them and,
    if not given, a zero-filled workspace).  max_len: the host's bound on
    seq_lens, by default what the page table can hold."""
    import torch
    L, device = cache.layout, cache.device
    batch, heads = q.shape[0], q.shape[1]
    if max_len is None:
        max_len = max(1, page_table.shape[1] * L.page_size)
    out = _empty((batch, heads, L.head_dim), out_dtype or torch.bfloat16, device, stream)
    lse = _empty((batch, heads), torch.float32, device, stream) if return_lse else None
    if workspace is None:
        n = grinqh_attention_workspace_bytes(L, heads, batch, max_len)
        workspace = _empty((n,), torch.uint8, device, stream)
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(
                stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)):
            workspace.zero_()
    grinqh_decode_attention(cache, q, page_table, seq_lens, max_len, out, workspace, scale, lse, stream)
    return (out, lse) if return_lse else out


def grinqh_prefill_attention(q, k, v, cu_q, cu_k, out, causal: bool = True, scale=None, lse=None,
                             stream=None) -> None:
    """q: bf16 [total_q][n_q_heads][head_dim]; k, v: bf16
    [total_k][n_kv_heads][head_dim], token rows contiguous; cu_q, cu_k: int32
    [batch + 1]; out: bf16 or fp32 [total_q][n_q_heads][head_dim], contiguous."""
    import torch
    device = _tensor(q, "q")
    _tensor(k, "k", device)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens][heads][head_dim]")
    total_q, heads, dim = q.shape
    total_k, kv_heads = k.shape[0], k.shape[1]
    q_stride = _rows(q, "q", heads, dim, device)
    k_stride = _rows(k, "k", kv_heads, dim, device)
    v_stride = _rows(v, "v", kv_heads, dim, device)
    if v.shape[0] != total_k:
        raise ValueError("k and v must hold the same tokens")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16, not {t.dtype}")
    batch = cu_q.numel() - 1
    if batch < 0 or cu_k.numel() != batch + 1:
        raise ValueError("cu_q and cu_k must both be [batch + 1]")
    _plain(cu_q, "cu_q", torch.int32, device, batch + 1)
    _plain(cu_k, "cu_k", torch.int32, device, batch + 1)
    _plain(out, "out", out.dtype, device, total_q * heads * dim)
    if lse is not None:
        _plain(lse, "lse", torch.float32, device, total_q * heads)
    a = PrefillAttentionArgs(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride, cu_q.data_ptr(), cu_k.data_ptr(),
        batch, total_q, total_k, heads, kv_heads, dim, int(bool(causal)), dim ** -0.5 if scale is None else scale,
        out.data_ptr(), _float_code(out.dtype, "out"), None if lse is None else lse.data_ptr())
    with _on(device):
        _check(load().grinqh_prefill_attention(ctypes.byref(a), _stream_of(device, stream)),
               "grinqh_prefill_attention")


def prefill_attention(q, k, v, cu_q, cu_k=None, causal: bool = True, scale=None, out_dtype=None,
                      return_lse: bool = False, stream=None):
    """Attention over packed prompts: out [total_q][n_q_heads][head_dim], and
    lse [total_q][n_q_heads] if asked for (allocates them).  cu_k defaults to
    cu_q (every prompt's keys are its own tokens)."""
    import torch
    device = _tensor(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [tokens][heads][head_dim]")
    out = _empty(tuple(q.shape), out_dtype or torch.bfloat16, device, stream)
    lse = _empty(tuple(q.shape[:2]), torch.float32, device, stream) if return_lse else None
    grinqh_prefill_attention(q, k, v, cu_q, cu_q if cu_k is None else cu_k, out, causal, scale, lse, stream)
    return (out, lse) if return_lse else out
