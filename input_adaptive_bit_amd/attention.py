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

import ctypes

try:
    import torch
except ImportError:                              # the host calls below need no torch
    torch = None

from .grinqh import (GRINQH_BF16, GRINQH_EINVAL, GRINQH_F32, GrinqhError, KVLayout, KVPools, PrefillAttentionArgs,
                     _check, load)


if torch is not None:
    _CODES = {torch.bfloat16: GRINQH_BF16, torch.float32: GRINQH_F32}
    _BF16, _I32, _I64 = torch.bfloat16, torch.int32, torch.int64

_COUNTER_BYTES = 16384                           # of a decode attention's workspace, zero before its first use
_LONGEST = 1 << 28                               # max_len that the library takes


# ------------------------------------------------------------------ host ----

def _fit(x, bits: int = 32) -> int:
    """x, or the end of the type's range nearest to it: ctypes would drop the
    higher bits, and the library refuses either end of every size."""
    return max(-1 << bits - 1, min(int(x), (1 << bits - 1) - 1))


def grinqh_kv_layout_init(n_kv_heads: int, head_dim: int, page_size: int, n_pages: int, bits: int) -> KVLayout:
    L = KVLayout()
    _check(load().grinqh_kv_layout_init(_fit(n_kv_heads), _fit(head_dim), _fit(page_size), _fit(n_pages), _fit(bits),
                                        ctypes.byref(L)), "grinqh_kv_layout_init")
    return L


def grinqh_kv_code_bytes(L: KVLayout) -> int:
    return int(load().grinqh_kv_code_bytes(ctypes.byref(L)))


def grinqh_kv_grid_bytes(L: KVLayout) -> int:
    return int(load().grinqh_kv_grid_bytes(ctypes.byref(L)))


def grinqh_debug_kv_row(L: KVLayout, slot: int, head: int) -> int:
    return int(load().grinqh_debug_kv_row(ctypes.byref(L), _fit(slot, 64), _fit(head)))


def grinqh_debug_page_row(L: KVLayout, page: int, head: int, t: int) -> int:
    return int(load().grinqh_debug_page_row(ctypes.byref(L), _fit(page), _fit(head),
                                              int(t) if 0 <= t < 1 << 31 else -1))


def grinqh_attention_workspace_bytes(L: KVLayout, n_q_heads: int, batch: int, max_len: int) -> int:
    return int(load().grinqh_attention_workspace_bytes(ctypes.byref(L), _fit(n_q_heads), _fit(batch), _fit(max_len)))


# ---------------------------------------------------------------- checks ----
#
# Each call tests all its conditions in one expression, which costs a program
# 2 us a call, and only if one fails goes through them one by one to say which.


def _tensor(t, name, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t.device


def _plain(t, name, dtype, device, numel):
    """The address of a contiguous tensor of one type with at least numel elements."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.get_device() == device.index
            and t.is_contiguous() and t.numel() >= numel):
        return t.data_ptr()
    _tensor(t, name, device)                     # the reason why not
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} is too small ({t.numel()} < {numel} elements)")
    return t.data_ptr()


def _floats(t, name, device, numel):
    """The same for a tensor of a type that _float_code takes."""
    _float_code(t.dtype if isinstance(t, torch.Tensor) else None, name)
    return _plain(t, name, t.dtype, device, numel)


def _float_code(dtype, name) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, not {dtype}")
    return code


def _rows(t, name, heads, dim, device):
    """Token stride in elements of [tokens][heads][dim] whose token rows are
    each contiguous (the tokens may lie further apart)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == device.index):
        _tensor(t, name, device)                 # the reason why not
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens][{heads}][{dim}], not {list(shape)}")
    if stride[2] != 1 or (heads > 1 and stride[1] != dim):
        raise ValueError(f"a token's rows of {name} must be contiguous (strides {stride})")
    if shape[0] < 2:
        return heads * dim                   # one token: its distance to the next is never used
    if stride[0] < heads * dim:
        raise ValueError(f"the tokens of {name} must not overlap (strides {stride})")
    return stride[0]


def _raw_stream(device, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if hasattr(stream, "cuda_stream"):
        if getattr(stream, "device", device) != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return stream.cuda_stream
    return int(stream)


def _run(name, device, stream, *args) -> None:
    """Calls an entry point whose last argument is the stream, with the tensors'
    device current."""
    call, raw = getattr(load(), name), _raw_stream(device, stream)
    if torch._C._cuda_getDevice() == device.index:
        status = call(*args, raw)
    else:
        with torch.cuda.device(device):
            status = call(*args, raw)
    if status:
        _check(status, name)


def _empty(shape, dtype, device, stream):
    """An output that belongs to the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_as(t, dtype, device, stream):
    """An output of t's shape."""
    if stream is None and t.dtype is dtype and t.device == device:       # the shorter way there
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _empty(t.shape, dtype, device, stream)


def _workspace(n, device, stream):
    """A decode attention's workspace, ready for its first call, on the call's stream."""
    if stream is None:
        if n <= 1 << 20:
            return torch.zeros(n, dtype=torch.uint8, device=device)
        w = torch.empty(n, dtype=torch.uint8, device=device)
        w[:_COUNTER_BYTES].zero_()               # sooner than to fill all of a large one
        return w
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return _workspace(n, device, None)


# ------------------------------------------------------------------ cache ---

class KVCache:
    """One layer's paged cache: the layout and the tensors that hold its rows.

    k_codes, v_codes: uint8 [n_pages][n_kv_heads][page_size][row_bytes];
    k_grid, v_grid: float16 [n_pages][n_kv_heads][page_size][2], not used (and
    may be None) at 16 bits.
    """

    def __init__(self, layout: KVLayout, k_codes, v_codes, k_grid=None, v_grid=None):
        n, g = grinqh_kv_code_bytes(layout), grinqh_kv_grid_bytes(layout) // 2
        if n == 0:
            raise GrinqhError(GRINQH_EINVAL, "KVCache")
        self.device = _tensor(k_codes, "k_codes")
        pools = [_plain(k_codes, "k_codes", torch.uint8, self.device, n),
                 _plain(v_codes, "v_codes", torch.uint8, self.device, n)]
        if g:
            pools += [_plain(k_grid, "k_grid", torch.float16, self.device, g),
                      _plain(v_grid, "v_grid", torch.float16, self.device, g)]
        self.layout, self.k_codes, self.v_codes, self.k_grid, self.v_grid = layout, k_codes, v_codes, k_grid, v_grid
        self.n_kv_heads, self.head_dim = layout.n_kv_heads, layout.head_dim
        self._pools = KVPools(*pools)
        self._refs = ctypes.byref(layout), ctypes.byref(self._pools)
        self._pointers = ctypes.pointer(layout), ctypes.pointer(self._pools)


def new_kv_cache(n_kv_heads: int, head_dim: int, page_size: int, n_pages: int, bits: int, device=None) -> KVCache:
    """A cache of zeros on `device`."""
    L = grinqh_kv_layout_init(n_kv_heads, head_dim, page_size, n_pages, bits)
    device = device or "cuda"
    rows = (n_pages, n_kv_heads, page_size)
    codes = [torch.zeros(*rows, L.row_bytes, dtype=torch.uint8, device=device) for _ in range(2)]
    grid = [torch.zeros(*rows, 2, dtype=torch.float16, device=device) if bits < 16 else None for _ in range(2)]
    return KVCache(L, *codes, *grid)


def new_attention_workspace(L: KVLayout, n_q_heads: int, batch: int, max_len: int, device=None):
    """A zero-filled workspace tensor for grinqh_decode_attention on `device`: for
    calls of up to this batch and max_len."""
    n = grinqh_attention_workspace_bytes(L, n_q_heads, batch, max_len)
    if n == 0:
        raise GrinqhError(GRINQH_EINVAL, "grinqh_attention_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def grinqh_kv_write(cache: KVCache, k, v, slots, stream=None) -> None:
    """k, v: bf16 or fp32 [tokens][n_kv_heads][head_dim], token rows contiguous;
    slots: int64 [tokens]."""
    device, heads, dim = cache.device, cache.n_kv_heads, cache.head_dim
    index, width = device.index, heads * dim
    try:
        n, kh, kd = k.shape
        (ks, k1, k2), (vs, v1, v2) = k.stride(), v.stride()
        fits = (kh == heads and kd == dim and k2 == v2 == 1 and (k1 == v1 == dim or heads == 1)
                and (n < 2 or (ks >= width and vs >= width)) and v.shape == k.shape and v.dtype is k.dtype
                and k.dtype in _CODES and slots.dtype is _I64 and slots.is_contiguous() and slots.numel() == n
                and k.get_device() == v.get_device() == slots.get_device() == index)
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        _rows(k, "k", heads, dim, device)
        _rows(v, "v", heads, dim, device)
        _plain(slots, "slots", _I64, device, k.shape[0])
        if v.shape[0] != k.shape[0] or slots.numel() != k.shape[0]:
            raise ValueError("k, v and slots must name the same number of tokens")
        if v.dtype != k.dtype:
            raise TypeError("k and v must have one dtype")
        _float_code(k.dtype, "k")
    if n < 2:
        ks = vs = width                          # one token: its distance to the next is never used
    _run("grinqh_kv_write", device, stream, *cache._refs, k.data_ptr(), v.data_ptr(), _CODES[k.dtype], ks, vs, n,
         slots.data_ptr())


def grinqh_kv_read(cache: KVCache, slots, k, v, stream=None) -> None:
    """k, v: bf16 or fp32 [tokens][n_kv_heads][head_dim], contiguous, overwritten."""
    device = cache.device
    n = slots.numel()
    width = n * cache.n_kv_heads * cache.head_dim
    _run("grinqh_kv_read", device, stream, *cache._refs, _plain(slots, "slots", _I64, device, n), n,
         _floats(k, "k", device, width), _plain(v, "v", k.dtype, device, width), _float_code(k.dtype, "k"))


def kv_write(cache: KVCache, k, v, slots, stream=None) -> None:
    """Write new tokens' keys and values into their slots (grinqh_kv_write)."""
    grinqh_kv_write(cache, k, v, slots, stream)


def kv_read(cache: KVCache, slots, out_dtype=None, stream=None):
    """(k, v) of the slots, [tokens][n_kv_heads][head_dim] (allocates them)."""
    device, heads, dim = cache.device, cache.n_kv_heads, cache.head_dim
    at = _plain(slots, "slots", _I64, device, 0)
    n, dtype = slots.numel(), out_dtype or _BF16
    code = _float_code(dtype, "out_dtype")
    if stream is None:                           # the shorter way to the same tensor
        both = torch.empty_strided((2, n, heads, dim), (n * heads * dim, heads * dim, dim, 1), dtype=dtype, device=device)
    else:
        both = _empty((2, n, heads, dim), dtype, device, stream)
    k = both.data_ptr()
    _run("grinqh_kv_read", device, stream, *cache._refs, at, n, k, k + both.nbytes // 2, code)
    return torch.unbind(both)


# -------------------------------------------------------------- attention ---

def grinqh_decode_attention(cache: KVCache, q, page_table, seq_lens, max_len: int, out, workspace, scale=None,
                            lse=None, stream=None) -> None:
    """q: bf16 or fp32 [batch][n_q_heads][head_dim], token rows contiguous;
    page_table: int32 [batch][max_pages]; seq_lens: int32 [batch]; out: bf16 or
    fp32, contiguous; lse: fp32 [batch][n_q_heads] or None; scale: default
    head_dim ** -0.5."""
    device, dim = cache.device, cache.head_dim
    index = device.index
    try:
        batch, heads, last = q.shape
        (q_stride, s1, s2), (rows, max_pages), (table_stride, t1) = q.stride(), page_table.shape, page_table.stride()
        width = heads * dim
        fits = (last == dim and s2 == 1 and (s1 == dim or heads == 1) and rows == batch and (t1 == 1 or max_pages < 2)
                and (batch < 2 or q_stride >= width) and q.dtype in _CODES and out.dtype in _CODES
                and page_table.dtype is _I32 and seq_lens.dtype is _I32 and seq_lens.is_contiguous()
                and seq_lens.numel() >= batch and out.is_contiguous() and out.numel() >= batch * width
                and workspace.is_contiguous() and q.get_device() == page_table.get_device() == seq_lens.get_device()
                == out.get_device() == workspace.get_device() == index)
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a [batch][n_q_heads][head_dim] tensor")
        _rows(q, "q", q.shape[1], dim, device)
        _float_code(q.dtype, "q")
        _tensor(page_table, "page_table", device)
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != q.shape[0]:
            raise ValueError("page_table must be int32 [batch][max_pages]")
        if page_table.shape[1] > 1 and page_table.stride(1) != 1:
            raise ValueError("the rows of page_table must be contiguous")
        _plain(seq_lens, "seq_lens", _I32, device, q.shape[0])
        _floats(out, "out", device, q.numel())
        _tensor(workspace, "workspace", device)
        raise ValueError("workspace must be contiguous")
    if batch < 2:
        q_stride, table_stride = width, max_pages
    _run("grinqh_decode_attention", device, stream, *cache._refs, q.data_ptr(), _CODES[q.dtype], q_stride, heads,
         page_table.data_ptr(), table_stride, max_pages, seq_lens.data_ptr(), batch,
         max_len if 0 < max_len <= _LONGEST else 0, dim ** -0.5 if scale is None else scale, out.data_ptr(),
         _CODES[out.dtype], None if lse is None else _plain(lse, "lse", torch.float32, device, batch * heads), workspace.data_ptr(),
         workspace.nbytes)


def decode_attention(cache: KVCache, q, page_table, seq_lens, max_len=None, scale=None, out_dtype=None,
                     return_lse: bool = False, workspace=None, stream=None):
    """Attention of one new token of every sequence over its cached tokens:
    out [batch][n_q_heads][head_dim], and lse if asked for (allocates them and,
    if not given, a workspace).  max_len: the host's bound on seq_lens, by default
    what the page table can hold; a long cache is cut into parts by it, so one
    near the longest length is faster."""
    device = cache.device
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [batch][n_q_heads][head_dim] tensor")
    batch, heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError(f"q must be [batch][n_q_heads][{cache.head_dim}], not {list(q.shape)}")
    if max_len is None:
        max_len = min(max(1, page_table.shape[1] * cache.layout.page_size), _LONGEST)
    out = _empty_as(q, out_dtype or torch.bfloat16, device, stream)
    lse = _empty((batch, heads), torch.float32, device, stream) if return_lse else None
    if workspace is None:
        workspace = _workspace(grinqh_attention_workspace_bytes(cache.layout, heads, batch, max_len), device, stream)
    grinqh_decode_attention(cache, q, page_table, seq_lens, max_len, out, workspace, scale, lse, stream)
    return (out, lse) if return_lse else out


def _prefill_args(q, k, v, cu_q, cu_k, out, causal, scale, lse):
    """The checked arguments of a prefill attention, without a workspace."""
    device = _tensor(q, "q")
    index = device.index
    try:
        (total_q, heads, dim), (total_k, kv_heads, kd) = q.shape, k.shape
        (qs, q1, q2), (ks, k1, k2), (vs, v1, v2) = q.stride(), k.stride(), v.stride()
        q_width, width, ends = heads * dim, kv_heads * dim, cu_q.numel()
        fits = (kd == dim and q2 == k2 == v2 == 1 and (q1 == dim or heads == 1) and (k1 == v1 == dim or kv_heads == 1)
                and (total_q < 2 or qs >= q_width) and (total_k < 2 or (ks >= width and vs >= width))
                and v.shape == k.shape and q.dtype is k.dtype is v.dtype is _BF16 and cu_q.dtype is cu_k.dtype is _I32
                and cu_q.is_contiguous() and cu_k.is_contiguous() and cu_k.numel() == ends > 0 and out.dtype in _CODES
                and out.is_contiguous() and out.numel() >= total_q * q_width and k.get_device() == v.get_device()
                == cu_q.get_device() == cu_k.get_device() == out.get_device() == index)
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError("q and k must be [tokens][heads][head_dim]")
        _rows(q, "q", q.shape[1], q.shape[2], device)
        _rows(k, "k", k.shape[1], q.shape[2], device)
        _rows(v, "v", k.shape[1], q.shape[2], device)
        if v.shape[0] != k.shape[0]:
            raise ValueError("k and v must hold the same tokens")
        if q.dtype != _BF16 or k.dtype != _BF16 or v.dtype != _BF16:
            raise TypeError(f"q, k and v must be bfloat16, not {q.dtype}, {k.dtype}, {v.dtype}")
        _plain(cu_q, "cu_q", _I32, device, 1)
        _plain(cu_k, "cu_k", _I32, device, 1)
        if cu_k.numel() != cu_q.numel():
            raise ValueError("cu_q and cu_k must both be [batch + 1]")
        _floats(out, "out", device, q.numel())
    return PrefillAttentionArgs(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), qs if total_q > 1 else q_width, ks if total_k > 1 else width,
        vs if total_k > 1 else width, cu_q.data_ptr(), cu_k.data_ptr(), ends - 1 if ends <= 1 << 31 else -1,
        total_q, total_k, heads, kv_heads, dim, bool(causal), dim ** -0.5 if scale is None else scale,
        out.data_ptr(), _CODES[out.dtype], None if lse is None else _plain(lse, "lse", torch.float32, device, total_q * heads))


def grinqh_prefill_attention_workspace_bytes(q, k, v, cu_q, cu_k, out, causal: bool = True) -> int:
    """Workspace with which grinqh_prefill_attention splits these tensors' keys
    (0: it does not)."""
    a = _prefill_args(q, k, v, cu_q, cu_k, out, causal, None, None)
    return int(load().grinqh_prefill_attention_workspace_bytes(ctypes.byref(a)))


def grinqh_prefill_attention(q, k, v, cu_q, cu_k, out, causal: bool = True, scale=None, lse=None, workspace=None,
                             stream=None) -> None:
    """q: bf16 [total_q][n_q_heads][head_dim]; k, v: bf16
    [total_k][n_kv_heads][head_dim], token rows contiguous; cu_q, cu_k: int32
    [batch + 1]; out: bf16 or fp32 [total_q][n_q_heads][head_dim], contiguous;
    workspace: any contents, or None (the keys are not split then)."""
    a = _prefill_args(q, k, v, cu_q, cu_k, out, causal, scale, lse)
    if workspace is not None:
        _tensor(workspace, "workspace", q.device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if workspace.numel():
            a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.nbytes
    _run("grinqh_prefill_attention", q.device, stream, ctypes.byref(a))


def prefill_attention(q, k, v, cu_q, cu_k=None, causal: bool = True, scale=None, out_dtype=None,
                      return_lse: bool = False, stream=None):
    """Attention over packed prompts: out [total_q][n_q_heads][head_dim], and
    lse [total_q][n_q_heads] if asked for (allocates them, and the workspace).
    cu_k defaults to cu_q (every prompt's keys are its own tokens). Rows behind
    the last sequence are left as they are allocated."""
    device = _tensor(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [tokens][heads][head_dim]")
    out = _empty_as(q, out_dtype or torch.bfloat16, device, stream)
    lse = _empty(q.shape[:2], torch.float32, device, stream) if return_lse else None
    a = _prefill_args(q, k, v, cu_q, cu_q if cu_k is None else cu_k, out, causal, scale, lse)
    n = load().grinqh_prefill_attention_workspace_bytes(ctypes.byref(a))
    if n:
        workspace = _empty((n,), torch.uint8, device, stream)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), n
    _run("grinqh_prefill_attention", device, stream, ctypes.byref(a))
    return (out, lse) if return_lse else out
