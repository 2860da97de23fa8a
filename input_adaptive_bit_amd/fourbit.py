"""Python binding of the products with 4-bit weights of libgrinqh.so
(include/grinqh.h): plain layers and layers grouped by expert.

As in grinqh.py, the functions with the C names take caller-allocated tensors;
the short names allocate their outputs and call the same entry points.  A call
runs on the device of its tensors, on `stream` or that device's current stream.
Argument marshalling only: there is no CPU fallback.
"""

from __future__ import annotations

import ctypes

try:
    import torch
except ImportError:                              # the host calls below need no torch
    torch = None

from .attention import _empty, _fit, _float_code, _plain, _run, _tensor
from .grinqh import GRINQH_EINVAL, ExpertArgs, FourbitLayout, GrinqhError, _check, load

if torch is not None:
    from .attention import _CODES
    _I32, _U8, _F16 = torch.int32, torch.uint8, torch.float16

_MOST_ROWS = 1 << 30                             # that a call of grinqh_quantize_rtn takes


# ------------------------------------------------------------------ host ----

def grinqh_fourbit_layout_init(d_in: int, d_out: int, group: int, n_experts: int = 1) -> FourbitLayout:
    L = FourbitLayout()
    _check(load().grinqh_fourbit_layout_init(_fit(d_in), _fit(d_out), _fit(group), _fit(n_experts), ctypes.byref(L)),
           "grinqh_fourbit_layout_init")
    return L


def grinqh_fourbit_code_bytes(L: FourbitLayout) -> int:
    return int(load().grinqh_fourbit_code_bytes(ctypes.byref(L)))


def grinqh_fourbit_grid_bytes(L: FourbitLayout) -> int:
    return int(load().grinqh_fourbit_grid_bytes(ctypes.byref(L)))


class FourbitWeight:
    """Packed 4-bit weights of one layer, or of a layer's experts: the layout and
    the tensors that hold codes (uint8) and scales and zero points (float16)."""

    def __init__(self, layout: FourbitLayout, codes, grid):
        n, g = grinqh_fourbit_code_bytes(layout), grinqh_fourbit_grid_bytes(layout) // 2
        if n == 0:
            raise GrinqhError(GRINQH_EINVAL, "FourbitWeight")
        self.device = _tensor(codes, "codes")
        self._at = _plain(codes, "codes", _U8, self.device, n), _plain(grid, "grid", _F16, self.device, g)
        self.layout, self.codes, self.grid = layout, codes, grid
        self.d_in, self.d_out, self.n_experts = layout.d_in, layout.d_out, layout.n_experts
        self._ref = ctypes.byref(layout)


# --------------------------------------------------------------- device -----

def grinqh_fourbit_pack(L: FourbitLayout, q, s, z, codes, grid, stream=None) -> None:
    """q: uint8 [n_experts][d_out][d_in]; s, z: float16 [n_experts][d_out][d_in / group];
    codes: uint8, grid: float16, of the layout's sizes (all contiguous)."""
    device = _tensor(q, "q")
    n = L.n_experts * L.d_out
    groups = L.d_in // L.group if L.group > 0 else 0
    if q.numel() != n * L.d_in:
        raise ValueError(f"q must be [{L.n_experts}][{L.d_out}][{L.d_in}], not {list(q.shape)}")
    _run("grinqh_fourbit_pack", device, stream, ctypes.byref(L), _plain(q, "q", _U8, device, n * L.d_in),
         _plain(s, "s", _F16, device, n * groups), _plain(z, "z", _F16, device, n * groups),
         _plain(codes, "codes", _U8, device, grinqh_fourbit_code_bytes(L)),
         _plain(grid, "grid", _F16, device, grinqh_fourbit_grid_bytes(L) // 2))


def _row_stride(x, d_in, device) -> int:
    """Elements between the rows of x [rows][d_in], each of them contiguous."""
    _tensor(x, "x", device)
    if x.dim() != 2 or x.shape[1] != d_in:
        raise ValueError(f"x must be [tokens][{d_in}], not {list(x.shape)}")
    if d_in > 1 and x.stride(1) != 1:
        raise ValueError(f"a row of x must be contiguous (strides {x.stride()})")
    _float_code(x.dtype, "x")
    if x.shape[0] < 2:
        return d_in                              # one row: its distance to the next is never used
    if x.stride(0) < d_in:
        raise ValueError(f"the rows of x must not overlap (strides {x.stride()})")
    return x.stride(0)


def _output(y, rows, d_out, device) -> int:
    _float_code(y.dtype if isinstance(y, torch.Tensor) else None, "y")
    return _plain(y, "y", y.dtype, device, rows * d_out)


def grinqh_fourbit_linear(weight: FourbitWeight, x, y, stream=None) -> None:
    """x: bf16 or fp32 [tokens][d_in], rows contiguous; y: bf16 or fp32 [tokens][d_out], contiguous, overwritten."""
    device, d_in, d_out = weight.device, weight.d_in, weight.d_out
    try:
        n, width = x.shape
        stride, s1 = x.stride()
        fits = (width == d_in and s1 == 1 and (n < 2 or stride >= d_in) and x.dtype in _CODES and y.dtype in _CODES
                and y.is_contiguous() and y.numel() >= n * d_out and x.get_device() == y.get_device() == device.index)
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        _row_stride(x, d_in, device)
        _output(y, x.shape[0], d_out, device)
        raise ValueError("x and y do not fit the weight")
    _run("grinqh_fourbit_linear", device, stream, weight._ref, x.data_ptr(), _CODES[x.dtype], stride if n > 1 else d_in, n,
         *weight._at, y.data_ptr(), _CODES[y.dtype])


def grinqh_expert_linear(weight: FourbitWeight, x, ends, y, rows=None, stream=None) -> None:
    """x: bf16 or fp32 [n_x][d_in], rows contiguous; ends: int32 [n_experts + 1];
    y: bf16 or fp32 [n_rows][d_out], contiguous; rows: int32 [n_rows] or None."""
    device, d_in, d_out = weight.device, weight.d_in, weight.d_out
    index = device.index
    try:
        n_x, width = x.shape
        n, out_width = y.shape
        stride, s1 = x.stride()
        fits = (width == d_in and out_width == d_out and s1 == 1 and (n_x < 2 or stride >= d_in) and x.dtype in _CODES
                and y.dtype in _CODES and y.is_contiguous() and ends.dtype is _I32 and ends.is_contiguous()
                and ends.numel() == weight.n_experts + 1 and x.get_device() == y.get_device() == ends.get_device() == index
                and (rows is None or (rows.dtype is _I32 and rows.is_contiguous() and rows.numel() == n
                                      and rows.get_device() == index)))
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        _row_stride(x, d_in, device)
        if not isinstance(y, torch.Tensor) or y.dim() != 2 or y.shape[1] != d_out:
            raise ValueError(f"y must be a [rows][{d_out}] tensor")
        _output(y, y.shape[0], d_out, device)
        _plain(ends, "ends", _I32, device, weight.n_experts + 1)
        if ends.numel() != weight.n_experts + 1:
            raise ValueError(f"ends must be [{weight.n_experts + 1}], not {list(ends.shape)}")
        if rows is not None:
            _plain(rows, "rows", _I32, device, y.shape[0])
            if rows.numel() != y.shape[0]:
                raise ValueError("rows must name a row of x for every row of y")
        raise ValueError("the operands do not fit the weight")
    a = ExpertArgs(x.data_ptr(), stride if n_x > 1 else d_in, _CODES[x.dtype], n_x, None if rows is None else rows.data_ptr(),
                   ends.data_ptr(), n, *weight._at, y.data_ptr(), _CODES[y.dtype])
    _run("grinqh_expert_linear", device, stream, weight._ref, ctypes.byref(a))


# ------------------------------------------------- allocating conveniences --

def fourbit_pack(q, s, z, stream=None) -> FourbitWeight:
    """Packs codes uint8 [d_out][d_in] (or [n_experts][d_out][d_in]) and float16 scales and zero
    points [..][d_in / group] (allocates what holds them)."""
    device = _tensor(q, "q")
    if q.dim() not in (2, 3) or not isinstance(s, torch.Tensor) or s.dim() != q.dim() or s.shape[-1] == 0:
        raise ValueError("q must be [d_out][d_in] or [n_experts][d_out][d_in], s and z with a column for every group")
    if s.shape[:-1] != q.shape[:-1] or q.shape[-1] % s.shape[-1] != 0:
        raise ValueError(f"s {list(s.shape)} does not fit q {list(q.shape)}")
    if not isinstance(z, torch.Tensor) or z.shape != s.shape:
        raise ValueError("z must have the shape of s")
    L = grinqh_fourbit_layout_init(q.shape[-1], q.shape[-2], q.shape[-1] // s.shape[-1], q.shape[0] if q.dim() == 3 else 1)
    codes = _empty((grinqh_fourbit_code_bytes(L),), _U8, device, stream)
    grid = _empty((grinqh_fourbit_grid_bytes(L) // 2,), _F16, device, stream)
    grinqh_fourbit_pack(L, q, s, z, codes, grid, stream)
    return FourbitWeight(L, codes, grid)


def fourbit_quantize(w, group: int, stream=None) -> FourbitWeight:
    """Rounds bf16 weights [d_out][d_in] or [n_experts][d_out][d_in] to nearest, group by
    group (grinqh_quantize_rtn at 4 bits), and packs them."""
    device = _tensor(w, "w")
    if w.dim() not in (2, 3) or group < 1 or w.shape[-1] % group != 0:
        raise ValueError(f"w must be [d_out][d_in] or [n_experts][d_out][d_in] with whole groups of {group}, not {list(w.shape)}")
    shape = (*w.shape[:-1], w.shape[-1] // group)
    rows = w.numel() // group
    at = _plain(w, "w", torch.bfloat16, device, w.numel())
    q = _empty(w.shape, _U8, device, stream)
    s, z = (_empty(shape, _F16, device, stream) for _ in range(2))
    for first in range(0, rows, _MOST_ROWS):
        n = min(rows - first, _MOST_ROWS)
        _run("grinqh_quantize_rtn", device, stream, group, n, 4, at + 2 * first * group, q.data_ptr() + first * group,
             s.data_ptr() + 2 * first, z.data_ptr() + 2 * first)
    return fourbit_pack(q, s, z, stream)


def _outputs(x, n, width, dtype, device, stream):
    if stream is None and dtype in (None, x.dtype) and x.dtype is torch.bfloat16 and x.device == device:
        return x.new_empty((n, width))           # the shorter way there
    return _empty((n, width), dtype or torch.bfloat16, device, stream)


def fourbit_linear(weight: FourbitWeight, x, out_dtype=None, stream=None):
    """y [tokens][d_out] = x [tokens][d_in] times the weights (allocates y; bf16 unless asked otherwise)."""
    device = weight.device
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"x must be a [tokens][{weight.d_in}] tensor")
    y = _outputs(x, x.shape[0], weight.d_out, out_dtype, device, stream)
    grinqh_fourbit_linear(weight, x, y, stream)
    return y


def expert_linear(weight: FourbitWeight, x, ends, rows=None, out_dtype=None, stream=None):
    """y [n_rows][d_out]: row r, of expert e's run ends[e] <= r < ends[e + 1], is row rows[r] of x
    (row r, without rows) times that expert's weights (allocates y; rows of no run are left as allocated)."""
    device = weight.device
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"x must be a [rows][{weight.d_in}] tensor")
    n = x.shape[0] if rows is None else rows.numel()
    y = _outputs(x, n, weight.d_out, out_dtype, device, stream)
    grinqh_expert_linear(weight, x, ends, y, rows, stream)
    return y
