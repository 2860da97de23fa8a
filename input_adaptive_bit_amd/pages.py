"""Python binding of grinqh_kv_extend and grinqh_kv_release: the pages of a
batch's sequences, handed out and taken back on the GPU (include/grinqh.h)."""

from __future__ import annotations

import ctypes
from typing import NamedTuple

try:
    import torch
except ImportError:                              # the host call below needs no torch
    torch = None

from .attention import _empty, _fit, _plain, _run, _tensor
from .grinqh import GRINQH_EINVAL, ExtendArgs, GrinqhError, load

if torch is not None:
    _I32, _I64, _U8 = torch.int32, torch.int64, torch.uint8


class Step(NamedTuple):
    """What the calls of a step take: slots and positions of its new tokens (packed, padded), the ends of the packed
    sequences, the new lengths, the number of unused pages, and how many sequences were refused."""
    slots: "torch.Tensor"
    positions: "torch.Tensor"
    cu_q: "torch.Tensor"
    cu_k: "torch.Tensor"
    seq_lens: "torch.Tensor"
    n_free: "torch.Tensor"
    refused: "torch.Tensor"


def grinqh_kv_extend_workspace_bytes(batch: int) -> int:
    return int(load().grinqh_kv_extend_workspace_bytes(_fit(batch)))


def _table(t, batch, device):
    """(address, row stride, columns) of an int32 [batch][max_pages] table whose rows are contiguous."""
    _tensor(t, "page_table", device)
    if t.dtype != _I32 or t.dim() != 2 or t.shape[0] != batch:
        raise ValueError(f"page_table must be int32 [{batch}][max_pages]")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("the rows of page_table must be contiguous")
    if batch > 1 and t.stride(0) < t.shape[1]:
        raise ValueError("the rows of page_table must not overlap")
    return t.data_ptr(), t.stride(0) if batch > 1 else t.shape[1], t.shape[1]


def _plan(page_table, seq_lens, n_new, free_pages, n_free):
    """(device, batch, columns, the leading fields of ExtendArgs) of the tensors that a plan reads."""
    try:
        device, (batch,) = seq_lens.device, seq_lens.shape
        index, (rows, columns), (stride, s1) = device.index, page_table.shape, page_table.stride()
        fits = (rows == batch and (s1 == 1 or columns < 2) and (batch < 2 or stride >= columns) and n_new.numel() == batch
                and page_table.dtype is seq_lens.dtype is n_new.dtype is free_pages.dtype is n_free.dtype is _I32
                and page_table.get_device() == n_new.get_device() == free_pages.get_device() == n_free.get_device() == index
                and seq_lens.is_contiguous() and n_new.is_contiguous() and free_pages.is_contiguous() and n_free.is_contiguous()
                and seq_lens.is_cuda and free_pages.numel() >= 1 and n_free.numel() >= 1)
    except (AttributeError, TypeError, ValueError):
        fits = False
    if fits:
        return device, batch, columns, (page_table.data_ptr(), stride if batch > 1 else columns, seq_lens.data_ptr(),
                                        n_new.data_ptr(), free_pages.data_ptr(), n_free.data_ptr())
    device = _tensor(seq_lens, "seq_lens")                    # one by one, to say what does not
    batch = seq_lens.numel()
    _tensor(n_new, "n_new", device)
    if n_new.numel() != batch:
        raise ValueError("n_new must be as long as seq_lens")
    table, stride, columns = _table(page_table, batch, device)
    return device, batch, columns, (table, stride, *(_plain(t, name, _I32, device, count) for name, t, count in (
        ("seq_lens", seq_lens, batch), ("n_new", n_new, batch), ("free_pages", free_pages, 1), ("n_free", n_free, 1))))


def grinqh_kv_extend(page_table, seq_lens, n_new, free_pages, n_free, page_size: int, step: Step, workspace,
                     stream=None) -> None:
    """page_table: int32 [batch][max_pages]; seq_lens, n_new: int32 [batch]; free_pages: int32 [n_pages];
    n_free: int32 [1]; step: the tensors to write (step.seq_lens and step.n_free may be seq_lens and n_free)."""
    device, batch, columns, inputs = _plan(page_table, seq_lens, n_new, free_pages, n_free)
    room = step.slots.numel()
    if step.positions.numel() != room:
        raise ValueError("step.positions must be as long as step.slots")
    _tensor(workspace, "workspace", device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    lens, left, refused, cu_q, cu_k, positions = (_plain(t, name, _I32, device, count) for name, t, count in (
        ("step.seq_lens", step.seq_lens, batch), ("step.n_free", step.n_free, 1), ("step.refused", step.refused, 1),
        ("step.cu_q", step.cu_q, batch + 1), ("step.cu_k", step.cu_k, batch + 1), ("step.positions", step.positions, room)))
    a = ExtendArgs(*inputs, _fit(batch), _fit(columns), _fit(page_size), _fit(free_pages.numel()), _fit(room), lens, left, refused, cu_q, cu_k,
                   _plain(step.slots, "step.slots", _I64, device, room), positions, workspace.data_ptr(), workspace.nbytes)
    _run("grinqh_kv_extend", device, stream, ctypes.byref(a))


def grinqh_kv_release(page_table, seq_lens, finished, free_pages, n_free, page_size: int, stream=None) -> None:
    """finished: uint8 or bool [batch]; the others as grinqh_kv_extend takes them, all written in place."""
    device = _tensor(seq_lens, "seq_lens")
    batch = seq_lens.numel()
    table, stride, columns = _table(page_table, batch, device)
    _tensor(finished, "finished", device)
    if finished.dtype not in (_U8, torch.bool) or finished.numel() != batch:
        raise ValueError(f"finished must be uint8 or bool [{batch}]")
    _run("grinqh_kv_release", device, stream, table, stride, _plain(seq_lens, "seq_lens", _I32, device, batch),
         _plain(finished, "finished", finished.dtype, device, batch), _fit(batch), columns, _fit(page_size),
         _plain(free_pages, "free_pages", _I32, device, 1), _plain(n_free, "n_free", _I32, device, 1), _fit(free_pages.numel()))


# ------------------------------------------------- allocating conveniences --

def new_page_list(n_pages: int, device=None):
    """(free_pages int32 [n_pages], n_free int32 [1]) of a pool whose pages are all unused; page 0 is handed out first."""
    if not 1 <= n_pages <= 1 << 24:
        raise GrinqhError(GRINQH_EINVAL, "new_page_list")
    device = device or "cuda"
    return torch.arange(n_pages - 1, -1, -1, dtype=_I32, device=device), torch.full((1,), n_pages, dtype=_I32, device=device)


def kv_extend(page_table, seq_lens, n_new, free_pages, n_free, page_size: int, capacity: int, in_place: bool = False,
              stream=None) -> Step:
    """Pages for n_new[b] tokens behind the seq_lens[b] cached ones of every sequence: writes the new pages into
    page_table and returns what the step's other calls take (allocates it; slots and positions hold `capacity` tokens).
    With in_place, seq_lens and n_free themselves are updated."""
    device, batch, columns, inputs = _plan(page_table, seq_lens, n_new, free_pages, n_free)
    if not 0 <= capacity <= 1 << 24:
        raise GrinqhError(GRINQH_EINVAL, "grinqh_kv_extend")
    # One allocation: slots (8 bytes each), what is 4 bytes wide, then the workspace (8 bytes a sequence and 16, on 16 bytes).
    # The call needs addresses only, and the library refuses every count that the types could not hold.
    kept = 0 if in_place else batch
    before = 3 * capacity + 2 * batch + kept + (3 if in_place else 4)
    ws = -before % 4 + 2 * batch + 4
    both = _empty((before + ws,), _I32, device, stream)
    slots, positions, cu_q, cu_k, lens, left, refused, _ = both.split_with_sizes(
        (2 * capacity, capacity, batch + 1, batch + 1, kept, 0 if in_place else 1, 1, ws))
    start = both.data_ptr()
    to_positions = start + 8 * capacity
    to_q = to_positions + 4 * capacity
    to_k = to_q + 4 * batch + 4
    to_lens = to_k + 4 * batch + 4
    to_left = to_lens + 4 * kept
    space = start + 4 * (before + -before % 4)
    if in_place:
        lens, left, to_lens, to_left, to_refused = seq_lens, n_free, inputs[2], inputs[5], to_left
    else:
        to_refused = to_left + 4
    a = ExtendArgs(*inputs, _fit(batch), _fit(columns), _fit(page_size), _fit(free_pages.numel()), capacity, to_lens, to_left,
                   to_refused, to_q, to_k, start, to_positions, space, 8 * batch + 16)
    _run("grinqh_kv_extend", device, stream, ctypes.byref(a))
    return Step(slots.view(_I64), positions, cu_q, cu_k, lens, left, refused)


def kv_release(page_table, seq_lens, finished, free_pages, n_free, page_size: int, stream=None) -> None:
    """Give the finished sequences' pages back (grinqh_kv_release)."""
    grinqh_kv_release(page_table, seq_lens, finished, free_pages, n_free, page_size, stream)
