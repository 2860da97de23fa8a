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


def grinqh_kv_extend(page_table, seq_lens, n_new, free_pages, n_free, page_size: int, step: Step, workspace,
                     stream=None) -> None:
    """page_table: int32 [batch][max_pages]; seq_lens, n_new: int32 [batch]; free_pages: int32 [n_pages];
    n_free: int32 [1]; step: the tensors to write (step.seq_lens and step.n_free may be seq_lens and n_free)."""
    device = _tensor(seq_lens, "seq_lens")
    batch, room = seq_lens.numel(), step.slots.numel()
    if step.positions.numel() != room or n_new.numel() != batch:
        raise ValueError("n_new must be as long as seq_lens, and positions as slots")
    table, stride, columns = _table(page_table, batch, device)
    _tensor(workspace, "workspace", device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    i32 = [_plain(t, name, _I32, device, count) for name, t, count in (
        ("seq_lens", seq_lens, batch), ("n_new", n_new, batch), ("free_pages", free_pages, 1), ("n_free", n_free, 1),
        ("step.seq_lens", step.seq_lens, batch), ("step.n_free", step.n_free, 1), ("step.refused", step.refused, 1),
        ("step.cu_q", step.cu_q, batch + 1), ("step.cu_k", step.cu_k, batch + 1), ("step.positions", step.positions, room))]
    a = ExtendArgs(table, stride, *i32[:4], _fit(batch), columns, _fit(page_size), _fit(free_pages.numel()), _fit(room), *i32[4:9],
                   _plain(step.slots, "step.slots", _I64, device, room), i32[9], workspace.data_ptr(), workspace.nbytes)
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
    device = _tensor(seq_lens, "seq_lens")
    if not 0 <= capacity <= 1 << 24:
        raise GrinqhError(GRINQH_EINVAL, "grinqh_kv_extend")
    batch = seq_lens.numel()
    # one allocation: slots first, the workspace (8 bytes a sequence and 16), then what is 4 bytes wide
    ws = 2 * batch + 4
    tail = 2 * capacity + (2 * capacity & 2)                 # the workspace lies on 16 bytes
    at = tail + ws
    sizes = (capacity, batch + 1, batch + 1, 0 if in_place else batch, 0 if in_place else 1, 1)
    both = _empty((at + sum(sizes),), _I32, device, stream)
    parts = torch.split(both, (2 * capacity, tail - 2 * capacity, ws, *sizes))
    slots, positions, cu_q, cu_k, lens, left, refused = parts[0].view(_I64), *parts[3:]
    step = Step(slots, positions, cu_q, cu_k, seq_lens if in_place else lens, n_free if in_place else left, refused)
    grinqh_kv_extend(page_table, seq_lens, n_new, free_pages, n_free, page_size, step, parts[2], stream)
    return step


def kv_release(page_table, seq_lens, finished, free_pages, n_free, page_size: int, stream=None) -> None:
    """Give the finished sequences' pages back (grinqh_kv_release)."""
    grinqh_kv_release(page_table, seq_lens, finished, free_pages, n_free, page_size, stream)
