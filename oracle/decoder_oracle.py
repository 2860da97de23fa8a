"""Plain fp64 CPU oracle of the products with 4-bit weights, of the norms and the
rotation of queries and keys, and of the cache's page plan.

TEST INFRASTRUCTURE ONLY, like grinqh_oracle.py: the library never calls it
and it never calls the library.
"""

from __future__ import annotations

import numpy as np


# -------------------------------------------------------- 4-bit weights --

def weights(q, s, z, group: int) -> np.ndarray:
    """fp64 [..., d_out][d_in] of codes, scales and zero points: s * (q + 1/2) + z."""
    s, z = (np.repeat(np.asarray(v, np.float64), group, -1) for v in (s, z))
    return s * ((np.asarray(q, np.int64) & 15) + 0.5) + z


def packed_codes(q) -> np.ndarray:
    """uint32 [E][row_tiles][k_tiles][64][4] of codes [E][d_out][d_in], value by value."""
    q = np.asarray(q, np.int64) & 15
    E, d_out, d_in = q.shape
    rt, kt = -(-d_out // 16), -(-d_in // 128)
    full = np.zeros((E, rt * 16, kt * 128), np.int64)
    full[:, :d_out, :d_in] = q
    words = np.zeros((E, rt, kt, 64, 4), np.uint32)
    for lane in range(64):
        c, r = divmod(lane, 16)
        for m in range(4):
            for e in range(8):
                at = (3 + 4 * (e // 2) + 16 * (e % 2)) % 32
                code = full[:, r::16, 32 * m + 8 * c + e::128].astype(np.uint64)          # [E][rt][kt]
                two = code << np.uint64(at)
                words[:, :, :, lane, m] |= (two | two >> np.uint64(32)).astype(np.uint32)  # the four bits may go round
    return words


def packed_grid(s, z, group: int) -> np.ndarray:
    """fp16 [E][row_tiles][k_tiles * 128 / group][16][2] of [E][d_out][groups]."""
    E, d_out, groups = s.shape
    rt, padded = -(-d_out // 16), -(-groups * group // 128) * (128 // group)
    out = np.zeros((E, rt, padded, 16, 2), np.float16)
    for j in range(d_out):
        out[:, j // 16, :groups, j % 16, 0] = s[:, j]
        out[:, j // 16, :groups, j % 16, 1] = z[:, j]
    return out


def linear(x, q, s, z, group: int):
    """y [n][d_out] of x [n][d_in], and the sum of the magnitudes that fp32 sums go through."""
    x = np.asarray(x, np.float64)
    s64, z64 = (np.repeat(np.asarray(v, np.float64), group, -1) for v in (s, z))
    codes = np.asarray(q, np.int64) & 15
    size = np.abs(s64) * (16 + codes) + np.abs(z64 - 15.5 * s64)
    with np.errstate(invalid="ignore"):
        return x @ weights(q, s, z, group).T, np.abs(x) @ size.T


def experts(x, ends, rows, n_rows: int, q, s, z, group: int):
    """(y, sizes, written) of rows grouped by expert; rows of no run are not written."""
    d_out = q.shape[1]
    y, size, written = np.zeros((n_rows, d_out)), np.zeros((n_rows, d_out)), np.zeros(n_rows, bool)
    ends = np.clip(ends, 0, n_rows)
    src = np.arange(n_rows) if rows is None else np.asarray(rows)
    real = (src >= 0) & (src < len(x))
    taken = np.where(real[:, None], np.asarray(x, np.float64)[np.where(real, src, 0)], 0.0)
    for e in range(len(q)):
        a, b = ends[e], ends[e + 1]
        if a < b:
            y[a:b], size[a:b] = linear(taken[a:b], q[e], s[e], z[e], group)
            written[a:b] = True
    return y, size, written


# ------------------------------------------------------- norm and rotation --

def rope(x, positions, freqs, weight=None, eps: float = 0.0, neighbours: bool = False):
    """(y, sizes) of x [tokens][heads][D]: |a| + |b| of the pair that an output comes from."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = len(freqs)
    y, size = x.copy(), np.abs(x)
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if neighbours else (p, p + half)
        angle = np.asarray(positions, np.float64) * freqs[p]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        size[..., i] = size[..., j] = np.abs(a) + np.abs(b)
    return y, size


# -------------------------------------------------------------------- pages --

def extend(table, lens, new, free, n_free: int, page: int, capacity: int):
    """One step, sequence after sequence, in Python integers.  Returns a dict of
    what the library writes; table is copied."""
    table = np.array(table, np.int64)
    batch, columns = table.shape
    n_pages = len(free)
    n_free = min(max(n_free, 0), n_pages)
    slots, positions = np.full(capacity, -1, np.int64), np.zeros(capacity, np.int64)
    out_lens, cu_q, cu_k = [], [0], [0]
    wanted_pages = taken = refused = 0
    for b in range(batch):
        old, fresh = max(int(lens[b]), 0), max(int(new[b]), 0)
        held, total = -(-old // page), -(-(old + fresh) // page)
        possible = total <= columns and total - held <= n_pages          # by some step, if not by this one
        wanted_pages += total - held if possible else 0
        begin = cu_q[-1]
        granted = fresh == 0 or (possible and wanted_pages <= n_free and begin + fresh <= capacity)
        if granted:
            for i in range(held, total):
                table[b, i] = free[n_free - 1 - taken]
                taken += 1
        else:
            refused += 1
        for t in range(begin, min(begin + fresh, capacity)):
            at = old + t - begin
            positions[t] = min(at, 2 ** 31 - 1)
            if granted and 0 <= table[b, at // page] < n_pages:
                slots[t] = table[b, at // page] * page + at % page
        cu_q.append(begin + fresh)
        out_lens.append(old + fresh if granted else old)
        cu_k.append(cu_k[-1] + out_lens[-1])
    top = 2 ** 31 - 1
    return {"table": table, "slots": slots, "positions": positions, "seq_lens": np.minimum(np.array(out_lens, np.int64), top),
            "cu_q": np.minimum(cu_q, top), "cu_k": np.minimum(cu_k, top), "n_free": n_free - taken, "refused": refused}


def release(table, lens, finished, free, n_free: int, page: int):
    """(table, lens, free, n_free) after the finished sequences' pages are given back."""
    table, lens, free = np.array(table, np.int64), np.array(lens, np.int64), np.array(free, np.int64)
    n_pages = len(free)
    n_free = min(max(n_free, 0), n_pages)
    for b in range(len(lens)):
        if finished[b]:
            for i in range(min(-(-max(int(lens[b]), 0) // page), table.shape[1])):
                if 0 <= table[b, i] < n_pages:
                    if n_free < n_pages:
                        free[n_free] = table[b, i]
                        n_free += 1
                table[b, i] = -1
            lens[b] = 0
    return table, lens, free, n_free
