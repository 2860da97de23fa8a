"""Plain fp64 CPU oracle of the key-value cache and the attention calls.

TEST INFRASTRUCTURE ONLY, like grinqh_oracle.py: the library never calls it
and it never calls the library.

* Cache rows.  A row of head_dim values is quantised as a row of weights is
  (grinqh_oracle.quantize_rtn: min / max grid of interval midpoints, fp16 scale
  and zero point, every rounding decision in fp32); at 16 bits it is bf16.  At
  4 bits byte i holds values 2i (low half) and 2i + 1.  Pools are
  [page][head][token of the page][...]; slot = page * page_size + token.
* Attention.  o = sum_t p_t v_t, p = softmax of scale * q . k_t over the tokens
  that are seen; a query that sees none gets zeros and lse = -inf.
"""

from __future__ import annotations

import numpy as np

from . import grinqh_oracle as O


def bf16(x) -> np.ndarray:
    """Values of x rounded to bf16, as fp32."""
    return (O.round_to_bf16(np.asarray(x, np.float32)).astype(np.uint32) << 16).view(np.float32)


def quantise_rows(w, bits: int):
    """w [..., D] fp32 -> (stored bytes uint8 [..., D * bits / 8], grid fp16 [..., 2] or None)."""
    w = np.asarray(w, np.float32)
    D = w.shape[-1]
    if bits == 16:
        return np.ascontiguousarray(O.round_to_bf16(w)).view(np.uint8).reshape(*w.shape[:-1], 2 * D), None
    q, s, z = O.quantize_rtn(w.reshape(-1, D), bits)
    q = q.reshape(w.shape)
    grid = np.stack([s, z], -1).reshape(*w.shape[:-1], 2)
    if bits == 4:
        q = q[..., 0::2] | (q[..., 1::2] << 4)
    return q.astype(np.uint8), grid


def codes_of(stored, bits: int) -> np.ndarray:
    """Integer codes of stored rows (4 or 8 bits)."""
    if bits == 8:
        return stored.astype(np.int64)
    out = np.empty(stored.shape[:-1] + (2 * stored.shape[-1],), np.int64)
    out[..., 0::2] = stored & 15
    out[..., 1::2] = stored >> 4
    return out


def row_values(stored, grid, bits: int) -> np.ndarray:
    """fp64 values of stored rows."""
    if bits == 16:
        u = np.ascontiguousarray(stored).view(np.uint16).astype(np.uint32) << 16
        return u.view(np.float32).astype(np.float64)
    g = np.asarray(grid, np.float64)
    return g[..., :1] * (codes_of(stored, bits) + 0.5) + g[..., 1:]


def row_index(slot: int, head: int, n_kv_heads: int, page_size: int, n_pages: int) -> int:
    """Row of a slot and head, -1 outside the pool (Python integers)."""
    if slot < 0 or slot >= n_pages * page_size:
        return -1
    page, t = divmod(slot, page_size)
    return (page * n_kv_heads + head) * page_size + t


def attend(q, k, v, scale: float, seen=None):
    """One head: q [n][D], k, v [m][D], seen bool [n][m] or None (all).
    Returns o [n][D], lse [n] and p [n][m]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    a = scale * (q @ k.T)
    seen = np.ones(a.shape, bool) if seen is None else seen
    a = np.where(seen, a, -np.inf)
    top = a.max(1, keepdims=True) if a.shape[1] else np.full((len(q), 1), -np.inf)
    e = np.where(seen, np.exp(a - np.where(np.isneginf(top), 0.0, top)), 0.0)
    total = e.sum(1, keepdims=True)
    p = e / np.where(total == 0, 1.0, total)
    with np.errstate(divide="ignore"):
        lse = np.where(total[:, 0] == 0, -np.inf, np.log(total[:, 0]) + np.where(np.isneginf(top), 0.0, top)[:, 0])
    rows = np.nonzero(seen.any(0))[0]                    # what no query sees has no effect, NaN or not
    return p[:, rows] @ v[rows], lse, p


def causal_mask(n: int, m: int) -> np.ndarray:
    """Query i of n sees keys 0 .. i + m - n of m."""
    return np.arange(m)[None, :] <= np.arange(n)[:, None] + (m - n)
