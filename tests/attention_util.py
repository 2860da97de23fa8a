"""Inputs, device copies and error bounds for the cache and attention tests.

Bounds.  u = 2^-24 is half a step of fp32, 2^-8 of bf16.  With e_a the largest
error of a score, every weight p_t is off by at most a relative 2 e_a (numerator
and sum), so an output by 2 e_a sum p_t |v_t|.  A score is a dot product of D
terms (order unspecified: D u sum |q_d k_d|, the terms of a quantised key being
q_d s (c + 1/2) and q_d z), a few fp32 roundings of its parts and of the
exponent's argument (8 u (|a| + the same sum)).  The sum over m tokens adds m u
sum p_t |v_t|.  A weight that is rounded before its product with a value adds
that rounding's relative error, the output type its own.
"""

from __future__ import annotations

import numpy as np

from oracle import attention_oracle as A

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
W_PREFILL = 2.0 ** -8     # weights in bf16
W_DECODE = 2.0 ** -16     # weights as a sum of two bf16: the second rounds a remainder of 2^-8


def rows(rng, tokens, heads, dim, strong=0.03):
    """Unit normal rows, a few channels of every head four times as strong, as bf16 values in fp32."""
    x = rng.standard_normal((tokens, heads, dim)).astype(np.float32)
    x *= np.where(rng.random((1, heads, dim)) < strong, 4.0, 1.0).astype(np.float32)
    return A.bf16(x)


def head_bound(q, k_terms, k, v_abs, m, p, scale, weight, out, out_dtype):
    """Elementwise bound of one head's outputs [n][D] and of its lse [n].
    k_terms [m][D]: the largest magnitude of a key's terms; v_abs [m][D]: of a value's."""
    q = np.abs(np.asarray(q, np.float64))
    n_terms = 2 * q.shape[1]
    size = abs(scale) * (q @ np.asarray(k_terms, np.float64).T)                 # [n][m]
    seen = p > 0
    e_a = np.where(seen, (n_terms + 8) * U * size, 0.0).max(1, initial=0.0)     # [n]
    mass = p @ np.asarray(v_abs, np.float64)
    rel = weight + 2 * e_a + (m + 16) * U
    lse = e_a + (m + 16) * U
    return rel[:, None] * mass + HALF[out_dtype] * np.abs(out) + 1e-30, lse


def to_bf16(x, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev).to(torch.bfloat16)


def to_type(x, dtype, dev):
    import torch
    return to_bf16(x, dev) if dtype == "bf16" else torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev)


def inside(got, want, bound, what=""):
    """Every value within its bound; the same NaN."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    both = np.isnan(got) & np.isnan(want)
    same = got == want
    with np.errstate(invalid="ignore"):
        off = np.where(both | same, 0.0, np.abs(got - want))
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                           np.broadcast_to(bound, got.shape)[bad][:4])


class Cache:
    """Host copy of a paged cache beside the device's, filled by the oracle's quantiser."""

    def __init__(self, rng, lens, heads, dim, bits, page, dev, spare=3, fill=0xFF, k=None, v=None):
        import torch

        import input_adaptive_bit_amd as G
        self.lens, self.heads, self.dim, self.bits, self.page = list(lens), heads, dim, bits, page
        most = max(1, max(-(-n // page) for n in lens))
        need = sum(-(-n // page) for n in lens)
        self.n_pages = need + spare
        L = G.grinqh_kv_layout_init(heads, dim, page, self.n_pages, bits)
        shape = (self.n_pages, heads, page)
        self.stored = [np.full(shape + (L.row_bytes,), fill, np.uint8) for _ in range(2)]
        self.grid = [np.full(shape + (2,), np.nan, np.float16) if bits < 16 else None for _ in range(2)]
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), most), -1, np.int32)          # entries past a sequence are never used
        self.values, self.k_rows = [], []
        at = 0
        for b, n in enumerate(lens):
            pages = order[at:at + -(-n // page)]
            at += len(pages)
            self.table[b, :len(pages)] = pages
            kv = [rows(rng, n, heads, dim) if given is None else given[b] for given in (k, v)]
            for which in range(2):
                stored, grid = A.quantise_rows(kv[which], bits)
                for t in range(n):
                    self.stored[which][pages[t // page], :, t % page] = stored[t]
                    if bits < 16:
                        self.grid[which][pages[t // page], :, t % page] = grid[t]
        dev_codes = [torch.from_numpy(x).to(dev) for x in self.stored]
        dev_grid = [torch.from_numpy(x).to(dev) if x is not None else None for x in self.grid]
        self.dev = G.KVCache(L, *dev_codes, *dev_grid)
        self.dev_table = torch.from_numpy(self.table).to(dev)
        self.dev_lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)

    def row(self, b, t):
        page = self.table[b, t // self.page]
        return (page, t % self.page) if 0 <= page < self.n_pages else None

    def gathered(self, b, head, which, length=None):
        """fp64 values [m][D] of a sequence's tokens that exist, and the largest magnitudes of their terms."""
        n = self.lens[b] if length is None else length
        at = [r for r in (self.row(b, t) for t in range(n)) if r is not None]
        if not at:
            return np.zeros((0, self.dim)), np.zeros((0, self.dim))
        stored = np.array([self.stored[which][p, head, t] for p, t in at])
        if self.bits == 16:
            val = A.row_values(stored, None, 16)
            return val, np.abs(val)
        grid = np.array([self.grid[which][p, head, t] for p, t in at], np.float64)
        val, c = A.row_values(stored, grid, self.bits), A.codes_of(stored, self.bits)
        mid = 2.0 ** (self.bits - 1)
        s, z = grid[:, :1], grid[:, 1:]
        # keys: |s c| + |s / 2 + z|; values about the grid's middle: |s (c - mid)| + |z + s (mid + 1/2)|
        if which == 0:
            return val, np.abs(s) * c + np.abs(s / 2 + z)
        return val, np.abs(s) * np.abs(c - mid) + np.abs(z + s * (mid + 0.5))


def decode_reference(cache: Cache, q, scale, out_dtype, lens=None):
    """(o, bound, lse, lse bound) for q [batch][n_q_heads][D]."""
    batch, n_q, dim = q.shape
    group = n_q // cache.heads
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    lse, lse_bound = np.zeros((batch, n_q)), np.zeros((batch, n_q))
    for b in range(batch):
        for g in range(cache.heads):
            n = cache.lens[b] if lens is None else lens[b]
            k, kt = cache.gathered(b, g, 0, n)
            v, vt = cache.gathered(b, g, 1, n)
            h = slice(g * group, (g + 1) * group)
            o[b, h], lse[b, h], p = A.attend(q[b, h], k, v, scale)
            bound[b, h], lse_bound[b, h] = head_bound(q[b, h], kt, k, vt, len(k), p, scale, W_DECODE, o[b, h], out_dtype)
    return o, bound, lse, lse_bound


def prefill_reference(q, k, v, cu_q, cu_k, scale, causal, out_dtype):
    """The same for packed prompts (numpy, bf16 values); rows of no sequence stay 0."""
    n_q, group = q.shape[1], q.shape[1] // k.shape[1]
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    lse, lse_bound = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    for b in range(len(cu_q) - 1):
        a, z, c, d = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        mask = A.causal_mask(z - a, d - c) if causal else np.ones((z - a, d - c), bool)
        for h in range(n_q):
            kk, vv = k[c:d, h // group].astype(np.float64), v[c:d, h // group].astype(np.float64)
            o[a:z, h], lse[a:z, h], p = A.attend(q[a:z, h], kk, vv, scale, mask)
            bound[a:z, h], lse_bound[a:z, h] = head_bound(q[a:z, h], np.abs(kk), kk, np.abs(vv), d - c, p, scale,
                                                          W_PREFILL, o[a:z, h], out_dtype)
    return o, bound, lse, lse_bound
