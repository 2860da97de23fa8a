"""The cache's and attention's oracle, addressing, host checks and binding
refusals; no GPU (every library call here is host arithmetic or fails a host
check, so no kernel is launched)."""

import ctypes

import numpy as np
import pytest

import input_adaptive_bit_amd as G
from input_adaptive_bit_amd import grinqh as B
from oracle import attention_oracle as A

K64 = 1 << 16


# --------------------------------------------------------------- the oracle --

@pytest.mark.parametrize("bits", [4, 8])
def test_cached_rows_are_the_nearest_midpoints(bits):
    """Each value reads back as the midpoint of its interval: within half a
    step of it, up to the grid's own rounding to fp16."""
    rng = np.random.default_rng(bits)
    w = rng.standard_normal((50, 64)).astype(np.float32)
    stored, grid = A.quantise_rows(w, bits)
    assert stored.shape == (50, 64 * bits // 8)
    s = grid[:, :1].astype(np.float64)
    lo, hi = w.min(1, keepdims=True).astype(np.float64), w.max(1, keepdims=True).astype(np.float64)
    # half a step; z off by 2^-11 |lo|; s by 2^-11 s over 2^bits steps
    slack = np.abs(lo) * 2.0 ** -11 + (hi - lo) * 2.0 ** -11
    assert np.all(np.abs(A.row_values(stored, grid, bits) - w) <= s / 2 + slack)


def test_four_bit_rows_hold_even_values_in_the_low_half():
    w = np.arange(16, dtype=np.float32)[None] + 0.5
    w[0, 0], w[0, 15] = 0.0, 16.0
    stored, grid = A.quantise_rows(w, 4)
    assert grid.tolist() == [[1.0, 0.0]]
    assert stored[0].tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert A.codes_of(stored, 4)[0].tolist() == list(range(16))


def test_sixteen_bit_rows_are_bf16():
    w = np.array([[1.0, 1.00390625, -2.5, 3.0e38]], np.float32)
    stored, grid = A.quantise_rows(w, 16)
    assert grid is None and A.row_values(stored, None, 16)[0, :3].tolist() == [1.0, 1.0, -2.5]


def test_attention_of_equal_scores_is_the_mean_and_of_one_token_its_value():
    v = np.arange(12.0).reshape(4, 3)
    o, lse, p = A.attend(np.zeros((2, 3)), np.ones((4, 3)), v, 1.0)
    assert np.allclose(o, v.mean(0)) and np.allclose(lse, np.log(4)) and np.allclose(p, 0.25)
    o, lse, _ = A.attend([[2.0]], [[3.0]], [[7.0]], 0.5)
    assert o[0, 0] == 7.0 and lse[0] == 3.0


def test_attention_matches_the_weighted_sum_written_out():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 5)), rng.standard_normal((6, 5)), rng.standard_normal((6, 5))
    seen = A.causal_mask(3, 6)
    o, lse, _ = A.attend(q, k, v, 0.7, seen)
    for i in range(3):
        w = [np.exp(0.7 * sum(q[i] * k[j])) for j in range(6) if j <= i + 3]
        want = sum(x * v[j] for j, x in enumerate(w)) / sum(w)
        assert np.allclose(o[i], want) and np.isclose(lse[i], np.log(sum(w)))


def test_causal_mask_ends_at_the_last_key_and_leaves_rows_empty():
    assert A.causal_mask(2, 4).tolist() == [[True, True, True, False], [True] * 4]
    assert A.causal_mask(3, 1).tolist() == [[False], [False], [True]]
    o, lse, _ = A.attend(np.ones((3, 2)), np.full((1, 2), np.nan), np.full((1, 2), np.nan), 1.0, np.zeros((3, 1), bool))
    assert np.all(o == 0) and np.all(np.isneginf(lse))


# --------------------------------------------------------------- addressing --

@pytest.mark.parametrize("heads,page,n_pages", [(1, 16, 1), (8, 64, 1000), (5, 256, 1 << 24), (1024, 128, 70000)])
def test_rows_of_slots(heads, page, n_pages):
    """The row the kernels use, and -1 for every slot outside the pool; pools
    of more than 2^32 rows among them."""
    L = G.grinqh_kv_layout_init(heads, 128, page, n_pages, 8)
    total = page * n_pages
    rng = np.random.default_rng(page)
    slots = [0, 1, page - 1, page, total - 1, total, total + 1, -1, -page, 2 ** 62, -2 ** 63, 2 ** 32, 2 ** 31 - 1]
    slots += [int(x) for x in rng.integers(0, total, 200)]
    for slot in slots:
        for head in {0, heads // 2, heads - 1}:
            want = A.row_index(slot, head, heads, page, n_pages)
            assert G.grinqh_debug_kv_row(L, slot, head) == want
            assert -1 <= want < heads * total
    assert G.grinqh_debug_kv_row(L, 0, -1) == -1 and G.grinqh_debug_kv_row(L, 0, heads) == -1
    rows = [G.grinqh_debug_kv_row(L, s, h) for s in range(min(total, 40)) for h in range(min(heads, 9))]
    assert len(set(rows)) == len(rows)


@pytest.mark.parametrize("heads,page,n_pages", [(1, 16, 1), (8, 64, 1000), (5, 256, 1 << 24)])
def test_rows_of_page_table_entries(heads, page, n_pages):
    """An entry of the pool gives its token's row; any other entry a row that
    lies in the pool, marked as not to be used."""
    L = G.grinqh_kv_layout_init(heads, 128, page, n_pages, 8)
    for entry in (0, 1, n_pages - 1, n_pages, n_pages + 7, -1, -2 ** 31, 2 ** 31 - 1):
        for head in {0, heads - 1}:
            for t in (0, 15, page - 1, page, 5 * page + 3, 2 ** 28 - 1):
                got = G.grinqh_debug_page_row(L, entry, head, t)
                if 0 <= entry < n_pages:
                    assert got == A.row_index(entry * page + t % page, head, heads, page, n_pages)
                else:
                    assert 0 <= -1 - got < heads * page * n_pages
    assert G.grinqh_debug_page_row(L, 0, heads, 0) == -1 and G.grinqh_debug_page_row(L, 0, 0, -1) == -1


def test_layout_sizes():
    L = G.grinqh_kv_layout_init(8, 128, 64, 10, 4)
    assert (L.row_bytes, G.grinqh_kv_code_bytes(L), G.grinqh_kv_grid_bytes(L)) == (64, 10 * 8 * 64 * 64, 10 * 8 * 64 * 4)
    L = G.grinqh_kv_layout_init(1, 256, 16, 1 << 24, 16)
    assert (L.row_bytes, G.grinqh_kv_code_bytes(L), G.grinqh_kv_grid_bytes(L)) == (512, (1 << 28) * 512, 0)
    bad = B.KVLayout(8, 128, 64, 10, 4, 63)
    assert G.grinqh_kv_code_bytes(bad) == 0 and G.grinqh_kv_grid_bytes(bad) == 0
    assert G.grinqh_debug_kv_row(bad, 0, 0) == -1


@pytest.mark.parametrize("bad", [(0, 128, 64, 1, 8), (1025, 128, 64, 1, 8), (1, 96, 64, 1, 8), (1, 0, 64, 1, 8),
                                 (1, 128, 8, 1, 8), (1, 128, 48, 1, 8), (1, 128, 512, 1, 8), (1, 128, 64, 0, 8),
                                 (1, 128, 64, (1 << 24) + 1, 8), (1, 128, 64, 1, 2), (1, 128, 64, 1, 32),
                                 (1, 1 << 30, 64, 1, 8), (1, 128, 64, 1, -8)])
def test_layouts_outside_the_ranges_are_refused(bad):
    with pytest.raises(G.GrinqhError):
        G.grinqh_kv_layout_init(*bad)
    assert B.load().grinqh_kv_layout_init(1, 128, 64, 1, 8, None) == B.GRINQH_EINVAL


# -------------------------------------------------------------- host checks --

def _pools(a=16):
    return B.KVPools(a * K64 * 16, (a + 16) * K64 * 16, (a + 32) * K64 * 16, (a + 48) * K64 * 16)


def test_cache_calls_check_their_arguments_before_any_device_call():
    lib = G.load()
    L = G.grinqh_kv_layout_init(2, 64, 16, 8, 8)
    P = _pools()
    K, V, S = K64, 2 * K64, 3 * K64

    def write(L=L, P=P, k=K, v=V, dt=0, ks=128, vs=128, n=4, s=S):
        return lib.grinqh_kv_write(None if L is None else ctypes.byref(L), None if P is None else ctypes.byref(P), k, v,
                                   dt, ks, vs, n, s, None)

    def read(L=L, P=P, k=K, v=V, dt=0, n=4, s=S):
        return lib.grinqh_kv_read(None if L is None else ctypes.byref(L), None if P is None else ctypes.byref(P), s, n,
                                  k, v, dt, None)

    for call in (write, read):
        for key in ("L", "P", "k", "v", "s"):
            assert call(**{key: None}) == B.GRINQH_EINVAL, key
        assert call(dt=2) == B.GRINQH_EINVAL
        assert call(n=-1) == B.GRINQH_EINVAL and call(n=(1 << 24) + 1) == B.GRINQH_EINVAL
        assert call(n=0) == B.GRINQH_OK                       # nothing to do, nothing launched
        assert call(k=K + 8) == B.GRINQH_EALIGN and call(v=V + 2) == B.GRINQH_EALIGN
        assert call(s=S + 4) == B.GRINQH_EALIGN
        for field in ("k_codes", "v_codes", "k_grid", "v_grid"):
            for value, status in ((None, B.GRINQH_EINVAL), (getattr(P, field) + 8, B.GRINQH_EALIGN)):
                bad = B.KVPools(P.k_codes, P.v_codes, P.k_grid, P.v_grid)
                setattr(bad, field, value)
                assert call(P=bad) == status, field
            assert call(k=getattr(P, field) + 64) == B.GRINQH_EINVAL, field      # overlaps the pool
            assert call(v=getattr(P, field) + 64) == B.GRINQH_EINVAL, field
        assert call(L=B.KVLayout(2, 64, 16, 8, 8, 63)) == B.GRINQH_EINVAL
    for key in ("ks", "vs"):
        assert write(**{key: 127}) == B.GRINQH_EINVAL                             # tokens would overlap
        assert write(**{key: 132}) == B.GRINQH_EALIGN
        assert write(**{key: (1 << 24) + 8}) == B.GRINQH_EINVAL
        assert write(dt=1, **{key: 130}) == B.GRINQH_EALIGN
    assert read(v=K + 512) == B.GRINQH_EINVAL                                     # outputs overlap


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_rows_are_not_written_to_pools_that_share_memory(bits):
    """Keys and values are written at the same time: one buffer for both, or pools that overlap, would mix them."""
    lib = G.load()
    L = G.grinqh_kv_layout_init(2, 64, 16, 8, bits)
    apart, codes, grid = _pools(), G.grinqh_kv_code_bytes(L), G.grinqh_kv_grid_bytes(L)
    sizes = dict(k_codes=codes, v_codes=codes, k_grid=grid, v_grid=grid)
    for one in sizes:
        for other in sizes:
            for at in (0, -sizes[one] + 16, sizes[other] - 16):
                if one != other and sizes[one] and sizes[other]:
                    P = B.KVPools(apart.k_codes, apart.v_codes, apart.k_grid, apart.v_grid)
                    setattr(P, one, getattr(P, other) + at)
                    assert lib.grinqh_kv_write(ctypes.byref(L), ctypes.byref(P), K64, 2 * K64, 0, 128, 128, 4, 3 * K64,
                                               None) == B.GRINQH_EINVAL, (one, other, at)


@pytest.mark.parametrize("bits", [4, 16])
def test_slots_must_not_lie_where_rows_are_stored(bits):
    """In a pool that kv_write fills, in an output of kv_read."""
    lib = G.load()
    L = G.grinqh_kv_layout_init(2, 64, 16, 8, bits)
    P = _pools()
    codes, grid = G.grinqh_kv_code_bytes(L), G.grinqh_kv_grid_bytes(L)
    for field, size in (("k_codes", codes), ("v_codes", codes), ("k_grid", grid), ("v_grid", grid)):
        for at in (0, -24, size - 8):
            if size:
                assert lib.grinqh_kv_write(ctypes.byref(L), ctypes.byref(P), K64, 2 * K64, 0, 128, 128, 4,
                                           getattr(P, field) + at, None) == B.GRINQH_EINVAL, (field, at)
    for out in (K64, 2 * K64):
        for at in (0, -24, 4 * 128 * 2 - 8):
            assert lib.grinqh_kv_read(ctypes.byref(L), ctypes.byref(P), out + at, 4, K64, 2 * K64, 0, None) == B.GRINQH_EINVAL


def test_decode_attention_checks_its_arguments_before_any_device_call():
    lib = G.load()
    L = G.grinqh_kv_layout_init(2, 64, 16, 8, 8)
    P = _pools()
    Q, T, N, OUT, LSE, WS = (K64 * k for k in range(1, 7))

    def call(L=L, P=P, q=Q, qd=0, qs=8 * 64, nq=8, t=T, ts=4, mp=4, n=N, b=3, ml=64, sc=0.1, o=OUT, od=0, lse=LSE,
             ws=WS, wsb=1 << 40):
        return lib.grinqh_decode_attention(None if L is None else ctypes.byref(L), None if P is None else ctypes.byref(P),
                                           q, qd, qs, nq, t, ts, mp, n, b, ml, sc, o, od, lse, ws, wsb, None)

    for key in ("L", "P", "q", "t", "n", "o", "ws"):
        assert call(**{key: None}) == B.GRINQH_EINVAL, key
    for key, value in (("qd", 3), ("od", -1), ("nq", 7), ("nq", 0), ("nq", 1026), ("mp", 0), ("ts", 3), ("b", -1),
                       ("b", (1 << 20) + 1), ("ml", 0), ("ml", (1 << 28) + 1), ("sc", float("nan")),
                       ("sc", float("inf")), ("sc", -2e30), ("qs", 8 * 64 - 8), ("qs", (1 << 24) + 8), ("o", Q + 64)):
        assert call(**{key: value}) == B.GRINQH_EINVAL, (key, value)
    for key, value in (("q", Q + 8), ("qs", 8 * 64 + 4), ("t", T + 2), ("n", N + 1), ("o", OUT + 8), ("lse", LSE + 2),
                       ("ws", WS + 64)):
        assert call(**{key: value}) == B.GRINQH_EALIGN, (key, value)
    assert call(wsb=0) == B.GRINQH_ENOSPACE
    assert call(b=0) == B.GRINQH_OK
    for bad in (dict(n_q_heads=7), dict(batch=-1), dict(max_len=0), dict(L=B.KVLayout(2, 64, 16, 8, 8, 60))):
        a = dict(dict(L=L, n_q_heads=8, batch=3, max_len=64), **bad)
        assert G.grinqh_attention_workspace_bytes(**a) == 0
    assert G.grinqh_attention_workspace_bytes(L, 8, 3, 64) % 256 == 0


@pytest.mark.parametrize("bits", [4, 16])
def test_decode_attention_refuses_to_write_where_it_reads(bits):
    """out, lse and the workspace against q, the page table, the lengths, the pools and one another, at both ends."""
    lib = G.load()
    L = G.grinqh_kv_layout_init(2, 64, 16, 8, bits)
    ws = G.grinqh_attention_workspace_bytes(L, 8, 3, 64)
    sizes = dict(q=3 * 512 * 2, t=(2 * 6 + 4) * 4, n=12, out=3 * 512 * 4, lse=3 * 8 * 4, ws=ws, k=G.grinqh_kv_code_bytes(L),
                 v=G.grinqh_kv_code_bytes(L), kg=G.grinqh_kv_grid_bytes(L), vg=G.grinqh_kv_grid_bytes(L))
    good = {name: (i + 1) << 24 for i, name in enumerate(sizes)}

    def status(**at):
        a = dict(good, **at)
        P = B.KVPools(a["k"], a["v"], a["kg"], a["vg"])
        return lib.grinqh_decode_attention(ctypes.byref(L), ctypes.byref(P), a["q"], 0, 512, 8, a["t"], 6, 4, a["n"], 3, 64,
                                           0.1, a["out"], 1, a["lse"], a["ws"], ws, None)

    for written in ("out", "lse", "ws"):
        for other in sizes:
            if other == written or not sizes[other]:
                continue
            step = {"out": 16, "lse": 4, "ws": 256}[written]
            below = (sizes[written] - 1) // step * step
            for at in (0, -below, (sizes[other] - 1) // step * step):
                assert status(**{written: good[other] + at}) == B.GRINQH_EINVAL, (written, other, at)


@pytest.mark.parametrize("heads,dim,bits,n_q", [(8, 128, 8, 32), (8, 128, 4, 64), (1, 256, 16, 16), (2, 64, 4, 6), (4, 128, 8, 96),
                                                (12, 64, 16, 12), (48, 64, 8, 48)])
def test_decode_workspace_of_a_programs_largest_call_serves_its_smaller_ones(heads, dim, bits, n_q):
    """The size never falls as batch or length grow, and a call takes a workspace of the size asked for any larger one.
    (q and out overlap, which is refused after the workspace was found large enough: nothing is launched.)"""
    lib = G.load()
    L = G.grinqh_kv_layout_init(heads, dim, 64, 8, bits)
    P = _pools(1 << 20)
    batches = [*range(1, 66), 96, 127, 128, 129, 192, 193, 256, 384, 385, 511, 512, 513, 1000, 4097, 1 << 20]
    lengths = [1, 128, 129, 256, 257, 384, 385, 500, 511, 512, 513, 768, 1000, 1024, 1025, 2000, 2049, 3001, 4096, 5000, 8192,
               9001, 12288, 16384, 16385, 24065, 32768, 40000, 65536, 100001, 131071, 131072, 1 << 20, 1 << 28]
    need = np.array([[G.grinqh_attention_workspace_bytes(L, n_q, b, n) for n in lengths] for b in batches], np.int64)
    assert np.all(need % 256 == 0) and np.all(np.diff(need, axis=0) >= 0) and np.all(np.diff(need, axis=1) >= 0)

    def status(b, n, size):
        q = 1 << 16
        return lib.grinqh_decode_attention(ctypes.byref(L), ctypes.byref(P), q, 0, n_q * dim, n_q, 1 << 43, 1 << 24, 1 << 24,
                                           1 << 44, b, n, 0.1, q, 0, None, 1 << 42, size, None)

    for i, b in enumerate(batches):
        for j, n in enumerate(lengths):
            if b * heads * -(-n_q // heads // 16) <= 1 << 23:
                assert status(b, n, int(need[i, j])) == B.GRINQH_EINVAL, (b, n)
    assert status(1, 32768, 0) == B.GRINQH_ENOSPACE


def test_prefill_attention_checks_its_arguments_before_any_device_call():
    lib = G.load()
    Q, K, V, CQ, CK, OUT, LSE = (K64 * 16 * k for k in range(1, 8))
    good = dict(q=Q, k=K, v=V, q_stride=512, k_stride=128, v_stride=128, cu_q=CQ, cu_k=CK, batch=2, total_q=10,
                total_k=12, n_q_heads=8, n_kv_heads=2, head_dim=64, causal=1, scale=0.1, out=OUT, out_dtype=0, lse=LSE)

    def call(**kw):
        return lib.grinqh_prefill_attention(ctypes.byref(B.PrefillAttentionArgs(**dict(good, **kw))), None)

    assert lib.grinqh_prefill_attention(None, None) == B.GRINQH_EINVAL
    for key in ("q", "k", "v", "cu_q", "cu_k", "out"):
        assert call(**{key: None}) == B.GRINQH_EINVAL, key
    for key, value in (("batch", -1), ("batch", (1 << 20) + 1), ("total_q", -1), ("total_q", (1 << 24) + 1),
                       ("total_k", -1), ("total_k", (1 << 24) + 1), ("n_q_heads", 7), ("n_q_heads", 1026),
                       ("n_kv_heads", 0), ("head_dim", 96), ("scale", float("nan")), ("scale", 2e30), ("out_dtype", 2),
                       ("q_stride", 504), ("k_stride", 120), ("v_stride", 64), ("q_stride", (1 << 24) + 8),
                       ("out", Q + 64), ("out", K + 64), ("out", V + 64)):
        assert call(**{key: value}) == B.GRINQH_EINVAL, (key, value)
    assert call(workspace=64) == B.GRINQH_EALIGN
    few = dict(q_stride=512, total_q=20, total_k=9000, batch=1)
    need = lib.grinqh_prefill_attention_workspace_bytes(ctypes.byref(B.PrefillAttentionArgs(**dict(good, **few))))
    assert need > 0 and need % 4 == 0
    assert call(**few, workspace=K64 * 16 * 9, workspace_bytes=need - 1) == B.GRINQH_ENOSPACE
    assert lib.grinqh_prefill_attention_workspace_bytes(None) == 0
    for key, value in (("head_dim", 96), ("batch", -1), ("n_q_heads", 7), ("total_q", 5000)):     # the last: filled already
        a = B.PrefillAttentionArgs(**dict(good, **dict(few, **{key: value})))
        assert (lib.grinqh_prefill_attention_workspace_bytes(ctypes.byref(a)) == 0) == (key != "total_q"), key
    for key, value in (("q", Q + 8), ("k", K + 2), ("v", V + 4), ("cu_q", CQ + 2), ("cu_k", CK + 1), ("out", OUT + 8),
                       ("lse", LSE + 1), ("q_stride", 516), ("k_stride", 132), ("v_stride", 129)):
        assert call(**{key: value}) == B.GRINQH_EALIGN, (key, value)
    assert call(total_q=0) == B.GRINQH_OK and call(batch=0) == B.GRINQH_OK


def test_prefill_attention_refuses_to_write_where_it_reads():
    """out, lse and a workspace that is used against q, k, v, the ends and one another, at both ends of each."""
    lib = G.load()
    a = dict(q_stride=512, k_stride=128, v_stride=128, batch=1, total_q=20, total_k=9000, n_q_heads=8, n_kv_heads=2,
             head_dim=64, causal=1, scale=0.1, out_dtype=1)
    ws = lib.grinqh_prefill_attention_workspace_bytes(ctypes.byref(B.PrefillAttentionArgs(**a)))
    assert ws > 0
    sizes = dict(q=20 * 512 * 2, k=9000 * 128 * 2, v=9000 * 128 * 2, cu_q=8, cu_k=8, out=20 * 512 * 4, lse=20 * 8 * 4,
                 workspace=ws)
    good = {name: (i + 1) << 24 for i, name in enumerate(sizes)}
    for written, step in (("out", 16), ("lse", 4), ("workspace", 256)):
        for other in sizes:
            below = (sizes[written] - 1) // step * step
            for at in (0, -below, (sizes[other] - 1) // step * step):
                if other != written:
                    p = B.PrefillAttentionArgs(**a, **dict(good, **{written: good[other] + at}), workspace_bytes=ws)
                    assert lib.grinqh_prefill_attention(ctypes.byref(p), None) == B.GRINQH_EINVAL, (written, other, at)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        G.prefill_attention(x, x, x, cu)
    with pytest.raises(TypeError):
        G.prefill_attention([1], x, x, cu)
    L = G.grinqh_kv_layout_init(2, 64, 16, 8, 16)
    pool = torch.zeros(G.grinqh_kv_code_bytes(L), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        G.KVCache(L, pool, pool)
    with pytest.raises(G.GrinqhError):
        G.KVCache(B.KVLayout(2, 64, 16, 8, 16, 1), pool, pool)
    with pytest.raises(G.GrinqhError):
        G.new_attention_workspace(L, 3, 1, 10)


def test_prefill_workspace_of_many_empty_sequences():
    """A sequence without queries has no tile: the workspace and the limit follow
    from the sequences that can have one, at most a query each."""
    lib = G.load()
    sizes = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, causal=1, scale=0.1, q_stride=1024, k_stride=256, v_stride=256)

    def need(**kw):
        return lib.grinqh_prefill_attention_workspace_bytes(ctypes.byref(B.PrefillAttentionArgs(**dict(sizes, **kw))))

    for queries in (1, 10, 40):
        tiles, parts = queries * 4 // 128 + queries, 32                    # of a key-value head; of its keys, at most
        for batch in (1, 2, 100, 5000, 1 << 20):
            assert need(batch=batch, total_q=queries, total_k=1 << 24) <= tiles * 2 * parts * 128 * 130 * 4, (queries, batch)


def test_binding_refuses_sizes_that_do_not_fit_32_bits():
    """2^32 + n is not n: layouts, workspaces, the bound on the lengths and the number of sequences."""
    import torch
    from input_adaptive_bit_amd import attention as N
    good = (2, 64, 16, 8, 8)
    for at in range(5):
        for wrap in (2 ** 32, -2 ** 32, 2 ** 40):
            with pytest.raises(G.GrinqhError):
                G.grinqh_kv_layout_init(*(x + wrap * (i == at) for i, x in enumerate(good)))
    L = G.grinqh_kv_layout_init(*good)
    for at in range(3):
        for wrap in (2 ** 32, -2 ** 32):
            sizes = [x + wrap * (i == at) for i, x in enumerate((4, 3, 100))]
            assert G.grinqh_attention_workspace_bytes(L, *sizes) == 0
            with pytest.raises(G.GrinqhError):
                G.new_attention_workspace(L, *sizes)
    for wrap in (2 ** 32, -2 ** 32):
        assert G.grinqh_debug_kv_row(L, 3, 1 + wrap) == -1 and G.grinqh_debug_kv_row(L, 3 + wrap * 2 ** 32, 1) == -1
        assert G.grinqh_debug_page_row(L, 3, 1 + wrap, 0) == -1 and G.grinqh_debug_page_row(L, 3, 1, wrap * 2) == -1
        assert G.grinqh_debug_page_row(L, 3 + wrap, 1, 0) < 0

    class Sizes:
        """Stands for tensors on a GPU where only their sizes are asked for."""
        def __init__(self, *shape, dtype=torch.bfloat16):
            self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device("cuda", 0), True
            self.strides = [int(np.prod(shape[i + 1:], dtype=object)) for i in range(len(shape))]

        stride = lambda self: self.strides                       # noqa: E731
        numel = lambda self: self.shape.numel()                  # noqa: E731
        get_device = lambda self: 0                              # noqa: E731
        is_contiguous = lambda self: True                        # noqa: E731
        data_ptr = lambda self: 1 << 20                          # noqa: E731
        nbytes = 1 << 30

    sent, orig = [], (N._run, torch.Tensor)
    N._run, torch.Tensor = (lambda *a: sent.append(a)), Sizes
    try:
        cache = type("C", (), dict(device=torch.device("cuda", 0), n_kv_heads=2, head_dim=64, layout=L, _refs=()))()
        q, i32 = Sizes(3, 4, 64), torch.int32
        for max_len, passed in ((100, 100), (1 << 28, 1 << 28), (0, 0), (-5, 0), (2 ** 32 + 100, 0), (100 - 2 ** 32, 0)):
            N.grinqh_decode_attention(cache, q, Sizes(3, 7, dtype=i32), Sizes(3, dtype=i32), max_len, q, Sizes(64))
            assert sent.pop()[12] == passed
        for ends, batch in ((3, 2), ((1 << 20) + 1, 1 << 20), (2 ** 32 + 3, -1)):
            cu = Sizes(ends, dtype=i32)
            assert N._prefill_args(q, Sizes(5, 2, 64), Sizes(5, 2, 64), cu, cu, q, True, None, None).batch == batch
    finally:
        N._run, torch.Tensor = orig


def test_binding_says_what_does_not_fit():
    """Every condition of the calls' joint test has its own message."""
    import torch
    from input_adaptive_bit_amd import attention as N

    class Fake:
        """Stands for a tensor on a GPU."""
        def __init__(self, *shape, dtype=torch.bfloat16, stride=None, device=torch.device("cuda", 0)):
            self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, device, device.type == "cuda"
            c = [1]
            for n in reversed(shape[1:]):
                c.insert(0, c[0] * n)
            self._stride = tuple(stride or c)

        def stride(self, i=None):
            return self._stride if i is None else self._stride[i]

        def dim(self):
            return len(self.shape)

        def numel(self):
            return self.shape.numel()

        def get_device(self):
            return self.device.index if self.is_cuda else -1

        def is_contiguous(self):
            return all(n < 2 or s == c for n, s, c in zip(self.shape, self._stride, Fake(*self.shape)._stride))

        def data_ptr(self):
            return 4096

        nbytes = 1 << 20

    sent = []
    orig = N._run, torch.Tensor
    N._run = lambda name, *a: sent.append(name)
    torch.Tensor = Fake
    try:
        cache = type("C", (), dict(device=torch.device("cuda", 0), n_kv_heads=2, head_dim=64, _refs=()))()
        cpu, i32, i64, f16 = torch.device("cpu"), torch.int32, torch.int64, torch.float16
        rows = lambda n=3, **kw: Fake(n, 2, 64, **kw)                                                  # noqa: E731

        def refuse(call, *good, **bad):
            call(*good)
            assert sent.pop()
            for at, others in bad.items():
                for other in others:
                    a = list(good)
                    a[int(at[1:])] = other
                    with pytest.raises((TypeError, ValueError)):
                        call(*a)
                    assert not sent, (call, at)

        shapes = [rows(4), Fake(3, 2, 32), Fake(3, 1, 64), Fake(3, 128), rows(stride=(64, 64, 1)), rows(stride=(128, 1, 2)),
                  rows(dtype=f16), rows(dtype=torch.float32), rows(device=cpu), rows(device=torch.device("cuda", 1)), None]
        slots = [Fake(4, dtype=i64), Fake(3, dtype=i32), Fake(3, dtype=i64, stride=(2,)), Fake(3, dtype=i64, device=cpu), 7]
        refuse(lambda *a: N.grinqh_kv_write(cache, *a), rows(), rows(), Fake(3, dtype=i64), _0=shapes, _1=shapes, _2=slots)

        ints = [Fake(2, dtype=i32), Fake(3, dtype=i64), Fake(3, dtype=i32, stride=(2,)), Fake(3, dtype=i32, device=cpu), None]
        q, out = Fake(3, 8, 64), Fake(3, 8, 64)
        refuse(lambda q, t, n, o, w: N.grinqh_decode_attention(cache, q, t, n, 10, o, w),
               q, Fake(3, 5, dtype=i32), Fake(3, dtype=i32), out, Fake(64),
               _0=[Fake(3, 8, 32), Fake(3, 512), Fake(3, 8, 64, stride=(64, 64, 1)), Fake(3, 8, 64, dtype=f16),
                   Fake(3, 8, 64, device=cpu), Fake(4, 8, 64), 1],
               _1=[Fake(2, 5, dtype=i32), Fake(3, 5, dtype=i64), Fake(3, 5, dtype=i32, stride=(10, 2)), Fake(15, dtype=i32),
                   Fake(3, 5, dtype=i32, device=cpu)],
               _2=ints, _3=[Fake(3, 7, 64), Fake(3, 8, 64, dtype=f16), Fake(3, 8, 64, stride=(1024, 64, 1)), None],
               _4=[Fake(64, device=cpu), Fake(64, stride=(2,))])

        wide = [Fake(4, 2, 32), Fake(4, 128), Fake(4, 2, 64, stride=(64, 64, 1)), Fake(4, 2, 64, dtype=torch.float32),
                Fake(4, 2, 64, device=cpu), None]
        refuse(lambda *a: N.grinqh_prefill_attention(*a), q, Fake(4, 2, 64), Fake(4, 2, 64), Fake(3, dtype=i32),
               Fake(3, dtype=i32), out, _0=[Fake(3, 8, 64, dtype=torch.float32), Fake(3, 8, 64, device=cpu), Fake(24, 64)],
               _1=wide, _2=wide + [Fake(5, 2, 64)], _3=ints, _4=ints,
               _5=[Fake(3, 7, 64), Fake(3, 8, 64, dtype=f16), Fake(3, 8, 64, device=cpu)])
    finally:
        N._run, torch.Tensor = orig


def test_binding_takes_the_stride_of_a_token_and_refuses_other_views():
    import torch
    from input_adaptive_bit_amd import attention as N
    device = torch.device("cpu")
    orig, N._tensor = N._tensor, lambda t, name, device=None: t.device
    try:
        fused = torch.zeros(5, 12, 64)
        assert N._rows(fused[:, 8:10], "k", 2, 64, device) == 12 * 64
        assert N._rows(fused[:1, 8:10], "k", 2, 64, device) == 2 * 64        # one token has no next
        assert N._rows(torch.zeros(5, 1, 64).transpose(0, 1).transpose(0, 1), "k", 1, 64, device) == 64
        assert N._rows(torch.zeros(0, 2, 64), "k", 2, 64, device) == 128
        for bad in (fused.transpose(1, 2), fused[:, ::2], fused[..., ::2], torch.zeros(1, 2, 64).expand(5, 2, 64)):
            with pytest.raises(ValueError):
                N._rows(bad, "k", bad.shape[1], bad.shape[2], device)
    finally:
        N._tensor = orig
