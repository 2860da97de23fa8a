"""The 4-bit products', the rotation's and the page plan's oracle, host checks
and binding refusals; no GPU (every library call here is host arithmetic or fails
a host check, so no kernel is launched)."""

import ctypes
import os

import numpy as np
import pytest

import input_adaptive_bit_amd as G
from input_adaptive_bit_amd import grinqh as B
from oracle import decoder_oracle as O

K = 1 << 24                                       # places in memory that nothing overlaps


# --------------------------------------------------------------- the oracle --

def test_weights_are_midpoints_of_their_groups():
    q = np.array([[0, 1, 15, 7]])
    w = O.weights(q, np.array([[2.0, 0.5]]), np.array([[-1.0, 3.0]]), 2)
    assert w.tolist() == [[0.0, 2.0, 10.75, 6.75]]


def test_product_written_out():
    rng = np.random.default_rng(0)
    q, s, z = rng.integers(0, 16, (3, 64)), rng.random((3, 2)), rng.standard_normal((3, 2))
    x = rng.standard_normal((2, 64))
    y, size = O.linear(x, q, s, z, 32)
    for t in range(2):
        for j in range(3):
            want = sum(x[t, i] * (s[j, i // 32] * (q[j, i] + 0.5) + z[j, i // 32]) for i in range(64))
            assert np.isclose(y[t, j], want) and size[t, j] >= abs(want)


def test_packed_words_hold_each_code_where_the_header_says():
    """Every code alone, at the bits that grinqh.h names."""
    for j, i in ((0, 0), (15, 127), (3, 45), (16, 128), (20, 200)):
        q = np.zeros((1, 32, 256), np.int64)
        q[0, j, i] = 15
        words = O.packed_codes(q)
        m, c, e = i % 128 // 32, i % 32 // 8, i % 8
        lane = 16 * c + j % 16
        word = int(words[0, j // 16, i // 128, lane, m])
        assert word == sum(1 << (3 + 4 * (e // 2) + 16 * (e % 2) + k) % 32 for k in range(4))
        assert np.count_nonzero(words) == 1


def test_experts_take_their_runs_and_gathered_rows():
    rng = np.random.default_rng(1)
    q, s, z = rng.integers(0, 16, (2, 3, 32)), rng.random((2, 3, 1)), rng.standard_normal((2, 3, 1))
    x = rng.standard_normal((4, 32))
    y, _, written = O.experts(x, np.array([1, 3, 4]), np.array([0, 3, -1, 2, 9]), 5, q, s, z, 32)
    assert written.tolist() == [False, True, True, True, False]
    assert np.allclose(y[1], x[3] @ O.weights(q[0], s[0], z[0], 32).T) and np.all(y[2] == 0)
    assert np.allclose(y[3], x[2] @ O.weights(q[1], s[1], z[1], 32).T)


def test_rotation_keeps_lengths_and_angles_between_positions():
    rng = np.random.default_rng(2)
    x, freqs = rng.standard_normal((1, 1, 8)), np.array([1.0, 0.1])
    for neighbours in (False, True):
        a, _ = O.rope(x, [5], freqs, neighbours=neighbours)
        assert np.isclose((a ** 2).sum(), (x ** 2).sum()) and np.array_equal(a[..., 4:], x[..., 4:])
        back, _ = O.rope(a, [-5], freqs, neighbours=neighbours)
        assert np.allclose(back, x)
    quarter, _ = O.rope(np.array([[[1.0, 0.0]]]), [1], np.array([np.pi / 2]))
    assert np.allclose(quarter, [[[0.0, 1.0]]])
    normed, _ = O.rope(np.array([[[3.0, 4.0]]]), [0], np.array([0.3]), [2.0, 1.0], 0.0)
    assert np.allclose(normed, np.array([6.0, 4.0]) / np.sqrt(12.5))


def test_extend_written_out():
    """Two sequences of pages of 16: one fills its page and takes a new one, one begins; the third finds none left."""
    got = O.extend([[4, -1], [-1, -1], [-1, -1]], [15, 0, 0], [2, 3, 1], [7, 9, -1, -1, -1, -1, -1, -1, -1, -1], 2, 16, 8)
    assert got["table"].tolist() == [[4, 9], [7, -1], [-1, -1]]
    assert got["slots"].tolist() == [79, 144, 112, 113, 114, -1, -1, -1] and got["positions"].tolist() == [15, 16, 0, 1, 2, 0, 0, 0]
    assert got["seq_lens"].tolist() == [17, 3, 0] and got["cu_q"].tolist() == [0, 2, 5, 6] and got["cu_k"].tolist() == [0, 17, 20, 20]
    assert got["n_free"] == 0 and got["refused"] == 1
    table, lens, free, n = O.release(got["table"], got["seq_lens"], [1, 0, 0], [7, 9, -1, -1, -1, -1, -1, -1, -1, -1], 0, 16)
    assert table.tolist() == [[-1, -1], [7, -1], [-1, -1]] and free[:2].tolist() == [4, 9] and n == 2 and lens.tolist() == [0, 3, 0]


# -------------------------------------------------------------- 4-bit weights --

def test_fourbit_layout_sizes():
    L = G.grinqh_fourbit_layout_init(4096, 14336, 128, 8)
    assert (L.k_tiles, L.row_tiles) == (32, 896)
    assert G.grinqh_fourbit_code_bytes(L) == 8 * 4096 * 14336 // 2 and G.grinqh_fourbit_grid_bytes(L) == 8 * 14336 * 32 * 4
    L = G.grinqh_fourbit_layout_init(160, 17, 32)
    assert G.grinqh_fourbit_code_bytes(L) == 2 * 2 * 1024 and G.grinqh_fourbit_grid_bytes(L) == 2 * 2 * 4 * 64
    for field, value in (("k_tiles", 1), ("row_tiles", 3), ("group", 16), ("n_experts", 0), ("d_in", 161)):
        bad = G.grinqh_fourbit_layout_init(160, 17, 32)
        setattr(bad, field, value)
        assert G.grinqh_fourbit_code_bytes(bad) == 0 and G.grinqh_fourbit_grid_bytes(bad) == 0


@pytest.mark.parametrize("bad", [(0, 16, 32, 1), (128, 0, 32, 1), (128, 16, 16, 1), (128, 16, 256, 1), (160, 16, 64, 1), (32, 16, 64, 1),
                                 (128, 16, 32, 0), (128, 16, 32, 1025), ((1 << 20) + 128, 16, 128, 1), (128, (1 << 20) + 1, 128, 1),
                                 (1 << 20, 1 << 20, 128, 4), (128 + 2 ** 32, 16, 128, 1), (128, 16 + 2 ** 32, 128, 1),
                                 (128, 16, 128 + 2 ** 32, 1), (128, 16, 128, 1 + 2 ** 32), (-128, 16, 128, 1)])
def test_fourbit_layouts_outside_the_ranges_are_refused(bad):
    with pytest.raises(G.GrinqhError):
        G.grinqh_fourbit_layout_init(*bad)
    assert B.load().grinqh_fourbit_layout_init(128, 16, 32, 1, None) == B.GRINQH_EINVAL


def test_fourbit_calls_check_their_arguments_before_any_device_call():
    lib = G.load()
    L, E = G.grinqh_fourbit_layout_init(256, 40, 64), G.grinqh_fourbit_layout_init(256, 40, 64, 3)

    def pack(L=L, q=K, s=2 * K, z=3 * K, c=4 * K, g=5 * K):
        return lib.grinqh_fourbit_pack(None if L is None else ctypes.byref(L), q, s, z, c, g, None)

    def linear(L=L, x=K, xd=0, xs=256, n=5, c=2 * K, g=3 * K, y=4 * K, yd=0):
        return lib.grinqh_fourbit_linear(None if L is None else ctypes.byref(L), x, xd, xs, n, c, g, y, yd, None)

    def experts(L=E, **kw):
        a = dict(x=K, x_stride=256, x_dtype=0, n_x=4, rows=2 * K, ends=3 * K, n_rows=9, codes=4 * K, grid=5 * K, y=6 * K, y_dtype=0)
        return lib.grinqh_expert_linear(None if L is None else ctypes.byref(L), ctypes.byref(B.ExpertArgs(**dict(a, **kw))), None)

    for call, names in ((pack, "Lqszcg"), (linear, ("L", "x", "c", "g", "y")), (experts, ("L", "x", "ends", "codes", "grid", "y"))):
        for name in names:
            assert call(**{name: None}) == B.GRINQH_EINVAL, name
    assert lib.grinqh_expert_linear(ctypes.byref(E), None, None) == B.GRINQH_EINVAL
    assert linear(L=E) == B.GRINQH_EINVAL                                             # several experts are not one layer
    for key, value in (("q", K + 4), ("s", 2 * K + 1), ("z", 3 * K + 1), ("c", 4 * K + 8), ("g", 5 * K + 4)):
        assert pack(**{key: value}) == B.GRINQH_EALIGN, key
    for key, value in (("xd", 2), ("yd", -1), ("n", -1), ("n", (1 << 20) + 1), ("xs", 248), ("xs", (1 << 24) + 8)):
        assert linear(**{key: value}) == B.GRINQH_EINVAL, (key, value)
    for key, value in (("x", K + 8), ("xs", 260), ("c", 2 * K + 8), ("g", 3 * K + 2), ("y", 4 * K + 1)):
        assert linear(**{key: value}) == B.GRINQH_EALIGN, (key, value)
    assert linear(xd=1, xs=258) == B.GRINQH_EALIGN and linear(yd=1, y=4 * K + 2) == B.GRINQH_EALIGN
    for key, value in (("x_dtype", 7), ("y_dtype", 2), ("n_rows", -1), ("n_rows", (1 << 20) + 1), ("n_x", 0), ("n_x", (1 << 20) + 1),
                       ("x_stride", 255)):
        assert experts(**{key: value}) == B.GRINQH_EINVAL, (key, value)
    for key, value in (("x", K + 2), ("x_stride", 257), ("rows", 2 * K + 2), ("ends", 3 * K + 1), ("codes", 4 * K + 4), ("grid", 5 * K + 8),
                       ("y", 6 * K + 1)):
        assert experts(**{key: value}) == B.GRINQH_EALIGN, (key, value)
    assert linear(n=0) == B.GRINQH_OK and experts(n_rows=0) == B.GRINQH_OK            # nothing to do, nothing launched


def test_fourbit_calls_refuse_to_write_where_they_read():
    lib = G.load()
    E = G.grinqh_fourbit_layout_init(256, 40, 64, 3)
    codes, grid = G.grinqh_fourbit_code_bytes(E), G.grinqh_fourbit_grid_bytes(E)
    sizes = dict(x=(3 * 264 + 256) * 2, rows=36, ends=16, codes=codes, grid=grid, y=9 * 40 * 2)
    good = {name: (i + 1) * K for i, name in enumerate(sizes)}
    for other in sizes:
        for at in (0, -(sizes["y"] - 2), (sizes[other] - 1) // 16 * 16):
            if other != "y":
                a = B.ExpertArgs(**dict(good, y=good[other] + at), x_stride=264, x_dtype=0, n_x=4, n_rows=9, y_dtype=0)
                assert lib.grinqh_expert_linear(ctypes.byref(E), ctypes.byref(a), None) == B.GRINQH_EINVAL, (other, at)
    sizes = dict(q=3 * 40 * 256, s=3 * 40 * 4 * 2, z=3 * 40 * 4 * 2, codes=codes, grid=grid)
    good = {name: (i + 1) * K for i, name in enumerate(sizes)}
    for written in ("codes", "grid"):
        for other in sizes:
            for at in (0, -(sizes[written] - 1) // 16 * 16 + 16, (sizes[other] - 1) // 16 * 16):
                if other != written:
                    a = dict(good, **{written: good[other] + at})
                    assert lib.grinqh_fourbit_pack(ctypes.byref(E), *a.values(), None) == B.GRINQH_EINVAL, (written, other, at)


# -------------------------------------------------------------------- rope --

def _rope(**kw):
    cache, pools = kw.pop("cache", None), kw.pop("pools", None)
    a = dict(q=K, k=2 * K, v=None, q_stride=512, k_stride=128, v_stride=128, n_tokens=4, n_q_heads=8, n_kv_heads=2, head_dim=64,
             dtype=0, q_weight=3 * K, k_weight=4 * K, weight_dtype=1, eps=1e-6, positions=5 * K, freqs=6 * K, rope_dim=32, neighbours=0,
             q_out=7 * K, k_out=8 * K, q_out_stride=512, k_out_stride=128, slots=None)
    a.update(kw)
    p = B.RopeArgs(**a)
    if cache is not None:
        p.cache, p.pools = ctypes.pointer(cache), ctypes.pointer(pools)
    return G.load().grinqh_qk_rope(ctypes.byref(p), None)


def test_rope_checks_its_arguments_before_any_device_call():
    L = G.grinqh_kv_layout_init(2, 64, 16, 8, 8)
    P = B.KVPools(*((20 + i) * K for i in range(4)))
    cached = dict(cache=L, pools=P, v=9 * K, slots=10 * K)
    assert G.load().grinqh_qk_rope(None, None) == B.GRINQH_EINVAL
    for key in ("q", "k", "positions", "freqs", "q_out", "k_out"):
        assert _rope(**{key: None}) == B.GRINQH_EINVAL, key
    for key in ("v", "slots"):
        assert _rope(**dict(cached, **{key: None})) == B.GRINQH_EINVAL, key
    for key, value in (("n_tokens", -1), ("n_tokens", (1 << 24) + 1), ("n_q_heads", 0), ("n_q_heads", 1025), ("n_kv_heads", 0),
                       ("head_dim", 96), ("head_dim", 32), ("rope_dim", -16), ("rope_dim", 72), ("rope_dim", 80), ("rope_dim", 8),
                       ("dtype", 2), ("weight_dtype", 5), ("eps", -1e-3), ("eps", float("nan")), ("eps", float("inf")),
                       ("q_stride", 504), ("k_stride", 120), ("q_out_stride", 511), ("k_out_stride", 127),
                       ("q_stride", (1 << 24) + 8)):
        assert _rope(**{key: value}) == B.GRINQH_EINVAL, (key, value)
    for key, value in (("q", K + 8), ("k", 2 * K + 2), ("q_weight", 3 * K + 4), ("k_weight", 4 * K + 8), ("positions", 5 * K + 2),
                       ("freqs", 6 * K + 4), ("q_out", 7 * K + 8), ("k_out", 8 * K + 4), ("q_stride", 516), ("k_stride", 132),
                       ("q_out_stride", 514), ("k_out_stride", 129)):
        assert _rope(**{key: value}) == B.GRINQH_EALIGN, (key, value)
    assert _rope(**dict(cached, v_stride=127)) == B.GRINQH_EINVAL and _rope(**dict(cached, v=9 * K + 8)) == B.GRINQH_EALIGN
    assert _rope(**dict(cached, slots=10 * K + 4)) == B.GRINQH_EALIGN
    for bad in ((4, 64, 16, 8, 8), (2, 128, 16, 8, 8)):
        assert _rope(**dict(cached, cache=G.grinqh_kv_layout_init(*bad))) == B.GRINQH_EINVAL
    assert _rope(**dict(cached, pools=B.KVPools(None, 21 * K, 22 * K, 23 * K))) == B.GRINQH_EINVAL
    assert _rope(**dict(cached, cache=B.KVLayout(2, 64, 16, 8, 8, 1))) == B.GRINQH_EINVAL
    assert _rope(n_tokens=0) == B.GRINQH_OK


def test_rope_refuses_outputs_over_what_it_reads():
    """At both ends; in place only as a whole, and between a fused projection's rows only where no row is shared."""
    L = G.grinqh_kv_layout_init(2, 64, 16, 8, 8)
    codes, grid = G.grinqh_kv_code_bytes(L), G.grinqh_kv_grid_bytes(L)
    sizes = dict(q=4 * 512 * 2, k=4 * 128 * 2, v=4 * 128 * 2, q_weight=256, k_weight=256, positions=16, freqs=128, slots=32,
                 q_out=4 * 512 * 2, k_out=4 * 128 * 2, kc=codes, vc=codes, kg=grid, vg=grid)
    good = {name: (i + 1) * K for i, name in enumerate(sizes)}

    def status(**at):
        a = dict(good, **at)
        pools = B.KVPools(*(a.pop(n) for n in ("kc", "vc", "kg", "vg")))
        return _rope(cache=L, pools=pools, **a)

    for written in ("q_out", "k_out", "kc", "vc", "kg", "vg"):
        for other in sizes:
            if other == written:
                continue
            first = 16 if (written, other) in (("q_out", "q"), ("k_out", "k")) else 0      # 0 there: in place
            for at in (first, -(sizes[written] - 16), (sizes[other] - 1) // 16 * 16):
                assert status(**{written: good[other] + at}) == B.GRINQH_EINVAL, (written, other, at)
    # rows of a fused projection, 12 heads a token: q at 0, k at 512, v at 640 elements
    fused = dict(q=K, k=K + 1024, v=K + 1280, q_stride=768, k_stride=768, v_stride=768, q_out_stride=768, k_out_stride=768)
    for at in (dict(q_out=K + 128, k_out=40 * K), dict(q_out=K + 256, k_out=40 * K), dict(q_out=40 * K, k_out=K + 1152),
               dict(q_out=40 * K, k_out=K + 1280), dict(q_out=40 * K, k_out=K + 896), dict(q_out=K, k_out=K),
               dict(q_out=K, k_out=K + 1024, k_out_stride=776), dict(q_out=40 * K, k_out=K + 1024 + 1536)):
        assert status(**dict(fused, **at)) == B.GRINQH_EINVAL, at


# ------------------------------------------------------------------- pages --

def test_extend_and_release_check_their_arguments_before_any_device_call():
    lib = G.load()
    names = ("page_table", "seq_lens", "n_new", "free_pages", "n_free", "new_lens", "n_free_out", "refused", "cu_q", "cu_k", "slots",
             "positions", "workspace")
    good = {n: (i + 1) * K for i, n in enumerate(names)}
    sizes = dict(table_stride=6, batch=5, max_pages=4, page_size=16, n_pages=30, capacity=50)
    need = G.grinqh_kv_extend_workspace_bytes(5)

    def extend(**kw):
        return lib.grinqh_kv_extend(ctypes.byref(B.ExtendArgs(**dict({**good, **sizes, "workspace_bytes": need}, **kw))), None)

    assert lib.grinqh_kv_extend(None, None) == B.GRINQH_EINVAL
    for name in names:
        assert extend(**{name: None}) == B.GRINQH_EINVAL, name
        assert extend(**{name: good[name] + (8 if name == "workspace" else 4 if name == "slots" else 2)}) == B.GRINQH_EALIGN, name
    for key, value in (("batch", -1), ("batch", (1 << 20) + 1), ("max_pages", 0), ("max_pages", (1 << 24) + 1), ("table_stride", 3),
                       ("page_size", 24), ("page_size", 0), ("n_pages", 0), ("n_pages", (1 << 24) + 1), ("capacity", -1),
                       ("capacity", (1 << 24) + 1), ("table_stride", (1 << 24) + 1)):
        assert extend(**{key: value}) == B.GRINQH_EINVAL, (key, value)
    assert extend(workspace_bytes=need - 1) == B.GRINQH_ENOSPACE
    assert need >= 40 and G.grinqh_kv_extend_workspace_bytes(-1) == 0 and G.grinqh_kv_extend_workspace_bytes(2 ** 32 + 5) == 0
    spans = dict(page_table=(4 * 6 + 4) * 4, seq_lens=20, n_new=20, free_pages=120, n_free=4, new_lens=20, n_free_out=4, refused=4,
                 cu_q=24, cu_k=24, slots=400, positions=200, workspace=need)
    for written in ("page_table", "new_lens", "n_free_out", "refused", "cu_q", "cu_k", "slots", "positions", "workspace"):
        for other in spans:
            if other == written:
                continue
            step = {"slots": 8, "workspace": 16}.get(written, 4)
            for at in (0, -((spans[written] - 1) // step * step), (spans[other] - 1) // step * step):
                if at == 0 and (written, other) in (("new_lens", "seq_lens"), ("n_free_out", "n_free")):
                    continue                                                        # in place
                assert extend(**{written: good[other] + at}) == B.GRINQH_EINVAL, (written, other, at)

    def release(t=K, ts=6, n=2 * K, f=3 * K, b=5, mp=4, ps=16, l=4 * K, c=5 * K, pages=30):
        return lib.grinqh_kv_release(t, ts, n, f, b, mp, ps, l, c, pages, None)

    for key in ("t", "n", "f", "l", "c"):
        assert release(**{key: None}) == B.GRINQH_EINVAL, key
    for key in ("t", "n", "l", "c"):
        assert release(**{key: 7 * K + 2}) == B.GRINQH_EALIGN, key
    for key, value in (("ts", 3), ("b", -1), ("mp", 0), ("ps", 8), ("pages", 0), ("t", 2 * K), ("n", 3 * K), ("l", K), ("c", 4 * K)):
        assert release(**{key: value}) == B.GRINQH_EINVAL, (key, value)
    assert release(b=0) == B.GRINQH_OK


# ----------------------------------------------------------------- binding --

def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    q, s = torch.zeros(16, 128, dtype=torch.uint8), torch.zeros(16, 1, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        G.fourbit_pack(q, s, s)
    with pytest.raises(TypeError):
        G.fourbit_pack([1], s, s)
    with pytest.raises(ValueError, match="GPU"):
        G.fourbit_quantize(torch.zeros(16, 128, dtype=torch.bfloat16), 32)
    L = G.grinqh_fourbit_layout_init(128, 16, 32)
    with pytest.raises(ValueError, match="GPU"):
        G.FourbitWeight(L, torch.zeros(1024, dtype=torch.uint8), torch.zeros(128, dtype=torch.float16))
    with pytest.raises(G.GrinqhError):
        G.FourbitWeight(B.FourbitLayout(128, 16, 32, 1, 1, 2), None, None)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        G.qk_rope(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))
    lens = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: G.kv_extend(torch.zeros(3, 4, dtype=torch.int32), lens, lens, lens, lens, 16, 8),
                 lambda: G.kv_release(torch.zeros(3, 4, dtype=torch.int32), lens, lens, lens, lens, 16)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for n in (0, -1, (1 << 24) + 1):
        with pytest.raises(G.GrinqhError):
            G.new_page_list(n, "cpu")
    free, n_free = G.new_page_list(3, "cpu")
    assert free.tolist() == [2, 1, 0] and n_free.tolist() == [3]


class Fake:
    """Stands for a tensor on a GPU."""
    def __init__(self, *shape, dtype=None, stride=None, device="cuda:0"):
        import torch
        self.shape, self.dtype, self.device = torch.Size(shape), dtype or torch.bfloat16, torch.device(device)
        self.is_cuda = self.device.type == "cuda"
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


def test_binding_says_what_does_not_fit(monkeypatch):
    """Every condition of the calls' joint tests has its own message."""
    import torch
    from input_adaptive_bit_amd import attention, fourbit, pages, rope
    sent = []
    for module in (fourbit, rope, pages):
        monkeypatch.setattr(module, "_run", lambda name, *a: sent.append(name))
    monkeypatch.setattr(torch, "Tensor", Fake)
    f32, f16, i32, i64, u8, f64 = torch.float32, torch.float16, torch.int32, torch.int64, torch.uint8, torch.float64
    far = "cuda:1"

    def refuse(call, *good, **bad):
        call(*good)
        assert sent.pop()
        for at, others in bad.items():
            for other in others:
                a = list(good)
                a[int(at[1:])] = other
                with pytest.raises((TypeError, ValueError, AttributeError)):
                    call(*a)
                assert not sent, (call, at)

    L, E = G.grinqh_fourbit_layout_init(64, 24, 32), G.grinqh_fourbit_layout_init(64, 24, 32, 3)
    one, many = (G.FourbitWeight(x, Fake(1 << 14, dtype=u8), Fake(1 << 12, dtype=f16)) for x in (L, E))
    x_bad = [Fake(5, 32), Fake(5, 64, dtype=f16), Fake(5, 64, device="cpu"), Fake(5, 64, device=far), Fake(5, 64, stride=(128, 2)),
             Fake(5, 64, stride=(32, 1)), Fake(5, 2, 32), None]
    y_bad = [Fake(5, 24, dtype=f16), Fake(5, 24, device=far), Fake(5, 24, stride=(48, 1)), None]
    refuse(lambda *a: fourbit.grinqh_fourbit_linear(one, *a), Fake(5, 64), Fake(5, 24), _0=x_bad, _1=y_bad + [Fake(4, 24)])
    refuse(lambda x, e, y, r: fourbit.grinqh_expert_linear(many, x, e, y, r), Fake(5, 64), Fake(4, dtype=i32), Fake(7, 24), Fake(7, dtype=i32),
           _0=x_bad, _1=[Fake(3, dtype=i32), Fake(5, dtype=i32), Fake(4, dtype=i64), Fake(4, dtype=i32, device=far), None],
           _2=y_bad + [Fake(7, 25), Fake(6, 24)], _3=[Fake(6, dtype=i32), Fake(7, dtype=i64), Fake(7, dtype=i32, device="cpu")])
    refuse(lambda *a: fourbit.grinqh_fourbit_pack(L, *a), Fake(24, 64, dtype=u8), Fake(24, 2, dtype=f16), Fake(24, 2, dtype=f16),
           Fake(2048, dtype=u8), Fake(256, dtype=f16), _0=[Fake(24, 32, dtype=u8), Fake(24, 64, dtype=i32), Fake(24, 64, dtype=u8, stride=(128, 1))],
           _1=[Fake(24, 1, dtype=f16), Fake(24, 2, dtype=f32)], _2=[Fake(24, 2, dtype=f16, device=far)], _3=[Fake(2047, dtype=u8)],
           _4=[Fake(255, dtype=f16), None])

    rows = lambda h=2, n=3, **kw: Fake(n, h, 64, **kw)                                                # noqa: E731
    shapes = lambda h: [rows(h, 4), Fake(3, h, 32), rows(h, stride=(64, 64, 1)), rows(h, dtype=f16), rows(h, dtype=f32),      # noqa: E731
                        rows(h, device="cpu"), rows(h, device=far), rows(h, stride=(64 * h, 1, h)), Fake(3, 64 * h), 1]
    refuse(lambda q, k, p, f, a, b, qw, kw: rope.grinqh_qk_rope(q, k, p, f, a, b, qw, kw), rows(4), rows(), Fake(3, dtype=i32),
           Fake(8, dtype=f64), rows(4), rows(), Fake(64), Fake(64), _0=shapes(4), _1=shapes(2)[:-1],
           _2=[Fake(2, dtype=i32), Fake(4, dtype=i32), Fake(3, dtype=i64), Fake(3, dtype=i32, stride=(2,)), None],
           _3=[Fake(8, dtype=f32), Fake(8, dtype=f64, device=far), Fake(8, dtype=f64, stride=(2,))], _4=shapes(4) + [None], _5=shapes(2) + [None],
           _6=[Fake(32), Fake(128), Fake(64, dtype=f16), Fake(64, dtype=f32), Fake(64, device=far)],
           _7=[Fake(32), Fake(64, dtype=f16), Fake(64, dtype=f32), Fake(64, stride=(2,))])
    layout = G.grinqh_kv_layout_init(2, 64, 16, 8, 16)
    cache = G.KVCache(layout, Fake(1 << 20, dtype=u8), Fake(1 << 20, dtype=u8))
    wide = G.KVCache(G.grinqh_kv_layout_init(4, 64, 16, 4, 16), Fake(1 << 20, dtype=u8), Fake(1 << 20, dtype=u8))
    refuse(lambda c, v, s, k: rope.grinqh_qk_rope(rows(4), rows(), Fake(3, dtype=i32), Fake(8, dtype=f64), rows(4), k, cache=c, v=v, slots=s),
           cache, rows(), Fake(3, dtype=i64), None, _0=[wide, None, 3], _1=shapes(2) + [None],
           _2=[Fake(2, dtype=i64), Fake(3, dtype=i32), Fake(3, dtype=i64, device=far), None])

    step = lambda **kw: pages.Step(**dict(dict(slots=Fake(9, dtype=i64), positions=Fake(9, dtype=i32), cu_q=Fake(4, dtype=i32),    # noqa: E731
                                               cu_k=Fake(4, dtype=i32), seq_lens=Fake(3, dtype=i32), n_free=Fake(1, dtype=i32),
                                               refused=Fake(1, dtype=i32)), **kw))
    ints = [Fake(2, dtype=i32), Fake(3, dtype=i64), Fake(3, dtype=i32, device=far), None]
    refuse(lambda t, n, w, f, c, s, ws: pages.grinqh_kv_extend(t, n, w, f, c, 16, s, ws), Fake(3, 5, dtype=i32), Fake(3, dtype=i32),
           Fake(3, dtype=i32), Fake(20, dtype=i32), Fake(1, dtype=i32), step(), Fake(64),
           _0=[Fake(2, 5, dtype=i32), Fake(3, 5, dtype=i64), Fake(3, 5, dtype=i32, stride=(10, 2)), Fake(3, 5, dtype=i32, stride=(4, 1)),
               Fake(15, dtype=i32), Fake(3, 5, dtype=i32, device=far)],
           _1=ints, _2=ints, _3=[Fake(20, dtype=i64), Fake(0, dtype=i32)], _4=[Fake(0, dtype=i32), Fake(1, dtype=i64)],
           _5=[step(slots=Fake(8, dtype=i64)), step(slots=Fake(9, dtype=i32)), step(positions=Fake(9, dtype=i64)), step(cu_q=Fake(3, dtype=i32)),
               step(cu_k=Fake(4, dtype=i32, device=far)), step(seq_lens=Fake(2, dtype=i32)), step(refused=Fake(1, dtype=f32))],
           _6=[Fake(64, device="cpu"), Fake(64, stride=(2,))])
    refuse(lambda t, n, d, f, c: pages.grinqh_kv_release(t, n, d, f, c, 16), Fake(3, 5, dtype=i32), Fake(3, dtype=i32), Fake(3, dtype=u8),
           Fake(20, dtype=i32), Fake(1, dtype=i32), _0=[Fake(2, 5, dtype=i32), Fake(3, 5, dtype=i64)], _1=[Fake(2, dtype=i32), Fake(3, dtype=i64)],
           _2=[Fake(2, dtype=u8), Fake(3, dtype=i32), Fake(3, dtype=u8, device=far)], _3=[Fake(20, dtype=i64)], _4=[Fake(1, dtype=f32)])


# --------------------------------------------------------------- the cases --

def test_operator_cases_are_what_the_file_says():
    """The measured cases' own arithmetic: names, sizes, the spread of the drawn ones."""
    import random
    import sys
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from perf import more_operators as M
    cases = M.listed()
    assert 4 <= len(cases) <= 12 and len({c["name"] for c in cases}) == len(cases)
    assert all(sum(c["op"] == op for c in cases) >= 2 for op in {c["op"] for c in cases})
    rng = random.Random(0)
    most = max(M.work(c)["flops"] for c in cases)
    for c in (M.draw(rng) for _ in range(200)):
        work = M.work(c)
        assert 0 < work["bytes"] and work["flops"] <= 1.05 * most
