"""GPU parity of the products with 4-bit weights (grinqh_fourbit_linear,
grinqh_expert_linear) with the fp64 oracle.

Bound.  A sum of n products in any order is off by at most n steps of fp32 of
the sum of their magnitudes (a step, 2^-23: the matrix cores may cut instead of
rounding).  A group's sum has group + 16 terms, their scaling and addition over
the groups 3 each, so an output is within (group + 3 groups + 32) 2^-23 of the
magnitudes s (16 + q) |x| + |z - 15.5 s| |x| that they go through, and its
type's rounding.
"""

import numpy as np
import pytest

from oracle import attention_oracle as A
from oracle import decoder_oracle as O
from tests.attention_util import HALF, inside, to_type
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import input_adaptive_bit_amd as G
    G.load()
    return require_gpu()


def make(rng, experts, d_in, d_out, group):
    groups = d_in // group
    q = rng.integers(0, 16, (experts, d_out, d_in)).astype(np.uint8)
    s = (rng.random((experts, d_out, groups)) * 0.01 + 0.001).astype(np.float16)
    z = (-8 * s.astype(np.float32) + 0.01 * rng.standard_normal(s.shape)).astype(np.float16)
    return q, s, z


def pack(q, s, z, dev):
    import input_adaptive_bit_amd as G
    import torch
    return G.fourbit_pack(*(torch.from_numpy(v).to(dev) for v in (q, s, z)))


def activations(rng, n, width, dtype):
    x = rng.standard_normal((n, width)).astype(np.float32)
    x *= np.where(rng.random(width) < 0.02, 8.0, 1.0).astype(np.float32)
    return A.bf16(x) if dtype == "bf16" else x


def bound(size, y, group, d_in, dtype):
    return (group + 3 * (d_in // group) + 32) * 2.0 ** -23 * size + HALF[dtype] * np.abs(y) + 1e-30


def check_linear(dev, rng, n, d_in, d_out, group, x_dtype, y_dtype, weight=None, packed=None):
    import input_adaptive_bit_amd as G
    import torch
    q, s, z = weight or make(rng, 1, d_in, d_out, group)
    w = packed or pack(q[0], s[0], z[0], dev)
    x = activations(rng, n, d_in, x_dtype)
    y = torch.full((n + 1, d_out), 7.0, dtype=torch.bfloat16 if y_dtype == "bf16" else torch.float32, device=dev)
    G.grinqh_fourbit_linear(w, to_type(x, x_dtype, dev), y[:n])
    want, size = O.linear(x, q[0], s[0], z[0], group)
    inside(y[:n].float().cpu().numpy(), want, bound(size, want, group, d_in, y_dtype))
    assert (y[n] == 7).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("experts,d_out,d_in", [(1, 1, 128), (1, 16, 128), (3, 37, 640), (2, 130, 384)])
def test_packed_layout_matches_the_oracle(dev, group, experts, d_out, d_in):
    say(f"fourbit_pack group={group} experts={experts} {d_in}->{d_out}")
    rng = np.random.default_rng(group + d_out)
    q, s, z = make(rng, experts, d_in - (group if d_in > 128 else 0), d_out, group)
    q = q + 16 * rng.integers(0, 16, q.shape).astype(np.uint8)                     # higher bits are masked
    w = pack(q, s, z, dev)
    assert np.array_equal(w.codes.cpu().numpy().view(np.uint32), O.packed_codes(q).ravel())
    assert np.array_equal(w.grid.cpu().numpy().view(np.uint16), O.packed_grid(s, z, group).ravel().view(np.uint16))


@pytest.mark.parametrize("group,d_in", [(32, 32), (32, 160), (64, 64), (64, 1344), (128, 128), (128, 2176)])
@pytest.mark.parametrize("n", [1, 2, 5, 6, 16, 17, 33, 65, 130, 300])
@pytest.mark.parametrize("x_dtype,y_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_products_match_the_oracle(dev, group, d_in, n, x_dtype, y_dtype):
    say(f"fourbit_linear n={n} d_in={d_in} group={group} {x_dtype}->{y_dtype}")
    check_linear(dev, np.random.default_rng(n + d_in), n, d_in, 8 * n % 61 + 52, group, x_dtype, y_dtype)


@pytest.mark.parametrize("d_out", [1, 2, 15, 16, 17, 31, 100, 129, 255, 256, 515])
@pytest.mark.parametrize("n", [1, 3, 40, 129])
def test_every_output_size(dev, d_out, n):
    say(f"fourbit_linear n={n} d_out={d_out}")
    rng = np.random.default_rng(d_out)
    for x_dtype, y_dtype in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")):
        check_linear(dev, rng, n, 256, d_out, 64, x_dtype, y_dtype)


@pytest.mark.parametrize("n,d_in,d_out,group", [(1, 4096, 4096, 128), (1, 14336, 4096, 64), (13, 4096, 14336, 128),
                                                (48, 8192, 1024, 32), (257, 4096, 1025, 128), (700, 1024, 2048, 32)])
def test_sizes_of_real_layers(dev, n, d_in, d_out, group):
    say(f"fourbit_linear n={n} {d_in}->{d_out} group={group}")
    check_linear(dev, np.random.default_rng(n), n, d_in, d_out, group, "bf16", "f32")


@pytest.mark.parametrize("x_dtype,n", [("bf16", 3), ("bf16", 7), ("bf16", 13), ("bf16", 90), ("f32", 1), ("f32", 4), ("f32", 7), ("f32", 13),
                                       ("f32", 40)])
@pytest.mark.parametrize("d_out,d_in,group", [(401, 288, 32), (8002, 192, 64), (12003, 256, 128)])
def test_few_and_many_outputs(dev, x_dtype, n, d_out, d_in, group):
    """Which kernel runs depends on the outputs too: narrow, wider and wide ones, with rows that do not fill them."""
    say(f"fourbit_linear n={n} {d_in}->{d_out} group={group} {x_dtype}")
    check_linear(dev, np.random.default_rng(n), n, d_in, d_out, group, x_dtype, "f32")


# Sizes whose products go through the tiles of 64 rows and of 128 rows: enough of them to fill the card.
TILED = [(1100, 2047), (2040, 4090)]


@pytest.mark.parametrize("n,d_out", TILED)
@pytest.mark.parametrize("group,d_in", [(32, 32), (32, 288), (64, 192), (64, 704), (128, 128), (128, 384), (128, 1152)])
def test_tiles_of_many_rows(dev, n, d_out, group, d_in):
    say(f"fourbit_linear n={n} {d_in}->{d_out} group={group}")
    for y_dtype in ("f32", "bf16"):
        check_linear(dev, np.random.default_rng(d_in), n, d_in, d_out, group, "bf16", y_dtype)


@pytest.mark.parametrize("n,d_out", TILED)
def test_tiles_of_strided_rows_results_off_alignment_and_values_that_are_not_finite(dev, n, d_out):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(n)
    q, s, z = make(rng, 1, 320, d_out, 64)
    w = pack(q[0], s[0], z[0], dev)
    x = to_type(activations(rng, n, 320, "bf16"), "bf16", dev)
    want = G.fourbit_linear(w, x, torch.float32)
    wide = torch.full((n + 50, 320 + 72), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:n, 64:384] = x
    flat = torch.full((n * d_out + 9,), 7.0, dtype=torch.float32, device=dev)
    for at in (0, 1, 5):
        y = flat[at:at + n * d_out].view(n, d_out)
        G.grinqh_fourbit_linear(w, wide[:n, 64:384], y)
        assert torch.equal(y, want) and (flat[:at] == 7).all() and (flat[at + n * d_out:] == 7).all()
        flat.fill_(7.0)
    x[3, 7], x[64, 319], x[n - 1, 0] = float("inf"), float("nan"), float("-inf")
    got = G.fourbit_linear(w, x, torch.float32)
    bad = [3, 64, n - 1]
    keep = torch.ones(n, dtype=torch.bool, device=dev)
    keep[bad] = False
    assert not torch.isfinite(got[bad]).any() and torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("counts,d_out", [([1, 0, 2, 19] + [0] * 60, 430), ([1, 0, 2, 9] + [0] * 60, 820), ([0, 3, 1, 1] * 16, 1023),
                                          ([12, 33, 0, 7], 3000), ([17, 33, 0, 50], 5001), ([700, 0, 600], 2050), ([1500, 540], 4000)])
@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gathered", [False, True])
def test_experts_of_many_outputs(dev, x_dtype, counts, d_out, gathered):
    """Few rows to many experts, more rows to few, tiles of many rows."""
    import input_adaptive_bit_amd as G
    import torch
    say(f"expert_linear counts={counts[:4]} d_out={d_out} {x_dtype} gathered={gathered}")
    rng = np.random.default_rng(d_out)
    q, s, z = make(rng, len(counts), 256, d_out, 32)
    w = pack(q, s, z, dev)
    n = sum(counts) + 6                                                            # rows of no run at both ends
    ends = np.concatenate([[2], 2 + np.cumsum(counts)]).astype(np.int32)
    n_x = 300 if gathered else n - 4                                               # fewer rows of x than of y: zeros
    x = activations(rng, n_x, 256, x_dtype)
    rows = rng.integers(-20, n_x + 20, n).astype(np.int32) if gathered else None
    y = torch.full((n, d_out), 7.0, dtype=torch.float32, device=dev)
    G.grinqh_expert_linear(w, to_type(x, x_dtype, dev), torch.from_numpy(ends).to(dev), y,
                           None if rows is None else torch.from_numpy(rows).to(dev))
    want, size, written = O.experts(x, ends, rows, n, q, s, z, 32)
    got = y.cpu().numpy()
    assert (got[~written] == 7).all() and not written.all()
    inside(got[written], want[written], bound(size[written], want[written], 32, 256, "f32"))


def test_tiles_in_a_graph_give_the_same_bits(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(8)
    q, s, z = make(rng, 1, 1024, 4096, 64)
    w = pack(q[0], s[0], z[0], dev)
    x = to_type(activations(rng, 2048, 1024, "bf16"), "bf16", dev)
    y, t = torch.empty(2048, 4096, device=dev), torch.empty(1100, 4096, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.grinqh_fourbit_linear(w, x, y)
        G.grinqh_fourbit_linear(w, x[:1100], t)
    other = torch.cuda.Stream()
    for turn in range(4):
        x.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), t.clone()
        other.wait_stream(torch.cuda.current_stream())
        G.grinqh_fourbit_linear(w, x, y)                                           # two calls at once
        G.grinqh_fourbit_linear(w, x[:1100], t, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], t)


def test_quantised_weights_are_the_rtn_of_each_group(dev):
    """fourbit_quantize against the weights' own rounding, and the product against both."""
    import input_adaptive_bit_amd as G
    import torch
    from oracle import grinqh_oracle as Q
    rng = np.random.default_rng(2)
    w = A.bf16(rng.standard_normal((3, 40, 256)).astype(np.float32) * 0.02)
    packed = G.fourbit_quantize(to_type(w, "bf16", dev), 64)
    q, s, z = Q.quantize_rtn(w.reshape(-1, 64), 4)
    q, s, z = q.reshape(w.shape), s.reshape(3, 40, 4), z.reshape(3, 40, 4)
    assert np.array_equal(packed.codes.cpu().numpy().view(np.uint32), O.packed_codes(q).ravel())
    assert np.array_equal(packed.grid.cpu().numpy().view(np.uint16), O.packed_grid(s, z, 64).ravel().view(np.uint16))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    again = G.fourbit_quantize(to_type(w, "bf16", dev), 64, stream=other)
    other.synchronize()
    assert torch.equal(again.codes, packed.codes) and torch.equal(again.grid, packed.grid)


@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [6, 14])
def test_rows_behind_the_last_do_not_matter(dev, x_dtype, n):
    """Columns that no row fills hold some row again: whatever lies behind x has no effect, and nothing behind y changes."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(n)
    q, s, z = make(rng, 1, 256, 9000, 64)
    w = pack(q[0], s[0], z[0], dev)
    x = to_type(activations(rng, n + 40, 256, x_dtype), x_dtype, dev)
    y = G.fourbit_linear(w, x[:n].clone(), torch.float32)
    x[n:] = float("nan")
    assert torch.equal(G.fourbit_linear(w, x[:n], torch.float32), y)


def ends_of(counts, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)


CASES = [
    # counts of each expert, rows before the first run, rows behind the last
    ([1], 0, 0), ([0, 0, 3], 0, 2), ([5, 0, 17, 1, 0], 3, 4), ([16, 32, 33, 64, 65], 0, 0), ([0, 0, 0], 2, 2),
    ([129, 0, 1, 300], 1, 0), ([1] * 70, 0, 5), ([0] * 130 + [2, 0, 40] + [1] * 30, 0, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("x_dtype,group,d_in,d_out", [("bf16", 128, 384, 70), ("bf16", 32, 160, 256), ("f32", 64, 192, 33)])
def test_experts_match_the_oracle(dev, case, gathered, x_dtype, group, d_in, d_out):
    import input_adaptive_bit_amd as G
    import torch
    counts, lead, tail = CASES[case]
    say(f"expert_linear case={case} gathered={gathered} {x_dtype} group={group} {d_in}->{d_out}")
    rng = np.random.default_rng(case)
    q, s, z = make(rng, len(counts), d_in, d_out, group)
    w = pack(q, s, z, dev)
    n = lead + sum(counts) + tail
    n_x = 11 if gathered else n
    x = activations(rng, n_x, d_in, x_dtype)
    rows = rng.integers(-1, n_x + 1, n).astype(np.int32) if gathered else None     # some name no row
    ends = ends_of(counts, lead)
    y = torch.full((n, d_out), 7.0, dtype=torch.float32, device=dev)
    G.grinqh_expert_linear(w, to_type(x, x_dtype, dev), torch.from_numpy(ends).to(dev), y,
                           None if rows is None else torch.from_numpy(rows).to(dev))
    want, size, written = O.experts(x, ends, rows, n, q, s, z, group)
    want[~written] = 7.0
    inside(y.cpu().numpy(), want, bound(size, want, group, d_in, "f32"))
    assert (y.cpu().numpy()[~written] == 7).all()


def test_many_rows_to_few_experts(dev):
    """Runs that take every kind of tile, in bf16 and fp32 outputs."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(0)
    counts = [700, 3, 0, 513]
    q, s, z = make(rng, 4, 512, 300, 128)
    w = pack(q, s, z, dev)
    x = activations(rng, sum(counts), 512, "bf16")
    ends = ends_of(counts)
    want, size, _ = O.experts(x, ends, None, len(x), q, s, z, 128)
    for dtype in ("bf16", "f32"):
        y = G.expert_linear(w, to_type(x, "bf16", dev), torch.from_numpy(ends).to(dev),
                            out_dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
        inside(y.float().cpu().numpy(), want, bound(size, want, 128, 512, dtype))


def test_ends_outside_the_rows_are_clamped(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(1)
    q, s, z = make(rng, 3, 128, 16, 32)
    w = pack(q, s, z, dev)
    x = activations(rng, 20, 128, "bf16")
    ends = np.array([-5, 7, 2 ** 31 - 1, 2 ** 31 - 1], np.int32)
    y = G.expert_linear(w, to_type(x, "bf16", dev), torch.from_numpy(ends).to(dev), out_dtype=torch.float32)
    want, size, written = O.experts(x, ends, None, 20, q, s, z, 32)
    assert written.all()
    inside(y.cpu().numpy(), want, bound(size, want, 32, 128, "f32"))


@pytest.mark.parametrize("n", [3, 40, 200])
def test_strided_rows_and_a_result_that_is_not_aligned(dev, n):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(n)
    q, s, z = make(rng, 1, 256, 36, 128)
    w = pack(q[0], s[0], z[0], dev)
    x = activations(rng, n, 256, "bf16")
    wide = torch.full((n, 256 + 72), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 64:320] = to_type(x, "bf16", dev)
    flat = torch.full((n * 36 + 9,), 7.0, dtype=torch.bfloat16, device=dev)
    for at in (0, 1, 5):
        y = flat[at:at + n * 36].view(n, 36)
        G.grinqh_fourbit_linear(w, wide[:, 64:320], y)
        want, size = O.linear(x, q[0], s[0], z[0], 128)
        inside(y.float().cpu().numpy(), want, bound(size, want, 128, 256, "bf16"))
        assert (flat[at + n * 36:] == 7).all()
        flat.fill_(7.0)


@pytest.mark.parametrize("n,x_dtype", [(4, "bf16"), (20, "bf16"), (150, "bf16"), (7, "f32")])
def test_what_is_not_finite_stays_in_its_row(dev, n, x_dtype):
    """An infinite or NaN activation makes its own row non-finite and leaves the others' bits alone."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(n)
    q, s, z = make(rng, 1, 384, 50, 64)
    w = pack(q[0], s[0], z[0], dev)
    x = activations(rng, n, 384, x_dtype)
    clean = G.fourbit_linear(w, to_type(x, x_dtype, dev), torch.float32)
    bad = x.copy()
    bad[1, 7], bad[2, 383] = np.inf, np.nan
    got = G.fourbit_linear(w, to_type(bad, x_dtype, dev), torch.float32)
    assert not torch.isfinite(got[1:3]).any()
    keep = [i for i in range(n) if i not in (1, 2)]
    assert torch.equal(got[keep], clean[keep])


def test_fp32_activations_keep_their_bits(dev):
    """Values that no bf16 holds, large, tiny and of both signs: the products see all 24 bits."""
    import input_adaptive_bit_amd as G
    rng = np.random.default_rng(9)
    d_in = 128
    q, s, z = np.full((1, 16, d_in), 3, np.uint8), np.ones((1, 16, 1), np.float16), np.full((1, 16, 1), -3.5, np.float16)
    q[0, np.arange(16), np.arange(16)] = 4                                           # w = 1 at (j, j), 0 elsewhere
    w = pack(q[0], s[0], z[0], dev)
    x = np.zeros((16, d_in), np.float32)
    values = (rng.standard_normal(16) * 10.0 ** rng.integers(-25, 30, 16)).astype(np.float32)
    for j in range(16):
        x[j, j] = values[j]
    y = G.fourbit_linear(w, to_type(x, "f32", dev), to_type(x, "f32", dev).dtype).cpu().numpy()
    # 20 x and 19.5 x are two roundings of a value 20 times as large
    assert np.all(np.abs(np.diagonal(y).astype(np.float64) - values) <= 3 * 20 * 2.0 ** -23 * np.abs(values))


def test_same_call_same_bits_and_graph_replays(dev):
    """Products captured in a graph, replayed between the program's own work, on changed inputs."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(4)
    q, s, z = make(rng, 4, 512, 96, 128)
    w = pack(q, s, z, dev)
    one = G.FourbitWeight(G.grinqh_fourbit_layout_init(512, 96, 128), w.codes, w.grid)       # the first expert alone
    x = to_type(activations(rng, 90, 512, "bf16"), "bf16", dev)
    ends = torch.tensor([0, 40, 41, 41, 90], dtype=torch.int32, device=dev)
    y, t = torch.empty(90, 96, device=dev), torch.empty(3, 96, device=dev)

    def step():
        G.grinqh_expert_linear(w, x, ends, y)
        G.grinqh_fourbit_linear(one, x[:3], t)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        x.copy_(to_type(activations(rng, 90, 512, "bf16"), "bf16", dev))
        ends.copy_(torch.tensor([0, 40 - 9 * turn, 41, 41 + turn, 90], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), t.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], t)


def test_another_stream(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(6)
    q, s, z = make(rng, 1, 256, 64, 128)
    w = pack(q[0], s[0], z[0], dev)
    x = to_type(activations(rng, 8, 256, "bf16"), "bf16", dev)
    want = G.fourbit_linear(w, x, torch.float32)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for stream in (other, other.cuda_stream):
        got = G.fourbit_linear(w, x, torch.float32, stream)
        other.synchronize()
        assert torch.equal(got, want)


def test_no_rows_and_no_tokens(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(6)
    q, s, z = make(rng, 2, 128, 16, 32)
    w, one = pack(q, s, z, dev), pack(q[0], s[0], z[0], dev)
    none = torch.empty(0, 128, dtype=torch.bfloat16, device=dev)
    assert G.fourbit_linear(one, none).shape == (0, 16)
    ends = torch.zeros(3, dtype=torch.int32, device=dev)
    rows = torch.empty(0, dtype=torch.int32, device=dev)
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device=dev)
    assert G.expert_linear(w, x, ends, rows).shape == (0, 16)
    assert G.expert_linear(w, none, ends).shape == (0, 16)
