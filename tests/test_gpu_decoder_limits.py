"""The 4-bit products and what goes with them at the ends of their ranges (GPU).
Bounds as in test_gpu_fourbit.py."""

import numpy as np
import pytest

from oracle import decoder_oracle as O
from tests.attention_util import inside, to_type
from tests.gpu_util import require_gpu, say
from tests.test_gpu_fourbit import activations, bound, check_linear, make, pack
from tests.test_gpu_pages import pool, run, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import input_adaptive_bit_amd as G
    G.load()
    return require_gpu()


# ------------------------------------------------------------ 4-bit products --

@pytest.mark.parametrize("n,d_in,group", [(1, 8192, 128), (1, 16640, 128), (1, 25216, 64), (1, 8256, 32), (2, 4096, 128), (4, 8320, 128),
                                          (5, 12480, 64), (5, 4128, 32), (5, 13024, 32)])
def test_fp32_rows_of_many_inputs(dev, n, d_in, group):
    """A wave's pieces of a few fp32 rows pass through its LDS several times over: each time every lane reads what the
    others wrote, and nobody overwrites what is still to be read."""
    say(f"fourbit_linear n={n} {d_in}->40 group={group} f32")
    check_linear(dev, np.random.default_rng(d_in), n, d_in, 40, group, "f32", "f32")


# ----------------------------------------------------------------- weights --

def test_more_rows_to_round_than_a_launch_has_workgroups(dev):
    """2^24 rows and more, a workgroup each, would be 2^32 work items."""
    import input_adaptive_bit_amd as G
    import torch
    from oracle import grinqh_oracle as Q
    n = (1 << 24) + 1003
    say(f"quantize_rtn {n} rows of 32")
    w = torch.randn(n, 32, generator=torch.Generator(device=dev).manual_seed(1), device=dev, dtype=torch.bfloat16)
    got = G.quantize_rtn(w, 4)
    for at in (0, (1 << 20) - 5, (1 << 23) - 5, (1 << 24) - 5, n - 10):
        want = Q.quantize_rtn(w[at:at + 10].float().cpu().numpy(), 4)
        for a, b in zip(got, want):
            assert np.array_equal(a[at:at + 10].cpu().numpy(), b), at


def test_experts_of_more_groups_than_a_launch_has_workgroups(dev):
    import input_adaptive_bit_amd as G
    import torch
    from oracle import grinqh_oracle as Q
    experts, d_out, d_in, group = 2, 16 * 16385, 1024, 32
    assert experts * d_out * d_in // group > 1 << 24
    say(f"fourbit_quantize {experts} experts {d_in}->{d_out} group={group}")
    w = torch.randn(experts, d_out, d_in, generator=torch.Generator(device=dev).manual_seed(2), device=dev, dtype=torch.bfloat16)
    packed = G.fourbit_quantize(w, group)
    codes = packed.codes.view(experts, d_out // 16, -1)
    grid = packed.grid.view(experts, d_out // 16, -1)
    for e, tile in ((0, 0), (0, 16384), (1, 0), (1, 16383), (1, 16384)):
        rows = w[e, 16 * tile:16 * tile + 16].float().cpu().numpy()
        q, s, z = Q.quantize_rtn(rows.reshape(-1, group), 4)
        assert np.array_equal(codes[e, tile].cpu().numpy().view(np.uint32), O.packed_codes(q.reshape(1, 16, d_in)).ravel()), (e, tile)
        want = O.packed_grid(s.reshape(1, 16, -1), z.reshape(1, 16, -1), group)
        assert np.array_equal(grid[e, tile].cpu().numpy().view(np.uint16), want.ravel().view(np.uint16)), (e, tile)


# ------------------------------------------------------------ the largest calls --

@pytest.mark.parametrize("n", [16 * 32768, 16 * 32768 + 1, 16 * 34002 - 5, 1 << 20])
@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
def test_rows_past_a_launchs_second_dimension(dev, n, x_dtype):
    say(f"fourbit_linear n={n} 32->16 {x_dtype}")
    check_linear(dev, np.random.default_rng(n), n, 32, 16, 32, x_dtype, "f32")


@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
def test_experts_rows_past_a_launchs_second_dimension(dev, x_dtype):
    import input_adaptive_bit_amd as G
    import torch
    say(f"expert_linear 2^20 - 3 rows to 5 experts {x_dtype}")
    rng = np.random.default_rng(3)
    n, counts = (1 << 20) - 3, [524283, 0, 13, 500000, 24000]
    ends = np.concatenate([[5], 5 + np.cumsum(counts)]).astype(np.int32)
    q, s, z = make(rng, 5, 32, 16, 32)
    x = activations(rng, 1000, 32, x_dtype)
    rows = rng.integers(-3, 1003, n).astype(np.int32)
    y = torch.full((n, 16), 7.0, dtype=torch.float32, device=dev)
    G.grinqh_expert_linear(pack(q, s, z, dev), to_type(x, x_dtype, dev), torch.from_numpy(ends).to(dev), y, torch.from_numpy(rows).to(dev))
    want, size, written = O.experts(x, ends, rows, n, q, s, z, 32)
    want[~written] = 7.0
    inside(y.cpu().numpy(), want, bound(size, want, 32, 32, "f32"))


def test_results_of_more_than_2_to_the_32_values(dev):
    """Through the tiles (bf16) and the other kernel, whose three dimensions then have more than 2^32 work items together."""
    import input_adaptive_bit_amd as G
    import torch
    n, d_out = 65536 + 17, 1 << 18
    rng = np.random.default_rng(4)
    q, s, z = make(rng, 1, 32, d_out, 32)
    w = pack(q[0], s[0], z[0], dev)
    x = activations(rng, n, 32, "bf16")
    y = torch.empty(n, d_out, dtype=torch.bfloat16, device=dev)
    at = [0, 4095, 8191, 8192, 16384, 32768, 40001, 65535, 65536, n - 1]
    want, size = O.linear(x[at], q[0], s[0], z[0], 32)
    for x_dtype in ("bf16", "f32"):
        say(f"fourbit_linear n={n} 32->{d_out} {x_dtype}")
        y.fill_(float("nan"))
        G.grinqh_fourbit_linear(w, to_type(x, x_dtype, dev), y)
        inside(y[at].float().cpu().numpy(), want, bound(size, want, 32, 32, "bf16"))
        assert all(torch.isfinite(y[i:i + 4096]).all() for i in range(0, n, 4096))


def test_experts_whose_weights_lie_past_4_gib(dev):
    import input_adaptive_bit_amd as G
    import torch
    experts, d_in, d_out, group = 72, 4096, 32768, 128
    say(f"expert_linear to {experts} experts {d_in}->{d_out}")
    g = torch.Generator(device=dev).manual_seed(5)
    q = torch.randint(0, 16, (experts, d_out, d_in), dtype=torch.uint8, device=dev, generator=g)
    s = (torch.rand(experts, d_out, d_in // group, device=dev, generator=g) * 0.01 + 0.001).half()
    z = (-8 * s.float()).half()
    w = G.fourbit_pack(q, s, z)
    assert w.codes.nbytes > 1 << 32
    rng = np.random.default_rng(5)
    for each in (3, 2000):                                                            # the kernel of few rows, and tiles
        counts = np.zeros(experts, np.int64)
        counts[[0, 33, 34, 64, 71]] = each
        ends = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
        x = to_type(activations(rng, int(counts.sum()), d_in, "bf16"), "bf16", dev)
        y = G.expert_linear(w, x, ends, out_dtype=torch.float32)
        for e in (0, 33, 34, 64, 71):
            at = torch.arange(int(ends[e]), int(ends[e + 1]), device=dev)[[0, 1, -1]]
            for j in (0, d_out - 512):
                want, size = O.linear(x[at].float().cpu().numpy(), *(v[e, j:j + 512].cpu().numpy() for v in (q, s, z)), group)
                inside(y[at, j:j + 512].cpu().numpy(), want, bound(size, want, group, d_in, "f32"))


@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d_out", [(1, 50), (3, 50), (6, 9000), (14, 9000), (40, 50), (200, 515), (1100, 2047)])
def test_nothing_behind_the_rows_is_read_or_written(dev, x_dtype, n, d_out):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(n)
    q, s, z = make(rng, 1, 256, d_out, 64)
    w = pack(q[0], s[0], z[0], dev)
    x = to_type(activations(rng, n + 140, 256, x_dtype), x_dtype, dev)
    alone = G.fourbit_linear(w, x[:n].clone(), torch.float32)
    x[n:] = float("nan")
    y = torch.full((n + 140, d_out), 7.0, dtype=torch.float32, device=dev)
    G.grinqh_fourbit_linear(w, x[:n], y[:n])
    assert torch.equal(y[:n], alone) and (y[n:] == 7).all()


@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,d_in", [(32, 160), (64, 192), (128, 128), (128, 1024)])
@pytest.mark.parametrize("n,d_out", [(1, 50), (4, 50), (7, 50), (14, 9000), (1100, 2047)])
def test_the_largest_activations(dev, x_dtype, group, d_in, n, d_out):
    """Groups full of +-2^115 against codes of 15: their sums with 16 + q are 128 * 31 * 2^115, inside fp32's range."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(n)
    q, s, z = make(rng, 1, d_in, d_out, group)
    q[0, :d_out // 2], s[:] = 15, 2.0 ** -4
    x = (2.0 ** 115 * rng.choice([-1.0, 1.0], (n, d_in))).astype(np.float32)
    x[::2] = 2.0 ** 115
    y = G.fourbit_linear(pack(q[0], s[0], z[0], dev), to_type(x, x_dtype, dev), torch.float32).cpu().numpy()
    want, size = O.linear(x, q[0], s[0], z[0], group)
    inside(y, want, bound(size, want, group, d_in, "f32"))


# ------------------------------------------------------------------- pages --

@pytest.mark.parametrize("batch", [5, 300, 1500])
@pytest.mark.parametrize("capacity", [2000, 60000])
@pytest.mark.parametrize("in_place", [False, True])
def test_requests_that_can_never_be_served_starve_nobody(dev, batch, capacity, in_place):
    """Requests past the table's columns, and past the whole pool, among ordinary ones that the list can serve."""
    rng = np.random.default_rng(batch)
    lens, new = rng.integers(0, 60, batch), rng.integers(1, 20, batch)
    if capacity == 2000:
        new = np.where(np.arange(batch) < 60, new, 0)
    new[0], new[2] = 1000, 161                                                        # 63 and 11 pages of 16
    lens[0], lens[2] = 0, 0
    for columns, n_pages, spare in ((10, None, 3 * batch), (100, None, 3 * batch), (100, None, 2), (10, None, 7)):
        table, free, n_free = pool(rng, lens, 16, columns, spare, n_pages)
        want = O.extend(table, lens, new, free, n_free, 16, capacity)
        say(f"kv_extend batch={batch} capacity={capacity} columns={columns} free={n_free} refused={want['refused']}")
        got = run(dev, table, lens, new, free, n_free, 16, capacity, in_place)
        same(got, want)
        if columns == 10 and spare > batch:
            assert got["refused"] == 2 and (got["seq_lens"][3:] == (lens + new)[3:]).all()
    few = np.array([0, 0, 3, 16][:batch])
    for n_free in (0, 1, 2, 5):                                                       # a pool of five pages
        table, free = np.full((4, 9), -1, np.int32), np.array([4, 0, 2, 1, 3], np.int32)
        table[2, 0], table[3, 0] = 1, 3
        same(run(dev, table, few, [81, 17, 14, 1], free, n_free, 16, 200, in_place), O.extend(table, few, [81, 17, 14, 1], free, n_free, 16, 200))
