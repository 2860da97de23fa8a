"""The 4-bit products and what goes with them at the ends of their ranges (GPU).
Bounds as in test_gpu_fourbit.py."""

import numpy as np
import pytest

from tests.gpu_util import require_gpu, say
from tests.test_gpu_fourbit import check_linear

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
    from oracle import decoder_oracle as O
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
