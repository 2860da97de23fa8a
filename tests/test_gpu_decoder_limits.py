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
