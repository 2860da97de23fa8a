"""What the 4-bit products' and the pages' calls do at the ends of their ranges,
without a GPU."""

import pytest

import input_adaptive_bit_amd as G
from tests.test_decoder_cpu import Fake


# ----------------------------------------------------------------- weights --

def test_weights_of_very_many_groups_are_rounded_in_pieces(monkeypatch):
    """grinqh_quantize_rtn takes 2^30 rows; 1024 experts of 4096 to 16384 in groups of 32 have twice as many."""
    import torch
    from input_adaptive_bit_amd import fourbit
    sent, packed = [], []
    monkeypatch.setattr(torch, "Tensor", Fake)
    monkeypatch.setattr(fourbit, "_run", lambda name, device, stream, *a: sent.append((name, stream, *a)))
    monkeypatch.setattr(fourbit, "_empty", lambda shape, dtype, device, stream: Fake(*shape, dtype=dtype))
    monkeypatch.setattr(fourbit, "fourbit_pack", lambda q, s, z, stream: packed.append((q, s, z, stream)))
    for shape, group in (((1024, 16384, 4096), 32), ((2 ** 20, 2 ** 15 + 32), 32), ((40, 256), 128)):
        rows = Fake(*shape).numel() // group
        fourbit.fourbit_quantize(Fake(*shape), group, 7)
        at = 0
        for name, stream, d_in, n, bits, w, q, s, z in sent:
            assert (name, stream, d_in, bits) == ("grinqh_quantize_rtn", 7, group, 4) and 1 <= n <= 1 << 30
            assert (w - 4096, q - 4096, s - 4096, z - 4096) == (2 * at * group, at * group, 2 * at, 2 * at)
            at += n
        assert at == rows
        q, s, z, stream = packed.pop()
        assert stream == 7 and q.shape == shape and s.shape == z.shape == (*shape[:-1], shape[-1] // group)
        sent.clear()


def test_weights_that_cannot_be_rounded_are_refused(monkeypatch):
    import torch
    from input_adaptive_bit_amd import attention, fourbit
    sent = []
    monkeypatch.setattr(torch, "Tensor", Fake)
    monkeypatch.setattr(fourbit, "_empty", lambda shape, dtype, device, stream: Fake(*shape, dtype=dtype))
    monkeypatch.setattr(attention, "load", lambda: type("Lib", (), {"grinqh_quantize_rtn": lambda *a: sent.append(a)}))
    for bad in (Fake(64, 128, dtype=torch.float32), Fake(64, 128, dtype=torch.float16)):
        with pytest.raises(TypeError):
            fourbit.fourbit_quantize(bad, 32)
    for bad, group in ((Fake(64, 128, stride=(1, 64)), 32), (Fake(64, 128, stride=(256, 1)), 128), (Fake(128), 32), (Fake(64, 120), 32),
                       (Fake(64, 128), 0)):
        with pytest.raises(ValueError):
            fourbit.fourbit_quantize(bad, group)
    far = type("Stream", (), {"cuda_stream": 5, "device": torch.device("cuda:1")})
    with pytest.raises(ValueError, match="stream"):
        fourbit.fourbit_quantize(Fake(64, 128), 32, far)
    assert not sent


# ---------------------------------------------------------------- products --

def _no_gpu():
    import torch
    return not torch.cuda.is_available()


@pytest.mark.skipif(not _no_gpu(), reason="without a GPU a call that passes its checks ends at the launch; with one it would run on these addresses")
@pytest.mark.parametrize("experts,rows,d_in,d_out", [(1024, 65536, 32, 1 << 20), (1024, 66000, 32, (1 << 20) - 3), (2, 1 << 20, 64, 1 << 18),
                                                     (1, 1 << 20, 32, 1 << 20), (1, 40, 32, 16), (8, 4094, 4096, 14336)])
def test_no_size_of_the_layout_is_refused(experts, rows, d_in, d_out):
    """Experts' runs that could have more tiles than a launch has workgroups are a call like any other."""
    import ctypes
    from input_adaptive_bit_amd import grinqh as B
    L = G.grinqh_fourbit_layout_init(d_in, d_out, 32, experts)
    at = [(i + 1) << 44 for i in range(6)]                                             # places that nothing overlaps
    for x_dtype in (B.GRINQH_BF16, B.GRINQH_F32):
        a = B.ExpertArgs(at[0], d_in, x_dtype, rows, at[1], at[2], rows, at[3], at[4], at[5], B.GRINQH_BF16)
        assert B.load().grinqh_expert_linear(ctypes.byref(L), ctypes.byref(a), None) in (B.GRINQH_ENODEV, B.GRINQH_EDEVICE)
        if experts == 1:
            status = B.load().grinqh_fourbit_linear(ctypes.byref(L), at[0], x_dtype, d_in, rows, at[3], at[4], at[5], B.GRINQH_BF16, None)
            assert status in (B.GRINQH_ENODEV, B.GRINQH_EDEVICE)


# ------------------------------------------------------------------- pages --

def test_a_request_that_can_never_be_served_takes_nothing_from_those_behind_it():
    """Pages of 16, 3 columns, a pool of 6 pages with 2 unused: 49 tokens pass the columns, 7 pages pass the pool."""
    from oracle import decoder_oracle as O
    free = [5, 3, -1, -1, -1, -1]
    got = O.extend([[-1] * 3] * 4, [0, 0, 0, 0], [49, 16, 0, 10], free, 2, 16, 80)
    assert got["refused"] == 1 and got["seq_lens"].tolist() == [0, 16, 0, 10] and got["n_free"] == 0
    assert got["table"].tolist() == [[-1] * 3, [3, -1, -1], [-1] * 3, [5, -1, -1]]
    assert got["slots"].tolist() == [-1] * 49 + list(range(48, 64)) + list(range(80, 90)) + [-1] * 5
    assert got["cu_q"].tolist() == [0, 49, 65, 65, 75] and got["cu_k"].tolist() == [0, 0, 16, 16, 26]
    got = O.extend([[-1] * 9] * 3, [0, 0, 0], [97, 33, 16], free, 2, 16, 200)
    # seven pages are more than the pool has; three are more than the list holds, and come before the next request
    assert got["refused"] == 3 and got["seq_lens"].tolist() == [0, 0, 0]
    got = O.extend([[-1] * 9] * 3, [0, 0, 0], [97, 17, 16], free, 2, 16, 200)
    assert got["refused"] == 2 and got["seq_lens"].tolist() == [0, 17, 0] and got["table"][1].tolist() == [3, 5] + [-1] * 7


def test_row_counts_past_32_bits_are_refused(monkeypatch):
    """2^32 + 5 rows of one weight are not five."""
    import torch
    from input_adaptive_bit_amd import grinqh
    monkeypatch.setattr(torch, "Tensor", Fake)
    size_of = {torch.bfloat16: 2, torch.uint8: 1, torch.float16: 2}
    monkeypatch.setattr(Fake, "element_size", lambda self: size_of[self.dtype], raising=False)
    for d_out, d_in in ((2 ** 32 + 5, 1), (2 ** 31, 32), (2 ** 30 + 1, 32), (5, 2 ** 32 + 16)):
        n = d_out * d_in
        q, s = Fake(n, dtype=torch.uint8), Fake(d_out, dtype=torch.float16)
        with pytest.raises(G.GrinqhError) as e:
            grinqh.grinqh_quantize_rtn(Fake(d_out, d_in), 4, q, s, s, stream=3)
        assert e.value.status == grinqh.GRINQH_EINVAL
