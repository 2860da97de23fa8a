"""GPU parity of the key-value cache (grinqh_kv_write, grinqh_kv_read) with the
CPU oracle: stored bytes and grids bit-identical, values read back exact."""

import numpy as np
import pytest

from oracle import attention_oracle as A
from tests.attention_util import rows, to_type
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import input_adaptive_bit_amd as G
    G.load()
    return require_gpu()


def _cache(heads, dim, page, n_pages, bits, dev, fill=0x5A):
    """A cache whose bytes are all `fill`, so that what is not to be written shows."""
    import input_adaptive_bit_amd as G
    c = G.new_kv_cache(heads, dim, page, n_pages, bits, dev)
    for t in (c.k_codes, c.v_codes):
        t.fill_(fill)
    for t in (c.k_grid, c.v_grid):
        if t is not None:
            t.fill_(-7.0)
    return c


def _same_halves(a, b):
    a, b = np.asarray(a, np.float16), np.asarray(b, np.float16)
    return np.all((np.isnan(a) & np.isnan(b)) | (a.view(np.uint16) == b.view(np.uint16)))


def _check(c, k, v, slots, bits, fill=0x5A):
    """The whole pool: written rows as the oracle has them, the others untouched."""
    L = c.layout
    for w, codes, grid in ((k, c.k_codes, c.k_grid), (v, c.v_codes, c.v_grid)):
        stored, g = A.quantise_rows(w, bits)
        want = np.full((L.n_pages, L.n_kv_heads, L.page_size, L.row_bytes), fill, np.uint8)
        want_g = np.full((L.n_pages, L.n_kv_heads, L.page_size, 2), -7.0, np.float16)
        for t, slot in enumerate(slots):
            if 0 <= slot < L.n_pages * L.page_size:
                want[slot // L.page_size, :, slot % L.page_size] = stored[t]
                if g is not None:
                    want_g[slot // L.page_size, :, slot % L.page_size] = g[t]
        assert np.array_equal(codes.cpu().numpy(), want)
        if bits < 16:
            assert _same_halves(grid.cpu().numpy(), want_g)


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 8, 128, 64), (1, 1, 64, 16), (37, 3, 64, 16), (130, 5, 128, 32),
                                                   (65, 2, 256, 256), (300, 8, 128, 128)])
def test_written_rows_match_the_oracle_and_read_back(dev, bits, dtype, tokens, heads, dim, page):
    import input_adaptive_bit_amd as G
    import torch
    say(f"kv_write bits={bits} {dtype} tokens={tokens} heads={heads} dim={dim} page={page}")
    rng = np.random.default_rng(tokens + heads + dim + bits)
    kv = [rng.standard_normal((tokens, heads, dim)).astype(np.float32) if dtype == "f32" else
          rows(rng, tokens, heads, dim) for _ in range(2)]
    n_pages = -(-tokens // page) + 2
    slots = rng.permutation(n_pages * page)[:tokens]
    c = _cache(heads, dim, page, n_pages, bits, dev)
    s = torch.from_numpy(slots).to(dev)
    G.kv_write(c, *(to_type(x, dtype, dev) for x in kv), s)
    torch.cuda.synchronize()
    _check(c, *kv, slots, bits)
    for w, f32, b16 in zip(kv, G.kv_read(c, s, torch.float32), G.kv_read(c, s)):
        stored, grid = A.quantise_rows(w, bits)
        want = A.row_values(stored, grid, bits).astype(np.float32)     # one rounding of the exact value
        assert np.array_equal(f32.cpu().numpy(), want)
        assert np.array_equal(b16.float().cpu().numpy(), A.bf16(want))


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_slots_outside_the_pool_are_skipped_and_read_as_zeros(dev, bits):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(bits)
    heads, dim, page, n_pages = 3, 64, 16, 4
    slots = np.array([5, -1, 63, 64, 2 ** 40, -2 ** 62, 0, 17], np.int64)
    kv = [rows(rng, len(slots), heads, dim) for _ in range(2)]
    c = _cache(heads, dim, page, n_pages, bits, dev)
    s = torch.from_numpy(slots).to(dev)
    G.kv_write(c, *(to_type(x, "bf16", dev) for x in kv), s)
    torch.cuda.synchronize()
    _check(c, *kv, slots, bits)
    again = torch.from_numpy(np.concatenate([slots, slots[::-1]])).to(dev)       # any order, more than once
    for w, got in zip(kv, G.kv_read(c, again, torch.float32)):
        want = A.row_values(*A.quantise_rows(w, bits), bits).astype(np.float32)
        want[(slots < 0) | (slots >= n_pages * page)] = 0.0
        assert np.array_equal(got.cpu().numpy(), np.concatenate([want, want[::-1]]))


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_that_are_not_ordinary(dev, bits):
    """Constant, zero, tiny, huge, NaN and infinite rows go as the oracle's do."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(3)
    w = rng.standard_normal((12, 1, 64)).astype(np.float32)
    w[0], w[1], w[2], w[3] = 0.0, -0.0, 2.5, -3e-8
    w[4] *= 1e-7
    w[5] *= 1e30
    w[6, 0, 3], w[6, 0, 60] = np.nan, np.nan
    w[7] = np.nan
    w[8, 0, 1] = np.inf
    w[9, 0, 0] = -np.inf
    w[10] = np.linspace(-1, 1, 64, dtype=np.float32)
    w[11, 0, :2] = [np.inf, -np.inf]
    slots = np.arange(12, dtype=np.int64)
    c = _cache(1, 64, 16, 1, bits, dev)
    t = torch.from_numpy(w).to(dev)
    with np.errstate(all="ignore"):
        G.kv_write(c, t, t, torch.from_numpy(slots).to(dev))
        torch.cuda.synchronize()
        _check(c, w, w, slots, bits)


def test_slices_of_a_fused_projection(dev):
    """k and v as views of [tokens][q | k | v] rows, on their own strides."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(9)
    tokens, n_q, heads, dim = 21, 4, 2, 128
    fused = rows(rng, tokens, n_q + 2 * heads, dim)
    t = to_type(fused, "bf16", dev)
    slots = rng.permutation(48)[:tokens].astype(np.int64)
    c = _cache(heads, dim, 16, 3, 8, dev)
    G.kv_write(c, t[:, n_q:n_q + heads], t[:, n_q + heads:], torch.from_numpy(slots).to(dev))
    torch.cuda.synchronize()
    _check(c, fused[:, n_q:n_q + heads], fused[:, n_q + heads:], slots, 8)


def test_no_tokens(dev):
    import input_adaptive_bit_amd as G
    import torch
    c = _cache(2, 64, 16, 1, 8, dev)
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=dev)
    G.kv_write(c, none, none, torch.zeros(0, dtype=torch.int64, device=dev))
    k, v = G.kv_read(c, torch.zeros(0, dtype=torch.int64, device=dev))
    assert k.shape == v.shape == (0, 2, 64)
    assert bool((c.k_codes == 0x5A).all())


@pytest.mark.parametrize("bits", [4, 16])
def test_more_rows_than_one_round_of_workgroups(dev, bits):
    """520 tokens of 1024 heads of 256: over 2^19 rows of 8 to a workgroup."""
    import input_adaptive_bit_amd as G
    import torch
    tokens, heads, dim, page = 520, 1024, 256, 16
    g = torch.Generator(device=dev).manual_seed(1)
    k = torch.randn(tokens, heads, dim, generator=g, device=dev).bfloat16()
    slots = torch.randperm(33 * page, generator=g, device=dev)[:tokens]
    c = G.new_kv_cache(heads, dim, page, 33, bits, dev)
    G.kv_write(c, k, k, slots)
    got, _ = G.kv_read(c, slots, torch.float32)
    for t in (0, 1, 255, 256, 257, 511, 512, 519):
        w = k[t].float().cpu().numpy()
        assert np.array_equal(got[t].cpu().numpy(), A.row_values(*A.quantise_rows(w, bits), bits).astype(np.float32))
    if bits == 16:
        assert torch.equal(got, k.float())


def test_pool_of_more_than_four_gigabytes(dev):
    import input_adaptive_bit_amd as G
    import torch
    heads, dim, page, n_pages = 8, 256, 256, 4400                     # 4.6 GB of bf16 keys
    c = G.new_kv_cache(heads, dim, page, n_pages, 16, dev)
    assert c.k_codes.numel() > 2 ** 32
    total = page * n_pages
    slots = torch.tensor([total - 1, 0, total // 2, 2 ** 20 + 3, total], device=dev)
    g = torch.Generator(device=dev).manual_seed(2)
    k = torch.randn(5, heads, dim, generator=g, device=dev).bfloat16()
    G.kv_write(c, k, -k, slots)
    got_k, got_v = G.kv_read(c, slots)
    k[4] = 0
    assert torch.equal(got_k, k) and torch.equal(got_v, -k)
    last = c.k_codes.view(torch.bfloat16)[-1, :, -1]
    assert torch.equal(last, k[0])


def test_write_and_read_on_another_stream_and_in_a_graph(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(5)
    c = _cache(2, 64, 16, 2, 8, dev)
    k = to_type(rows(rng, 4, 2, 64), "bf16", dev)
    slots = torch.tensor([3, 9, 20, -1], device=dev)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    G.kv_write(c, k, k, slots, stream=other)
    got, _ = G.kv_read(c, slots, torch.float32, stream=other)
    other.synchronize()
    want = A.row_values(*A.quantise_rows(k.float().cpu().numpy(), 8), 8).astype(np.float32)
    want[3] = 0
    assert np.array_equal(got.cpu().numpy(), want)
    out_k, out_v = torch.empty_like(k), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.kv_write(c, k, k, slots)
        G.grinqh_kv_read(c, slots, out_k, out_v)
    for seed in range(3):
        w = rows(np.random.default_rng(seed), 4, 2, 64)
        k.copy_(to_type(w, "bf16", dev))
        slots.copy_(torch.tensor([seed, 10 + seed, 31 - seed, 16], device=dev))
        graph.replay()
        torch.cuda.synchronize()
        want = A.bf16(A.row_values(*A.quantise_rows(w, 8), 8))
        assert np.array_equal(out_k.float().cpu().numpy(), want) and torch.equal(out_k, out_v)
