"""GPU parity of the norms and the rotation of queries and keys (grinqh_qk_rope)
with the fp64 oracle; what goes into the cache bit by bit.

Bound.  The mean of D squares is off by (D + 2) u relative (u = 2^-24), its root
by half of that, with two roundings each of root, quotient and products: (D / 2 +
8) u.  The fraction of a turn is rounded once (pi u radian) and sine and cosine
are within 4 u of it; product and sum round three times more.  So an output is
within (D / 2 + 20) u (|a| + |b|) of a cos - b sin, and its type's rounding.
"""

import numpy as np
import pytest

from oracle import attention_oracle as A
from oracle import decoder_oracle as O
from tests.attention_util import HALF, U, inside, to_type
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import input_adaptive_bit_amd as G
    G.load()
    return require_gpu()


def frequencies(turned, base=10000.0):
    return base ** -(np.arange(0, turned, 2) / max(turned, 1))


def inputs(rng, n, heads, kv, dim, dtype):
    """The fused projection's rows, as values of the type."""
    x = rng.standard_normal((n, heads + 2 * kv, dim)).astype(np.float32)
    return A.bf16(x) if dtype == "bf16" else x


def check(got, x, positions, freqs, weight, eps, neighbours, dtype, what):
    want, size = O.rope(x, positions, freqs, weight, eps, neighbours)
    D = x.shape[-1]
    bound = (D / 2 + 20) * U * size + HALF[dtype] * np.abs(want) + 1e-30
    inside(got.float().cpu().numpy(), want, bound, what)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("n,heads,kv,part,normed", [(1, 4, 1, 1, True), (1, 32, 8, 1, False), (7, 3, 3, 2, True), (50, 5, 1, 4, False),
                                                    (130, 12, 4, 1, True), (3, 2, 1, 0, True)])
def test_rows_match_the_oracle(dev, dim, dtype, neighbours, n, heads, kv, part, normed):
    import input_adaptive_bit_amd as G
    import torch
    turned = dim // part if part else 0
    say(f"qk_rope n={n} heads={heads}/{kv} dim={dim} turned={turned} {dtype} neighbours={neighbours} normed={normed}")
    rng = np.random.default_rng(n + dim + turned)
    rows = inputs(rng, n, heads, kv, dim, dtype)
    positions = rng.integers(0, 140000, n).astype(np.int32)
    freqs = frequencies(turned)
    weights = [(1 + 0.2 * rng.standard_normal(dim)).astype(np.float32) if normed else None for _ in range(2)]
    if dtype == "bf16":
        weights = [None if w is None else A.bf16(w) for w in weights]
    x = to_type(rows, dtype, dev)
    q, k = G.qk_rope(x[:, :heads], x[:, heads:heads + kv], torch.from_numpy(positions).to(dev), torch.from_numpy(freqs).to(dev),
                     *(None if w is None else to_type(w, dtype, dev) for w in weights), eps=1e-5, neighbours=neighbours)
    check(q, rows[:, :heads], positions, freqs, weights[0], 1e-5, neighbours, dtype, "q")
    check(k, rows[:, heads:heads + kv], positions, freqs, weights[1], 1e-5, neighbours, dtype, "k")


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,heads,kv,dim,page", [(1, 32, 8, 128, 64), (37, 3, 3, 64, 16), (300, 4, 2, 128, 128), (5, 2, 1, 256, 256)])
def test_the_cache_holds_the_rotated_keys_and_the_values(dev, bits, dtype, n, heads, kv, dim, page):
    """Bit for bit what kv_write makes of the rotated keys and of the values; slots outside the pool are passed over."""
    import input_adaptive_bit_amd as G
    import torch
    say(f"qk_rope cache bits={bits} {dtype} n={n} heads={heads}/{kv} dim={dim} page={page}")
    rng = np.random.default_rng(n + bits)
    x = to_type(inputs(rng, n, heads, kv, dim, dtype), dtype, dev)
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    n_pages = -(-n // page) + 2
    slots = rng.permutation(n_pages * page)[:n]
    slots[n // 2:n // 2 + n // 10] = [-1, n_pages * page, 2 ** 40][n % 3]
    slots = torch.from_numpy(slots).to(dev)
    positions = torch.from_numpy(rng.integers(0, 9000, n).astype(np.int32)).to(dev)
    freqs = torch.from_numpy(frequencies(dim)).to(dev)
    weight = to_type((1 + 0.2 * rng.standard_normal(dim)).astype(np.float32), "f32", dev)
    caches = [G.new_kv_cache(kv, dim, page, n_pages, bits, dev) for _ in range(3)]
    plain = G.qk_rope(q, k, positions, freqs, weight, weight)
    G.kv_write(caches[0], plain[1], v, slots)
    got = G.qk_rope(q, k, positions, freqs, weight, weight, cache=caches[1], v=v, slots=slots)
    only = G.qk_rope(q, k, positions, freqs, weight, weight, cache=caches[2], v=v, slots=slots, keys=False)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1]) and torch.equal(only[0], plain[0]) and only[1] is None
    for c in caches[1:]:
        assert torch.equal(c.k_codes, caches[0].k_codes) and torch.equal(c.v_codes, caches[0].v_codes)
        if bits < 16:
            assert torch.equal(c.k_grid, caches[0].k_grid) and torch.equal(c.v_grid, caches[0].v_grid)


@pytest.mark.parametrize("n,heads,kv,dim,turned,dtype,neighbours,bits", [
    (33001, 1, 1, 64, 64, "bf16", False, 0), (9001, 2, 1, 64, 32, "f32", True, 8), (20003, 3, 1, 128, 128, "bf16", False, 8),
    (9001, 2, 2, 128, 48, "f32", False, 16), (9002, 1, 1, 256, 256, "bf16", False, 4), (4099, 5, 1, 256, 128, "bf16", True, 16),
    (40000, 1, 1, 128, 0, "bf16", False, 16)])
def test_many_tokens_at_once(dev, n, heads, kv, dim, turned, dtype, neighbours, bits):
    """Several tokens to a workgroup: the bits of the same tokens a hundred at a time, and within the bound of the formula."""
    import input_adaptive_bit_amd as G
    import torch
    say(f"qk_rope n={n} heads={heads}/{kv} dim={dim} turned={turned} {dtype} neighbours={neighbours} bits={bits}")
    rng = np.random.default_rng(n)
    rows = inputs(rng, n, heads, kv, dim, dtype)
    x = to_type(rows, dtype, dev)
    positions = rng.integers(0, 140000, n).astype(np.int32)
    freqs, w = frequencies(turned), A.bf16(1 + 0.2 * rng.standard_normal(dim).astype(np.float32))
    at, f, weight = torch.from_numpy(positions).to(dev), torch.from_numpy(freqs).to(dev), to_type(w, "bf16", dev)
    slots = torch.from_numpy(rng.permutation(n + 50)[:n]).to(dev)
    caches = [G.new_kv_cache(kv, dim, 16, n // 16 + 1, bits, dev) if bits else None for _ in range(2)]

    def call(a, b, cache):
        more = {"cache": cache, "v": x[a:b, heads + kv:], "slots": slots[a:b]} if bits else {}
        return G.qk_rope(x[a:b, :heads], x[a:b, heads:heads + kv], at[a:b], f, weight, None, eps=1e-5, neighbours=neighbours, **more)

    q, k = call(0, n, caches[0])
    for a in range(0, n, max(100, n // 12)):
        b = min(a + 100, n)
        got = call(a, b, caches[1])
        assert torch.equal(got[0], q[a:b]) and torch.equal(got[1], k[a:b])
    if bits:
        G.kv_write(caches[1], k, x[:, heads + kv:], slots)
        assert torch.equal(caches[0].k_codes, caches[1].k_codes) and torch.equal(caches[0].v_codes, caches[1].v_codes)
        if bits < 16:
            assert torch.equal(caches[0].k_grid, caches[1].k_grid) and torch.equal(caches[0].v_grid, caches[1].v_grid)
    some = np.concatenate([np.arange(0, n, 37), np.arange(n - 20, n)])
    check(q[some], rows[some][:, :heads], positions[some], freqs, w, 1e-5, neighbours, dtype, "q")
    check(k[some], rows[some][:, heads:heads + kv], positions[some], freqs, None, 1e-5, neighbours, dtype, "k")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("n", [1, 9, 200])
def test_in_place_within_the_fused_projection(dev, dtype, neighbours, n):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(n)
    heads, kv, dim = 6, 2, 128
    x = to_type(inputs(rng, n, heads, kv, dim, dtype), dtype, dev)
    positions = torch.arange(n, dtype=torch.int32, device=dev)
    freqs = torch.from_numpy(frequencies(64)).to(dev)
    weight = to_type(np.linspace(0.5, 1.5, dim, dtype=np.float32), "f32", dev)
    q, k = G.qk_rope(x[:, :heads], x[:, heads:heads + kv], positions, freqs, weight, weight, neighbours=neighbours)
    v = x[:, heads + kv:].clone()
    y = x.clone()
    G.grinqh_qk_rope(y[:, :heads], y[:, heads:heads + kv], positions, freqs, y[:, :heads], y[:, heads:heads + kv], weight, weight,
                     neighbours=neighbours)
    assert torch.equal(y[:, :heads], q) and torch.equal(y[:, heads:heads + kv], k) and torch.equal(y[:, heads + kv:], v)


def test_far_and_negative_positions_and_any_frequency(dev):
    """Whole ranges: the last position of 31 bits, negative ones, frequencies of zero, above one and scaled."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(0)
    positions = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071, 10 ** 6 + 1, -7], np.int32)
    freqs = np.concatenate([frequencies(48), [0.0, 1.0, 3.7, 1e-12, -0.25, 2 * np.pi, np.pi / 2, 1 / 3]])
    rows = inputs(rng, len(positions), 2, 1, 64, "f32")
    x = to_type(rows, "f32", dev)
    q, k = G.qk_rope(x[:, :2], x[:, 2:3], torch.from_numpy(positions).to(dev), torch.from_numpy(freqs).to(dev))
    # An angle of 2^31 radians has an error of its own in fp64: 2^31 2^-52 in the product and in the turns
    want, size = O.rope(rows[:, :2], positions, freqs)
    bound = ((64 / 2 + 20) * U + np.abs(positions.astype(np.float64))[:, None, None] * 7 * 2.0 ** -51) * size + U * np.abs(want)
    inside(q.cpu().numpy(), want, bound)


def test_a_row_that_is_not_finite_stays_alone(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(1)
    rows = inputs(rng, 4, 3, 1, 64, "f32")
    x = to_type(rows, "f32", dev)
    positions, freqs = torch.arange(4, dtype=torch.int32, device=dev), torch.from_numpy(frequencies(32)).to(dev)
    w = torch.ones(64, device=dev)
    clean = G.qk_rope(x[:, :3], x[:, 3:4], positions, freqs, w, w)
    x[1, 1, 40], x[2, 0, 3], x[3, 3, 0] = float("nan"), float("inf"), float("nan")
    got = G.qk_rope(x[:, :3], x[:, 3:4], positions, freqs, w, w)
    hit = torch.zeros(4, 3, dtype=torch.bool, device=dev)
    hit[1, 1] = hit[2, 0] = True
    assert torch.equal(got[0][~hit], clean[0][~hit]) and torch.isnan(got[0][1, 1]).all()
    assert torch.equal(got[1][:3], clean[1][:3]) and torch.isnan(got[1][3]).all()
    # without a norm what is not turned stays its own value, and NaN stays in its pair
    plain = G.qk_rope(x[:, :3], x[:, 3:4], positions, freqs)
    assert torch.isnan(plain[0][1, 1]).sum() == 1 and (~torch.isfinite(plain[0][2, 0])).sum() <= 2


def test_norm_of_zero_rows_and_of_none(dev):
    import input_adaptive_bit_amd as G
    import torch
    x = torch.zeros(2, 3, 64, device=dev)
    w = torch.ones(64, device=dev)
    positions, freqs = torch.arange(2, dtype=torch.int32, device=dev), torch.from_numpy(frequencies(64)).to(dev)
    q, k = G.qk_rope(x[:, :2], x[:, 2:], positions, freqs, w, w)
    assert (q == 0).all() and (k == 0).all()
    none = G.qk_rope(x[:0, :2], x[:0, 2:], positions[:0], freqs, w, w)
    assert none[0].shape == (0, 2, 64) and none[1].shape == (0, 1, 64)


def test_one_norm_alone(dev):
    """A weight for the queries only leaves the keys unnormed, and the other way."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(3)
    rows = inputs(rng, 5, 2, 2, 128, "f32")
    x, w = to_type(rows, "f32", dev), to_type(np.linspace(1, 2, 128, dtype=np.float32), "f32", dev)
    positions, freqs = torch.arange(5, dtype=torch.int32, device=dev), torch.from_numpy(frequencies(128)).to(dev)
    both, none = G.qk_rope(x[:, :2], x[:, 2:4], positions, freqs, w, w), G.qk_rope(x[:, :2], x[:, 2:4], positions, freqs)
    q_only, k_only = (G.qk_rope(x[:, :2], x[:, 2:4], positions, freqs, *a) for a in ((w, None), (None, w)))
    assert torch.equal(q_only[0], both[0]) and torch.equal(q_only[1], none[1])
    assert torch.equal(k_only[0], none[0]) and torch.equal(k_only[1], both[1])


def test_graph_replays_and_another_stream(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(4)
    n, heads, kv, dim = 6, 4, 2, 128
    x = to_type(inputs(rng, n, heads, kv, dim, "bf16"), "bf16", dev)
    positions = torch.arange(n, dtype=torch.int32, device=dev)
    slots = torch.arange(n, dtype=torch.int64, device=dev)
    freqs, w = torch.from_numpy(frequencies(dim)).to(dev), torch.ones(dim, dtype=torch.bfloat16, device=dev)
    cache = G.new_kv_cache(kv, dim, 16, 4, 8, dev)
    out = torch.empty(n, heads, dim, dtype=torch.bfloat16, device=dev), torch.empty(n, kv, dim, dtype=torch.bfloat16, device=dev)

    def step(stream=None):
        G.grinqh_qk_rope(x[:, :heads], x[:, heads:heads + kv], positions, freqs, *out, w, w, cache=cache, v=x[:, heads + kv:],
                         slots=slots, stream=stream)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.Stream()
    for turn in range(3):
        x.copy_(to_type(inputs(rng, n, heads, kv, dim, "bf16"), "bf16", dev))
        positions.add_(1000)
        slots.copy_((torch.arange(n) * 7 + turn) % 64)
        cache.k_codes.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, cache.k_codes, cache.v_codes, cache.k_grid)]
        cache.k_codes.zero_()
        torch.cuda.synchronize()
        step(other)
        other.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*out, cache.k_codes, cache.v_codes, cache.k_grid)))
