"""GPU parity of decode_attention and prefill_attention with the fp64 oracle;
bounds from the roundings the calls document (tests/attention_util.py)."""

import numpy as np
import pytest

from oracle import attention_oracle as A
from tests.attention_util import Cache, decode_reference, inside, prefill_reference, rows, to_bf16, to_type
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import input_adaptive_bit_amd as G
    G.load()
    return require_gpu()


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _np(t):
    return t.float().cpu().numpy()


def _decode(c, q, q_dtype, out_dtype, dev, max_len=None, scale=None, lens=None, workspace=None, what=""):
    import input_adaptive_bit_amd as G
    import torch
    scale = c.dim ** -0.5 if scale is None else scale
    out, lse = G.decode_attention(c.dev, to_type(q, q_dtype, dev), c.dev_table, c.dev_lens, max_len, scale,
                                  _dt(out_dtype), True, workspace)
    torch.cuda.synchronize()
    o, bound, l, l_bound = decode_reference(c, q, scale, out_dtype, lens)
    inside(_np(out), o, bound, what + " out")
    inside(_np(lse), l, l_bound, what + " lse")
    return out


def _queries(rng, batch, n_q, dim, q_dtype):
    q = rng.standard_normal((batch, n_q, dim)).astype(np.float32)
    return A.bf16(q) if q_dtype == "bf16" else q


# ------------------------------------------------------------------- decode --

@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("heads,group,dim,page,lens", [
    (8, 4, 128, 64, [500]),
    (2, 1, 64, 16, [1, 2, 15, 16, 17, 31, 32, 33, 0]),
    (1, 7, 128, 32, [127, 128, 129, 0, 1]),
    (3, 8, 256, 128, [255, 257, 64]),
    (2, 16, 64, 256, [300, 5]),
    (1, 24, 128, 16, [100, 65]),
    (1, 64, 64, 32, [70]),
    (1, 16, 256, 64, [200, 70]),
    (5, 2, 128, 16, [63, 64, 65, 191, 193]),
])
def test_decode_matches_the_oracle(dev, bits, heads, group, dim, page, lens):
    say(f"decode bits={bits} heads={heads}x{group} dim={dim} page={page} lens={lens}")
    rng = np.random.default_rng(heads * 100 + group + dim + bits)
    c = Cache(rng, lens, heads, dim, bits, page, dev)
    for q_dtype, out_dtype in (("bf16", "bf16"), ("f32", "f32")):
        _decode(c, _queries(rng, len(lens), heads * group, dim, q_dtype), q_dtype, out_dtype, dev)


@pytest.mark.parametrize("bits,heads,group,dim,page,n", [(8, 1, 16, 256, 64, 9001), (4, 1, 16, 128, 16, 12345),
                                                         (16, 1, 24, 64, 128, 8000), (8, 2, 4, 128, 64, 20011), (4, 1, 8, 128, 128, 30001),
                                                         (16, 1, 2, 64, 16, 9000), (8, 1, 3, 256, 32, 5003)])
def test_decode_over_a_long_cache(dev, bits, heads, group, dim, page, n):
    """One sequence, many parts, joined."""
    say(f"decode long bits={bits} n={n}")
    rng = np.random.default_rng(n)
    c = Cache(rng, [n], heads, dim, bits, page, dev)
    q = _queries(rng, 1, heads * group, dim, "bf16")
    first = _decode(c, q, "bf16", "f32", dev)
    _decode(c, q, "bf16", "f32", dev, max_len=n)
    import torch
    assert torch.equal(first, _decode(c, q, "bf16", "f32", dev)), "the same call twice, the same bits"


@pytest.mark.parametrize("q_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group,page,n", [(64, 1, 16, 7003), (64, 8, 32, 5000), (128, 4, 64, 9001), (128, 8, 16, 6145),
                                              (128, 7, 256, 513), (256, 3, 64, 4100)])
def test_decode_of_four_bits_and_small_groups(dev, dim, group, page, n, q_dtype):
    """A head's tokens are weighed in two columns; ends in either half of a tile."""
    rng = np.random.default_rng(n)
    c = Cache(rng, [n], 1, dim, 4, page, dev)
    q = _queries(rng, 1, group, dim, q_dtype)
    for length in (n, n - 16, 17, 16, 1):
        c.dev_lens.fill_(length)
        _decode(c, q, q_dtype, "f32", dev, max_len=n, lens=[length], what=str(length))


@pytest.mark.parametrize("bits,group", [(8, 3), (16, 3), (4, 16), (4, 5)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_decode_of_full_queries_over_a_long_cache(dev, dim, bits, group):
    """fp32 queries in the largest workgroups.  They enter the scores as the sum of two bf16, which is off by half a step
    of half a step, 2^-16: a score by 2^-16 sum |q_d k_d|, an output by twice that of its sum p |v|."""
    import input_adaptive_bit_amd as G
    import torch
    say(f"decode fp32 queries bits={bits} group={group} dim={dim}")
    rng = np.random.default_rng(dim + bits + group)
    c = Cache(rng, [5003, 31], 4, dim, bits, 64, dev)
    q = _queries(rng, 2, 4 * group, dim, "f32")
    scale = dim ** -0.5
    for length in (5003, 4992, 33, 1, 0):
        for batch in (1, 2):
            lens = [length, 31][:batch]
            out, lse = G.decode_attention(c.dev, torch.from_numpy(q[:batch]).to(dev), c.dev_table[:batch],
                                          torch.tensor(lens, dtype=torch.int32, device=dev), 5003, out_dtype=torch.float32,
                                          return_lse=True)
            o, bound, l, l_bound = decode_reference(c, q[:batch], scale, "f32", lens)
            for b in range(batch):
                for h in range(4 * group):
                    (k, terms), (v, v_terms) = (c.gathered(b, h // group, which, lens[b]) for which in range(2))
                    if len(k):
                        _, _, p = A.attend(q[b, h:h + 1], k, v, scale)
                        off = 2.0 ** -16 * scale * (terms @ np.abs(q[b, h].astype(np.float64))).max()
                        bound[b, h] += 2 * off * (p @ v_terms)[0]
                        l_bound[b, h] += off
            inside(_np(out), o, bound, f"out, length {length}")
            inside(_np(lse), l, l_bound, f"lse, length {length}")


def test_decode_of_many_sequences_of_very_different_lengths(dev):
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 700, 40)] + [3001, 0, 1]
    c = Cache(rng, lens, 2, 64, 8, 32, dev)
    _decode(c, _queries(rng, len(lens), 6, 64, "bf16"), "bf16", "bf16", dev)


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_absent_pages_are_not_seen(dev, bits):
    """Entries below 0 or past the pool, at the start, inside and at the end;
    one sequence has no page at all."""
    import torch
    rng = np.random.default_rng(bits)
    c = Cache(rng, [100, 70, 90, 16, 400], 2, 64, bits, 16, dev)
    c.table[0, [0, 3, 6]] = [-1, c.n_pages, 2 ** 31 - 1]
    c.table[1, 4] = -2 ** 31
    c.table[2, :3] = -5
    c.table[3, 0] = c.n_pages + 100
    c.table[4, 5:20] = -1
    c.dev_table.copy_(torch.from_numpy(c.table))
    out = _decode(c, _queries(rng, 5, 4, 64, "bf16"), "bf16", "f32", dev)
    assert not out[3].any()


def test_lengths_outside_the_host_bound_are_clamped(dev):
    import torch
    rng = np.random.default_rng(1)
    c = Cache(rng, [96, 96, 96, 96], 2, 64, 8, 32, dev)
    q = _queries(rng, 4, 4, 64, "bf16")
    c.dev_lens.copy_(torch.tensor([-3, 2 ** 31 - 1, 50, -2 ** 31]))
    _decode(c, q, "bf16", "f32", dev, max_len=96, lens=[0, 96, 50, 0])
    _decode(c, q, "bf16", "f32", dev, max_len=40, lens=[0, 40, 40, 0])
    _decode(c, q, "bf16", "f32", dev, max_len=1 << 28, lens=[0, 96, 50, 0])       # the page table ends at 96


def test_decode_scales_and_extreme_scores(dev):
    """No, negative and very large scales: equal weights, one weight alone."""
    rng = np.random.default_rng(2)
    c = Cache(rng, [300, 33], 1, 128, 8, 64, dev)
    q = _queries(rng, 2, 5, 128, "bf16")
    for scale in (0.0, -0.05, 1e-20, 30.0, 1e4):
        _decode(c, q, "bf16", "f32", dev, scale=scale, what=f"scale {scale}")
    _decode(c, A.bf16(q * 100), "bf16", "f32", dev)


def test_queries_are_slices_of_a_fused_projection_and_the_table_is_wider(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(4)
    c = Cache(rng, [100, 37, 64], 2, 128, 8, 32, dev)
    fused = rows(rng, 3, 6 + 4, 128)
    t = to_bf16(fused, dev)
    wide = torch.full((3, 50), -1, dtype=torch.int32, device=dev)
    wide[:, 7:7 + c.table.shape[1]] = c.dev_table
    out = G.decode_attention(c.dev, t[:, :6], wide[:, 7:7 + c.table.shape[1]], c.dev_lens, 100,
                             out_dtype=torch.float32)
    o, bound, _, _ = decode_reference(c, fused[:, :6], 128 ** -0.5, "f32")
    inside(_np(out), o, bound)


def test_what_is_not_finite_in_unseen_tokens_has_no_effect_and_in_seen_ones_stays_in_its_head(dev):
    """The Cache helper fills every unused row with NaN; here a seen row of one
    head is NaN too."""
    import input_adaptive_bit_amd as G
    import torch
    for bits in (8, 16):
        rng = np.random.default_rng(6)
        c = Cache(rng, [77], 3, 64, bits, 32, dev)
        q = _queries(rng, 1, 6, 64, "bf16")
        base = _decode(c, q, "bf16", "f32", dev)
        page, t = c.row(0, 40)
        if bits == 16:
            c.dev.v_codes[page, 1, t] = 0xFF
        else:
            c.dev.v_grid[page, 1, t] = float("nan")
        out = G.decode_attention(c.dev, to_bf16(q, dev), c.dev_table, c.dev_lens, out_dtype=torch.float32)
        assert torch.isnan(out[0, 2:4]).all()
        assert torch.equal(out[0, :2], base[0, :2]) and torch.equal(out[0, 4:], base[0, 4:])


def test_one_workspace_for_calls_of_different_sizes_and_in_two_graphs(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(12)
    a = Cache(rng, [5000, 17], 2, 128, 8, 64, dev)
    b = Cache(rng, [900] * 7, 1, 64, 4, 16, dev)
    ws = torch.zeros(max(G.grinqh_attention_workspace_bytes(a.dev.layout, 8, 2, 5000),
                         G.grinqh_attention_workspace_bytes(b.dev.layout, 5, 7, 912)), dtype=torch.uint8, device=dev)
    qa, qb = _queries(rng, 2, 8, 128, "bf16"), _queries(rng, 7, 5, 64, "bf16")
    for _ in range(3):
        _decode(a, qa, "bf16", "f32", dev, workspace=ws, max_len=5000)
        _decode(b, qb, "bf16", "f32", dev, workspace=ws)
    graphs = []
    for c, q in ((a, qa), (b, qb)):
        q_dev = to_bf16(q, dev)
        out = torch.empty(q.shape, dtype=torch.float32, device=dev)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            G.grinqh_decode_attention(c.dev, q_dev, c.dev_table, c.dev_lens, c.table.shape[1] * c.page, out, ws)
        graphs.append((c, q_dev, out, g))
    for turn in range(4):
        for c, q_dev, out, g in graphs:
            q = _queries(rng, *out.shape, "bf16")
            q_dev.copy_(to_bf16(q, dev))
            lens = [max(0, n - 13 * turn) for n in c.lens]
            c.dev_lens.copy_(torch.tensor(lens))
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            o, bound, _, _ = decode_reference(c, q, c.dim ** -0.5, "f32", lens)
            inside(_np(out), o, bound, f"turn {turn}")


def test_the_workspace_of_the_largest_call_serves_smaller_ones(dev):
    """A batch that shrinks, with the longest of its lengths as the bound; then calls that make their own workspace."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(21)
    lens = [int(x) for x in rng.integers(1, 1600, 32)]
    c = Cache(rng, lens, 8, 64, 8, 64, dev)
    q = _queries(rng, 32, 16, 64, "bf16")
    q_dev = to_bf16(q, dev)
    o, bound, _, _ = decode_reference(c, q, 0.125, "f32")
    ws = G.new_attention_workspace(c.dev.layout, 16, 32, 8192, dev)
    assert ws.nbytes > 1 << 20
    for b in range(32, 0, -1):
        for max_len in (max(lens[:b]), 8192 - 13 * b):
            for w in (ws, None):
                out = G.decode_attention(c.dev, q_dev[:b], c.dev_table[:b], c.dev_lens[:b], max_len, out_dtype=torch.float32,
                                         workspace=w)
                inside(_np(out), o[:b], bound[:b], f"batch {b}, max_len {max_len}")
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = G.decode_attention(c.dev, q_dev, c.dev_table, c.dev_lens, 8192, out_dtype=torch.float32, stream=other)
    other.synchronize()
    inside(_np(out), o, bound, "another stream")


def test_decode_on_another_stream(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(13)
    c = Cache(rng, [3000], 2, 64, 8, 64, dev)
    q = _queries(rng, 1, 4, 64, "bf16")
    q_dev = to_bf16(q, dev)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = G.decode_attention(c.dev, q_dev, c.dev_table, c.dev_lens, out_dtype=torch.float32, stream=other)
    other.synchronize()
    o, bound, _, _ = decode_reference(c, q, 0.125, "f32")
    inside(_np(out), o, bound)


def test_decode_reads_pages_past_four_gigabytes(dev):
    import input_adaptive_bit_amd as G
    import torch
    heads, dim, page, n_pages = 8, 256, 256, 4400
    c = G.new_kv_cache(heads, dim, page, n_pages, 16, dev)
    table = torch.tensor([[n_pages - 1, 4096, 0, n_pages - 2]], dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(2)
    kv = torch.randn(2, 900, heads, dim, generator=g, device=dev).bfloat16()
    at = torch.arange(900, device=dev)
    G.kv_write(c, kv[0], kv[1], table[0].long()[at // page] * page + at % page)
    q = _queries(np.random.default_rng(0), 1, heads, dim, "bf16")
    out = G.decode_attention(c, to_bf16(q, dev), table, torch.tensor([900], dtype=torch.int32, device=dev),
                             out_dtype=torch.float32)
    k, v = (x.float().cpu().numpy() for x in kv)
    o, bound, _, _ = prefill_reference(q, k, v, [0, 1], [0, 900], dim ** -0.5, False, "f32")
    inside(_np(out), o, bound)


def test_no_sequences(dev):
    import input_adaptive_bit_amd as G
    import torch
    c = G.new_kv_cache(2, 64, 16, 1, 8, dev)
    out = G.decode_attention(c, torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev),
                             torch.zeros(0, 3, dtype=torch.int32, device=dev),
                             torch.zeros(0, dtype=torch.int32, device=dev))
    assert out.shape == (0, 4, 64)


# ------------------------------------------------------------------ prefill --

def _packed(rng, n_q, n_kv, dim, lens_q, lens_k, extra=0):
    cu_q, cu_k = np.concatenate([[0], np.cumsum(lens_q)]), np.concatenate([[0], np.cumsum(lens_k)])
    q, k, v = rows(rng, cu_q[-1] + extra, n_q, dim), rows(rng, cu_k[-1] + extra, n_kv, dim), \
        rows(rng, cu_k[-1] + extra, n_kv, dim)
    return q, k, v, cu_q.astype(np.int32), cu_k.astype(np.int32)


def _prefill(q, k, v, cu_q, cu_k, dev, causal=True, out_dtype="bf16", scale=None, what=""):
    import input_adaptive_bit_amd as G
    import torch
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out = torch.full(q.shape, 7.5, dtype=_dt(out_dtype), device=dev)
    lse = torch.full(q.shape[:2], 7.5, dtype=torch.float32, device=dev)
    G.grinqh_prefill_attention(to_bf16(q, dev), to_bf16(k, dev), to_bf16(v, dev), torch.from_numpy(cu_q).to(dev),
                               torch.from_numpy(cu_k).to(dev), out, causal, scale, lse)
    torch.cuda.synchronize()
    o, bound, l, l_bound = prefill_reference(q, k, v, cu_q, cu_k, scale, causal, out_dtype)
    n = cu_q[-1]
    inside(_np(out)[:n], o[:n], bound[:n], what + " out")
    inside(_np(lse)[:n], l[:n], l_bound[:n], what + " lse")
    assert bool((out[n:] == 7.5).all()) and bool((lse[n:] == 7.5).all()), "rows behind the last sequence"
    return out


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n_kv,group,dim,lens", [
    (2, 4, 128, [130]),
    (1, 1, 64, [1]),
    (2, 2, 64, [1, 2, 31, 32, 33, 63, 64, 65]),
    (1, 7, 128, [127, 128, 129, 0, 5]),
    (3, 1, 256, [255, 100, 1]),
    (2, 3, 128, [300, 0, 0, 17, 257]),
    (1, 5, 64, [513]),
    (1, 2, 256, [385]),
])
def test_prefill_matches_the_oracle(dev, causal, n_kv, group, dim, lens):
    say(f"prefill heads={n_kv}x{group} dim={dim} lens={lens} causal={causal}")
    rng = np.random.default_rng(sum(lens) + dim + group)
    args = _packed(rng, n_kv * group, n_kv, dim, lens, lens)
    for out_dtype in ("bf16", "f32"):
        _prefill(*args, dev, causal, out_dtype)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,lens_q,lens_k", [
    (64, [5, 130, 1], [300, 131, 1000]),          # cached beginnings
    (128, [64, 1, 200], [640, 65, 329]),
    (128, [100, 7, 40], [30, 0, 40]),             # fewer keys than queries: rows that see nothing
    (256, [33, 70], [200, 3]),
    (64, [0, 3, 0], [50, 3, 0]),                  # keys without queries
])
def test_prefill_with_other_numbers_of_keys_than_queries(dev, causal, dim, lens_q, lens_k):
    say(f"prefill dim={dim} q={lens_q} k={lens_k} causal={causal}")
    rng = np.random.default_rng(sum(lens_k) + dim)
    _prefill(*_packed(rng, 4, 2, dim, lens_q, lens_k), dev, causal, "f32")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,n_kv,group,lens_q,lens_k", [
    (128, 2, 4, [40], [5000]),
    (64, 1, 7, [9, 60, 3], [2100, 60, 1023]),             # parts for some, one for others
    (256, 1, 2, [20, 1], [1100, 2500]),
    (128, 1, 1, [1], [4111]),
    (64, 2, 3, [600, 30], [580, 3000]),                   # rows that see nothing beside split ones
])
def test_few_queries_over_many_keys_in_parts(dev, causal, dim, n_kv, group, lens_q, lens_k):
    import input_adaptive_bit_amd as G
    import torch
    say(f"prefill parts dim={dim} q={lens_q} k={lens_k} causal={causal}")
    rng = np.random.default_rng(sum(lens_k) + dim)
    q, k, v, cu_q, cu_k = _packed(rng, n_kv * group, n_kv, dim, lens_q, lens_k)
    o, bound, l, l_bound = prefill_reference(q, k, v, cu_q, cu_k, dim ** -0.5, causal, "f32")
    t = [to_bf16(x, dev) for x in (q, k, v)] + [torch.from_numpy(x).to(dev) for x in (cu_q, cu_k)]
    out, lse = G.prefill_attention(*t, causal, out_dtype=torch.float32, return_lse=True)
    n = G.grinqh_prefill_attention_workspace_bytes(*t, out, causal)
    assert n > 0, "the case is one whose keys are split"
    inside(_np(out), o, bound, "split")
    inside(_np(lse), l, l_bound, "split lse")
    again = torch.empty_like(out)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)                    # any contents
    G.grinqh_prefill_attention(*t, again, causal, workspace=ws)
    assert torch.equal(out, again)
    G.grinqh_prefill_attention(*t, again, causal)
    inside(_np(again), o, bound, "without a workspace")
    with pytest.raises(G.GrinqhError):
        G.grinqh_prefill_attention(*t, again, causal, workspace=ws[:256])


def test_rows_behind_the_last_sequence_and_batches_of_many(dev):
    rng = np.random.default_rng(3)
    _prefill(*_packed(rng, 2, 1, 64, [3, 50], [3, 50], extra=150), dev)
    lens = [int(x) for x in rng.integers(0, 20, 150)]              # more sequences than a wave has lanes
    _prefill(*_packed(rng, 2, 1, 64, lens, lens), dev)
    lens = [1] * 300 + [140]
    _prefill(*_packed(rng, 1, 1, 64, lens, lens), dev)


def test_prefill_scales_and_extreme_scores(dev):
    rng = np.random.default_rng(4)
    args = _packed(rng, 2, 1, 128, [150], [150])
    for scale in (0.0, -0.05, 1e-20, 30.0, 1e4):
        _prefill(*args, dev, True, "f32", scale, f"scale {scale}")
    q, k, v, cu_q, cu_k = args
    _prefill(A.bf16(q * 100), k, v, cu_q, cu_k, dev, True, "f32")


def _exact_prefill(q, k, v, cu_q, cu_k, scale, dev, want, split):
    """Runs a causal call whose scores q . k are exact in fp32, against want(scores [m] of one row, values [m][dim]) ->
    (output, lse).  Bounds, with u = 2^-24: an exponent (s - top) c is off by 4 u of itself (log2 e, its product with
    the scale, the product, exp2), and counts down to -128 only, so a weight is off by 2^-22 2^7 = 2^-15, as is the
    sum, and by 2^-8 where it is rounded to bf16; the sums by m u; lse = ln 2 (top c + log2 sum) by the roundings of
    log2 e, c, top c, the sum, ln 2 and the product, 8 u of its size, and by what the weights' sum is off by."""
    import input_adaptive_bit_amd as G
    import torch
    t = [to_bf16(x, dev) for x in (q, k, v)] + [torch.from_numpy(x).to(dev) for x in (cu_q, cu_k)]
    out, lse = G.prefill_attention(*t, scale=scale, out_dtype=torch.float32, return_lse=True)
    assert (G.grinqh_prefill_attention_workspace_bytes(*t, out) > 0) == split
    o, l, mass = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape)
    group = q.shape[1] // k.shape[1]
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(n):
            for h in range(q.shape[1]):
                keys = slice(cu_k[b], cu_k[b] + max(0, i + m - n + 1))
                s = k[keys, h // group].astype(np.float64) @ q[cu_q[b] + i, h].astype(np.float64)
                o[cu_q[b] + i, h], l[cu_q[b] + i, h] = want(s, v[keys, h // group].astype(np.float64))
                mass[cu_q[b] + i, h], _ = want(s, np.abs(v[keys, h // group]).astype(np.float64))
    u = 2.0 ** -24
    rel = 2.0 ** -8 + 2 * 2.0 ** -15 + (len(k) + 32) * u
    with np.errstate(over="ignore"):
        inside(_np(out), o, rel * mass + u * np.abs(o), f"out, scale {scale}")
        l32 = np.where(np.isfinite(l.astype(np.float32)), l, l.astype(np.float32))
        inside(_np(lse), l32, np.where(np.isfinite(l32), 8 * u * np.abs(l) + rel, 0.0), f"lse, scale {scale}")


@pytest.mark.parametrize("lens_q,lens_k,split", [([90], [90], False), ([3, 2], [2100, 1500], True)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_scores_far_from_zero_leave_the_largest_its_weight(dev, dim, lens_q, lens_k, split):
    """Scores of whole numbers times a scale so large that every key but the best of a row (or, where several share the
    largest score, those) weighs nothing."""
    rng = np.random.default_rng(dim)
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (lens_q, lens_k))
    q = rng.integers(-2, 3, (cu_q[-1], 4, dim)).astype(np.float32)
    k = rng.integers(-2, 3, (cu_k[-1], 2, dim)).astype(np.float32)
    v = rows(rng, cu_k[-1], 2, dim)
    for size, scale in ((1, 1e8), (1, 1e9), (1, 1e12), (1, 1e30), (4096, 1e30), (1, -1e8), (1, -1e12), (4096, -1e30)):
        say(f"prefill dim={dim} scale={scale} size={size} split={split}")

        def best(s, values):
            s = s * np.float64(np.float32(scale))
            at = s == s.max()
            return values[at].mean(0), s.max() + np.log(at.sum())

        _exact_prefill(q * size, k * size, v, cu_q, cu_k, scale, dev, best, split)


@pytest.mark.parametrize("lens_q,lens_k,split", [([90], [90], False), ([3, 2], [2100, 1500], True)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_scores_with_a_large_common_part(dev, dim, lens_q, lens_k, split):
    """Whole numbers 2^20 and 2^23 + 0 .. 60 times 1/2: a softmax of the small rest, rows whose maximum grows on the way
    and parts with maxima of their own.  Then equal scores of 3e4 . 3e4 at the usual scale: the mean."""
    rng = np.random.default_rng(dim + 1)
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (lens_q, lens_k))
    v = rows(rng, cu_k[-1], 1, dim)

    def softmax(scale):
        def want(s, values):
            a = s * scale
            e = np.exp(a - a.max())
            return e @ values / e.sum(), a.max() + np.log(e.sum())
        return want

    for power in (10, 11):
        q, k = np.zeros((cu_q[-1], 2, dim), np.float32), np.zeros((cu_k[-1], 1, dim), np.float32)
        q[..., 0], k[..., 0] = 2.0 ** power, 2.0 ** (10 if power == 10 else 12)
        q[..., 1], k[..., 1] = 1.0, rng.integers(0, 9, k.shape[:2])
        k[-40:, 0, 1] += rng.integers(0, 53, 40)
        _exact_prefill(q, k, v, cu_q, cu_k, 0.5, dev, softmax(0.5), split)
    q, k = (A.bf16(np.full((n, h, dim), 3e4, np.float32)) for n, h in ((cu_q[-1], 2), (cu_k[-1], 1)))
    _exact_prefill(q, k, v, cu_q, cu_k, dim ** -0.5, dev, softmax(np.float64(np.float32(dim ** -0.5))), split)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_row_far_from_zero_leaves_its_neighbours_alone(dev, dim):
    """One query 2^16 times as large, scores past 2^16 in its row alone: every other row keeps its bits."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(dim + 2)
    q, k, v, cu, _ = _packed(rng, 4, 2, dim, [200, 90], [200, 90])
    t = [to_bf16(x, dev) for x in (k, v)] + [torch.from_numpy(cu).to(dev)]
    base, lse = G.prefill_attention(to_bf16(q, dev), *t, out_dtype=torch.float32, return_lse=True)
    far = q.copy()
    far[137, 2] *= 65536.0
    out, far_lse = G.prefill_attention(to_bf16(far, dev), *t, out_dtype=torch.float32, return_lse=True)
    others = torch.ones(290, 4, dtype=torch.bool, device=dev)
    others[137, 2] = False
    assert torch.equal(out[others], base[others]) and torch.equal(far_lse[others], lse[others])
    # its largest score leads by more than 2^7: that key's value, in bf16 as it is
    s = k[:138, 1].astype(np.float64) @ far[137, 2].astype(np.float64) * dim ** -0.5
    first, second = np.argsort(s)[::-1][:2]
    assert s[first] - s[second] > 128 and abs(s[first]) > 2 ** 16
    assert np.array_equal(_np(out)[137, 2], v[first, 1])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_keys_that_are_not_seen_may_be_anything(dev, dim):
    """NaN and infinities in later keys, other sequences and rows behind the
    last: the queries that do not see them are those of a call without."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(5)
    q, k, v, cu_q, cu_k = _packed(rng, 2, 1, dim, [200, 90], [200, 90], extra=70)
    base = _prefill(q, k, v, cu_q, cu_k, dev, True, "f32")
    for bad in (np.nan, np.inf, -np.inf):
        k2, v2 = k.copy(), v.copy()
        k2[150:200], v2[150:200], k2[290:], v2[290:] = bad, bad, bad, bad
        out = G.prefill_attention(to_bf16(q, dev), to_bf16(k2, dev), to_bf16(v2, dev), torch.from_numpy(cu_q).to(dev),
                                  torch.from_numpy(cu_k).to(dev), out_dtype=torch.float32)
        assert torch.equal(out[:150], base[:150]) and torch.equal(out[200:290], base[200:290])
        if bad is np.nan:
            assert torch.isnan(out[150:200]).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_infinities_in_seen_values_go_where_the_formula_says(dev, dim):
    """Into the queries that see them and the dimension they are in: up, down,
    and NaN where both or a NaN is seen; in tiles seen whole and in part."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(9)
    q, k, v, cu_q, cu_k = _packed(rng, 2, 1, dim, [300], [300])
    t = [to_bf16(x, dev) for x in (q, k)] + [torch.from_numpy(x).to(dev) for x in (cu_q, cu_k)]
    base = G.prefill_attention(t[0], t[1], to_bf16(v, dev), *t[2:], scale=0.01, out_dtype=torch.float32)
    want = base.clone()
    bad = v.copy()
    for key, d, x in ((20, 3, np.inf), (100, 40, -np.inf), (150, 3, np.inf), (200, 40, np.inf), (250, 9, np.nan)):
        bad[key, 0, d] = x
        want[key:, :, d] += float(x)
    out = G.prefill_attention(t[0], t[1], to_bf16(bad, dev), *t[2:], scale=0.01, out_dtype=torch.float32)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.isposinf(), want.isposinf()) and torch.equal(out.isneginf(), want.isneginf())
    assert torch.equal(out[want.isfinite()], want[want.isfinite()])


def test_prefill_of_very_many_sequences(dev):
    """More than 64 x 64, empty ones among them, against one call for each run."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(10)
    lens = rng.integers(0, 5, 5000)
    lens[[17, 4999]] = [200, 90]
    q, k, v, cu, _ = _packed(rng, 2, 1, 64, lens, lens)
    t = [to_bf16(x, dev) for x in (q, k, v)]
    out = G.prefill_attention(*t, torch.from_numpy(cu).to(dev), out_dtype=torch.float32)
    for a, b in ((0, 40), (1000, 1050), (4960, 5000)):
        r = slice(cu[a], cu[b])
        o, bound, _, _ = prefill_reference(q[r], k[r], v[r], cu[a:b + 1] - cu[a], cu[a:b + 1] - cu[a], 0.125, True, "f32")
        inside(_np(out[r]), o, bound, f"{a}..{b}")
    for a in range(0, 5000, 50):
        r = slice(cu[a], cu[a + 50])
        if cu[a] < cu[a + 50]:
            few = G.prefill_attention(*(x[r] for x in t), torch.from_numpy(cu[a:a + 51] - cu[a]).to(dev),
                                      out_dtype=torch.float32)
            assert torch.equal(out[r], few), a


@pytest.mark.parametrize("dim", [64, 128])
def test_few_queries_of_many_sequences_in_parts(dev, dim):
    """Three of 300 sequences have queries, a fourth keys alone; with a workspace and without."""
    import ctypes
    import input_adaptive_bit_amd as G
    from input_adaptive_bit_amd import grinqh as B
    import torch
    rng = np.random.default_rng(dim)
    lens_q, lens_k = np.zeros(300, int), np.zeros(300, int)
    lens_q[[0, 130, 299]], lens_k[[0, 7, 130, 299]] = [1, 5, 2], [3000, 500, 2777, 1]
    q, k, v, cu_q, cu_k = _packed(rng, 8, 2, dim, lens_q, lens_k)
    o, bound, lse, lse_bound = prefill_reference(q, k, v, cu_q, cu_k, dim ** -0.5, True, "f32")
    t = [to_bf16(x, dev) for x in (q, k, v)]
    cu = [torch.from_numpy(x).to(dev) for x in (cu_q, cu_k)]
    a = B.PrefillAttentionArgs(batch=300, total_q=8, total_k=len(k), n_q_heads=8, n_kv_heads=2, head_dim=dim, causal=1)
    assert G.load().grinqh_prefill_attention_workspace_bytes(ctypes.byref(a)) > 0
    out, got = G.prefill_attention(*t, *cu, out_dtype=torch.float32, return_lse=True)
    inside(_np(out), o, bound, "in parts")
    inside(_np(got), lse, lse_bound, "lse")
    whole = torch.empty_like(out)
    G.grinqh_prefill_attention(*t, *cu, whole)
    inside(_np(whole), o, bound, "whole")


def test_tokens_that_lie_gigabytes_apart(dev):
    """The largest strides: rows of one buffer of 6.7 GB, against the same rows close together."""
    import input_adaptive_bit_amd as G
    import torch
    stride, n, dim = 1 << 24, 200, 64
    far = torch.empty(n * stride, dtype=torch.bfloat16, device=dev).as_strided((n, 4, dim), (stride, dim, 1))
    near = torch.randn(n, 4, dim, device=dev).to(torch.bfloat16)
    far.copy_(near)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    slots = torch.arange(n, device=dev)
    outs = []
    for x in (far, near):
        q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
        cache = G.new_kv_cache(1, dim, 64, 4, 8, device=dev)
        G.kv_write(cache, k, v, slots)
        table = torch.arange(4, dtype=torch.int32, device=dev).expand(n, 4)
        lens = torch.arange(1, n + 1, dtype=torch.int32, device=dev)
        outs.append((G.prefill_attention(q, k, v, cu), cache.k_codes, cache.v_grid,
                     G.decode_attention(cache, q, table.contiguous(), lens)))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_prefill_takes_slices_of_a_fused_projection(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(6)
    lens = [100, 33]
    fused = rows(rng, 133, 6 + 2 * 2, 128)
    t = to_bf16(fused, dev)
    cu = torch.tensor([0, 100, 133], dtype=torch.int32, device=dev)
    out, lse = G.prefill_attention(t[:, :6], t[:, 6:8], t[:, 8:], cu, return_lse=True)
    o, bound, l, l_bound = prefill_reference(fused[:, :6], fused[:, 6:8], fused[:, 8:], [0, 100, 133], [0, 100, 133],
                                             128 ** -0.5, True, "bf16")
    inside(_np(out), o, bound)
    inside(_np(lse), l, l_bound)


def test_sequence_bounds_outside_the_rows_are_clamped(dev):
    """Entries past the packed rows are taken as their end, so nothing outside
    the tensors is read or written."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(7)
    q, k, v, _, _ = _packed(rng, 2, 1, 64, [100], [100])
    t = [to_bf16(x, dev) for x in (q, k, v)]
    cu = torch.tensor([0, 40, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    out = G.prefill_attention(*t, cu, out_dtype=torch.float32)
    o, bound, _, _ = prefill_reference(q, k, v, [0, 40, 100], [0, 40, 100], 0.125, True, "f32")
    inside(_np(out), o, bound)


def test_prefill_in_a_graph_and_on_another_stream(dev):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(8)
    q, k, v, cu_q, cu_k = _packed(rng, 4, 2, 128, [140, 60], [140, 60])
    t = [to_bf16(x, dev) for x in (q, k, v)]
    cu = torch.from_numpy(cu_q).to(dev)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = G.prefill_attention(*t, cu, out_dtype=torch.float32, stream=other)
    other.synchronize()
    o, bound, _, _ = prefill_reference(q, k, v, cu_q, cu_k, 128 ** -0.5, True, "f32")
    inside(_np(out), o, bound)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.grinqh_prefill_attention(*t, cu, cu, out)
    for cut in (140, 1, 77, 199):
        cu.copy_(torch.tensor([0, cut, 200]))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        o, bound, _, _ = prefill_reference(q, k, v, [0, cut, 200], [0, cut, 200], 128 ** -0.5, True, "f32")
        inside(_np(out), o, bound, f"cut {cut}")


def test_no_rows(dev):
    import input_adaptive_bit_amd as G
    import torch
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=dev)
    cu = torch.zeros(3, dtype=torch.int32, device=dev)
    assert G.prefill_attention(none, none, none, cu).shape == (0, 2, 64)
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device=dev)
    out = G.prefill_attention(q, none, none, torch.tensor([0, 1, 4], dtype=torch.int32, device=dev), cu)
    assert not out.any()


# ----------------------------------------------------------------- together --

@pytest.mark.parametrize("bits", [4, 8, 16])
def test_a_conversation(dev, bits):
    """A prompt, some tokens and a second prompt through one cache, as a decoder
    runs them: every token's output is that of attention over the whole text
    (its own keys in full during its prompt, the cached ones otherwise)."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(bits)
    n_q, n_kv, dim, page = 8, 2, 128, 16
    prompt, steps, second = 150, 20, 45
    total = prompt + steps + second
    fused = rows(rng, total, n_q + 2 * n_kv, dim)
    t = to_bf16(fused, dev)
    q, k, v = t[:, :n_q], t[:, n_q:n_q + n_kv], t[:, n_q + n_kv:]
    n_pages = -(-total // page)
    c = G.new_kv_cache(n_kv, dim, page, n_pages + 2, bits, dev)
    table = torch.randperm(n_pages + 2, device=dev)[:n_pages].int()[None]
    at = torch.arange(total, device=dev)
    slots = table[0].long()[at // page] * page + at % page
    ws = G.new_attention_workspace(c.layout, n_q, 1, total, dev)
    got = torch.empty(total, n_q, dim, device=dev)

    cu = torch.tensor([0, prompt], dtype=torch.int32, device=dev)
    got[:prompt] = G.prefill_attention(q[:prompt], k[:prompt], v[:prompt], cu, out_dtype=torch.float32)
    G.kv_write(c, k[:prompt], v[:prompt], slots[:prompt])
    for i in range(prompt, prompt + steps):
        G.kv_write(c, k[i:i + 1], v[i:i + 1], slots[i:i + 1])
        got[i] = G.decode_attention(c, q[i:i + 1], table, torch.tensor([i + 1], dtype=torch.int32, device=dev), total,
                                    out_dtype=torch.float32, workspace=ws)[0]
    past = prompt + steps
    old_k, old_v = G.kv_read(c, slots[:past])
    got[past:] = G.prefill_attention(q[past:], torch.cat([old_k, k[past:]]), torch.cat([old_v, v[past:]]),
                                     torch.tensor([0, second], dtype=torch.int32, device=dev),
                                     torch.tensor([0, total], dtype=torch.int32, device=dev), out_dtype=torch.float32)
    torch.cuda.synchronize()

    def cached(x):
        return A.row_values(*A.quantise_rows(x, bits), bits).astype(np.float32)

    qf, kf, vf = fused[:, :n_q], fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:]
    o, bound, _, _ = prefill_reference(qf[:prompt], kf[:prompt], vf[:prompt], [0, prompt], [0, prompt], dim ** -0.5, True,
                                       "f32")
    inside(_np(got[:prompt]), o, bound, "prompt")
    kc, vc = cached(kf[:past]), cached(vf[:past])
    o, bound, _, _ = prefill_reference(qf[prompt:past], kc, vc, [0, steps], [0, past], dim ** -0.5, True, "f32")
    inside(_np(got[prompt:past]), o, bound, "tokens")
    kc, vc = np.concatenate([A.bf16(kc), kf[past:]]), np.concatenate([A.bf16(vc), vf[past:]])
    o, bound, _, _ = prefill_reference(qf[past:], kc, vc, [0, second], [0, total], dim ** -0.5, True, "f32")
    inside(_np(got[past:]), o, bound, "second prompt")
