"""The attention operators' cases: what is timed and compared, their plain
forms in elementary torch operations, and their values in 64 bits.

Three operators, as a decoder runs them between its fused q|k|v projection
and its o projection:

* "cache": rows of new tokens are quantised into a paged key-value cache
  (4 or 8 bits on the midpoint grid of the weights, per token and head, or
  kept as bfloat16) and read back, as a program does that goes on from a
  cached prompt;
* "decode": one new token of every sequence attends to the sequence's pages;
* "prefill": whole prompts, packed behind one another, causal, with grouped
  heads; a prompt may have more keys than queries (its cached beginning).

k, v and q are views of the fused projection's output rows
[tokens][(n_q + 2 n_kv) * head_dim], as the projection writes them.
"""

import math

import torch

own = False

# Sizes.  32 query heads over 8 key-value heads of 128 are the 8B shape whose
# linears (4096 -> 4096, 4096 -> 1024) the benchmark times, 64 over 8 the 70B
# shape (8192); the others are the further head layouts that are accepted.
_CACHE = "cache"
_DECODE = "decode"
_PREFILL = "prefill"


def listed():
    return [
        # one token of one sequence, every decode step of a batch-1 program
        {"name": "cache, 1 token, 8 bit", "op": _CACHE, "tokens": 1, "heads": 8, "dim": 128, "bits": 8, "page": 64,
         "dtype": "bf16"},
        # a prompt of ordinary length, into the smallest cache
        {"name": "cache, 2048 tokens, 4 bit", "op": _CACHE, "tokens": 2048, "heads": 8, "dim": 128, "bits": 4,
         "page": 16, "dtype": "bf16"},
        # a long prompt whose projection was kept in fp32; an odd count, so the last page is not full
        {"name": "cache, 16381 tokens, 8 bit, fp32", "op": _CACHE, "tokens": 16381, "heads": 8, "dim": 128, "bits": 8,
         "page": 128, "dtype": "f32"},
        # a short context: the smallest call, where latency counts
        {"name": "decode, 1 x 500, 8 bit", "op": _DECODE, "batch": 1, "longest": 500, "shortest": 500, "heads": 8,
         "group": 4, "dim": 128, "bits": 8, "page": 16},
        # one long conversation at batch 1
        {"name": "decode, 1 x 32768, 8 bit", "op": _DECODE, "batch": 1, "longest": 32768, "shortest": 32768, "heads": 8,
         "group": 4, "dim": 128, "bits": 8, "page": 64},
        # the longest context, 70B heads, the smallest cache
        {"name": "decode, 1 x 131071, 4 bit", "op": _DECODE, "batch": 1, "longest": 131071, "shortest": 131071,
         "heads": 8, "group": 8, "dim": 128, "bits": 4, "page": 128},
        # a batch of conversations of very different lengths
        {"name": "decode, 32 x 17..8192, 8 bit", "op": _DECODE, "batch": 32, "longest": 8192, "shortest": 17,
         "heads": 8, "group": 4, "dim": 128, "bits": 8, "page": 64},
        # a small model: ungrouped heads of 64, cache not quantised
        {"name": "decode, 7 x 1..3001, 16 bit", "op": _DECODE, "batch": 7, "longest": 3001, "shortest": 1,
         "heads": 12, "group": 1, "dim": 64, "bits": 16, "page": 32},
        # one short prompt
        {"name": "prefill, 1 x 130", "op": _PREFILL, "batch": 1, "longest": 130, "shortest": 130, "past": 0, "heads": 8,
         "group": 4, "dim": 128},
        # several prompts of different lengths in one call
        {"name": "prefill, 6 x 33..1200", "op": _PREFILL, "batch": 6, "longest": 1200, "shortest": 33, "past": 0,
         "heads": 8, "group": 4, "dim": 128},
        # a further question about cached text: few queries, many keys; heads of 64
        {"name": "prefill, 2 x 257..512 after 6000", "op": _PREFILL, "batch": 2, "longest": 512, "shortest": 257,
         "past": 6000, "heads": 4, "group": 7, "dim": 64},
        # one long prompt
        {"name": "prefill, 1 x 8192", "op": _PREFILL, "batch": 1, "longest": 8192, "shortest": 8192, "past": 0,
         "heads": 8, "group": 4, "dim": 128},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice([_CACHE, _DECODE, _PREFILL])
    dim = rng.choice([64, 128, 128, 256])
    bits = rng.choice([4, 8, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == _CACHE:
        heads = rng.choice([1, 2, 4, 5, 8, 12])
        most = max(2, 16381 * 8 * 128 // (heads * dim))
        return {"op": op, "tokens": _spread(rng, 1, min(most, 30000)), "heads": heads, "dim": dim, "bits": bits,
                "page": page, "dtype": rng.choice(["bf16", "f32"])}
    heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16, 24])
    while heads * group > 64:
        group //= 2
    if op == _DECODE:
        batch = _spread(rng, 1, 48)
        # cached values at most those of 32 conversations of 4096 in the 8B shape
        most = max(16, min(131072, 32 * 4096 * 8 * 128 // (batch * heads * dim)))
        longest = _spread(rng, 4, most)
        return {"op": op, "batch": batch, "longest": longest, "shortest": rng.randint(max(1, longest // 64), longest),
                "heads": heads, "group": group, "dim": dim, "bits": bits, "page": page}
    batch = _spread(rng, 1, 9)
    most = max(64, int(4096 * math.sqrt(32 * 128 / (heads * group * dim)) / batch))
    longest = _spread(rng, 8, min(most, 6000))
    return {"op": op, "batch": batch, "longest": longest, "shortest": rng.randint(max(1, longest // 32), longest),
            "past": rng.choice([0, 0, rng.randint(1, max(1, most))]), "heads": heads, "group": group, "dim": dim}


# ------------------------------------------------------------------ inputs --

def _lengths(c):
    """The sequences' lengths: from the longest down to the shortest, in an order that is neither."""
    b, hi, lo = c["batch"], c["longest"], c["shortest"]
    n = [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]
    return n[::2] + n[1::2][::-1]


def _projection(c, tokens, seed, dtype):
    """The fused projection's rows: unit normal, keys with a few strong channels of each head, as keys have."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_kv, dim = c["heads"], c["dim"]
    n_q = n_kv * c.get("group", 1)
    rows = torch.randn(tokens, n_q + 2 * n_kv, dim, generator=g, device="cuda")
    strong = torch.rand(n_kv, dim, generator=g, device="cuda") < 0.03
    rows[:, n_q:n_q + n_kv] *= torch.where(strong, 4.0, 1.0)
    return rows.to(dtype)


def _row_bytes(c):
    return c["dim"] * c["bits"] // 8


def _quantised(w, bits):
    """Codes and grid (scale, zero point) of rows on the midpoint grid: all steps in 32 bits, the grid in fp16."""
    w = w.float()
    if bits == 16:
        return w.to(torch.bfloat16).view(torch.uint8), torch.zeros(0, dtype=torch.float16, device=w.device)
    lo, hi = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
    grid = torch.cat([(hi - lo) * 2.0 ** -bits, lo], -1).half() + 0.0
    s, z = grid[..., :1].float(), grid[..., 1:].float()
    q = torch.where(s == 0, 0.0, torch.floor((w - z) / s).clamp(0, 2 ** bits - 1)).to(torch.uint8)
    return (q if bits == 8 else q[..., 0::2] | (q[..., 1::2] << 4)), grid


def _values(codes, grid, bits):
    """The values that rows of the cache stand for, in 32 bits."""
    if bits == 16:
        return codes.view(torch.bfloat16).float()
    q = codes if bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return grid[..., :1].float() * (q.float() + 0.5) + grid[..., 1:].float()


def _pools(c, n_pages):
    shape = (n_pages, c["heads"], c["page"])
    grid = (*shape, 2) if c["bits"] < 16 else (0,)
    return [torch.zeros(*shape, _row_bytes(c), dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros(*grid, dtype=torch.float16, device="cuda") for _ in range(2)]


def _handle(c, n_pages, pools):
    """What a program keeps of the framework's for its cache."""
    import input_adaptive_bit_amd as G
    layout = G.grinqh_kv_layout_init(c["heads"], c["dim"], c["page"], n_pages, c["bits"])
    return G.KVCache(layout, *pools)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    s = {"case": c}
    if c["op"] == _CACHE:
        n, page = c["tokens"], c["page"]
        rows = _projection(c, n, seed, torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        s["k"], s["v"] = rows[:, -2 * c["heads"]:-c["heads"]], rows[:, -c["heads"]:]
        used = -(-n // page)
        pages = torch.randperm(used + 3, generator=g, device="cuda")[:used]     # pages as a running server hands them out
        at = torch.arange(n, device="cuda")
        s["slots"] = pages[at // page] * page + at % page
        n_pages = used + 3
        s["pools"] = _pools(c, n_pages)
    elif c["op"] == _DECODE:
        lens, page = _lengths(c), c["page"]
        most = -(-max(lens) // page)
        n_pages = c["batch"] * most + 5
        rows = _projection(c, c["batch"], seed, torch.bfloat16)
        s["q"] = rows[:, :c["heads"] * c["group"]]
        s["pages"] = torch.randperm(n_pages, generator=g, device="cuda")[:c["batch"] * most].view(c["batch"], most).int()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["longest"] = c["longest"]
        s["pools"] = _pools(c, n_pages)
        strong = torch.where(torch.rand(c["heads"], 1, c["dim"], generator=g, device="cuda") < 0.03, 4.0, 1.0)
        for which in range(2):                                                   # keys, then values
            for at in range(0, n_pages, 4096):                                   # in pieces: the pool may be large
                w = torch.randn(s["pools"][which][at:at + 4096].shape[:3] + (c["dim"],), generator=g, device="cuda")
                codes, grid = _quantised((w * strong if which == 0 else w).bfloat16(), c["bits"])
                s["pools"][which][at:at + 4096] = codes
                if c["bits"] < 16:
                    s["pools"][2 + which][at:at + 4096] = grid
        if own:
            import input_adaptive_bit_amd as G
            s["workspace"] = G.new_attention_workspace(_handle(c, n_pages, s["pools"]).layout, c["heads"] * c["group"],
                                                       c["batch"], c["longest"])
    else:
        lens = _lengths(c)
        rows = _projection(c, sum(lens) + c["past"] * c["batch"], seed, torch.bfloat16)
        n_q = c["heads"] * c["group"]
        s["q"], s["k"], s["v"] = rows[:sum(lens), :n_q], rows[:, n_q:n_q + c["heads"]], rows[:, n_q + c["heads"]:]
        s["cu_q"] = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
        s["cu_k"] = torch.tensor([0] + [n + c["past"] for n in lens], device="cuda").cumsum(0).int()
    if own and "pools" in s:
        s["cache"] = _handle(c, n_pages, s["pools"])
    return s


# ------------------------------------------------------------- plain forms --

def _softmax_rows(scores):
    """Weights of masked scores; a row with nothing to attend to has none."""
    m = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def _cache_plain(s):
    c, page = s["case"], s["case"]["page"]
    at, row = s["slots"] // page, s["slots"] % page
    out = []
    for which, x in enumerate((s["k"], s["v"])):
        codes, grid = _quantised(x, c["bits"])
        s["pools"][which][at, :, row] = codes
        if c["bits"] < 16:
            s["pools"][2 + which][at, :, row] = grid
            grid = s["pools"][2 + which][at, :, row]
        out.append(_values(s["pools"][which][at, :, row], grid, c["bits"]).to(torch.bfloat16))
    return out


def _decode_plain(s):
    c = s["case"]
    b, h, dim = c["batch"], c["heads"], c["dim"]
    pages = s["pages"].long()
    k, v = (_values(s["pools"][i][pages], s["pools"][2 + i][pages] if c["bits"] < 16 else None, c["bits"])
            .transpose(1, 2).reshape(b, h, -1, dim) for i in range(2))
    q = s["q"].float().reshape(b, h, c["group"], dim)
    scores = torch.matmul(q, k.transpose(-1, -2)) * dim ** -0.5
    seen = torch.arange(k.shape[2], device="cuda") < s["lens"].view(b, 1, 1, 1)
    p = _softmax_rows(scores.masked_fill(~seen, -math.inf))
    return torch.matmul(p, v).reshape(b, h * c["group"], dim).to(torch.bfloat16)


def _prefill_plain(s):
    c = s["case"]
    h, dim, n_q, n_k = c["heads"], c["dim"], s["q"].shape[0], s["k"].shape[0]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    i, j = torch.arange(n_q, device="cuda"), torch.arange(n_k, device="cuda")
    seq_q, seq_k = torch.bucketize(i, cu_q[1:], right=True), torch.bucketize(j, cu_k[1:], right=True)
    last = cu_k[seq_q + 1] - cu_q[seq_q + 1] + i                                # the last key that query i sees
    seen = (seq_q[:, None] == seq_k) & (j <= last[:, None])
    q = s["q"].float().reshape(n_q, h, c["group"], dim).permute(1, 2, 0, 3).reshape(h, -1, dim)
    k, v = (x.float().transpose(0, 1) for x in (s["k"], s["v"]))
    scores = torch.matmul(q, k.transpose(-1, -2)).mul_(dim ** -0.5).view(h, c["group"], n_q, n_k)
    p = _softmax_rows(scores.masked_fill_(~seen, -math.inf)).view(h, -1, n_k)
    o = torch.matmul(p, v).view(h, c["group"], n_q, dim)
    return o.permute(2, 0, 1, 3).reshape(n_q, h * c["group"], dim).to(torch.bfloat16)


# ---------------------------------------------------------- the framework's --

def _cache_own(s):
    import input_adaptive_bit_amd as G
    G.kv_write(s["cache"], s["k"], s["v"], s["slots"])
    return list(G.kv_read(s["cache"], s["slots"], torch.bfloat16))


def _decode_own(s):
    import input_adaptive_bit_amd as G
    return G.decode_attention(s["cache"], s["q"], s["pages"], s["lens"], s["longest"], out_dtype=torch.bfloat16,
                              workspace=s["workspace"])


def _prefill_own(s):
    import input_adaptive_bit_amd as G
    return G.prefill_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out_dtype=torch.bfloat16)


def run(state):
    op = state["case"]["op"]
    if own:
        return {_CACHE: _cache_own, _DECODE: _decode_own, _PREFILL: _prefill_own}[op](state)
    return {_CACHE: _cache_plain, _DECODE: _decode_plain, _PREFILL: _prefill_plain}[op](state)


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    h, dim = c["heads"], c["dim"]
    if c["op"] == _CACHE:
        n = 2 * c["tokens"] * h
        row = _row_bytes(c) + (4 if c["bits"] < 16 else 0)
        # the new rows in, their codes out and in again, the values out
        return {"bytes": n * (dim * (2 if c["dtype"] == "bf16" else 4) + 2 * row + dim * 2), "flops": n * dim * 8}
    n_q, lens = h * c["group"], _lengths(c)
    if c["op"] == _DECODE:
        row = _row_bytes(c) + (4 if c["bits"] < 16 else 0)
        return {"bytes": 2 * sum(lens) * h * row + 4 * c["batch"] * n_q * dim, "flops": 4 * sum(lens) * n_q * dim}
    pairs = sum(n * (n + 1) // 2 + n * c["past"] for n in lens)
    keys = sum(lens) + c["past"] * c["batch"]
    return {"bytes": 2 * dim * (2 * sum(lens) * n_q + 2 * keys * h), "flops": 4 * pairs * n_q * dim}


# ------------------------------------------------------- values in 64 bits --

def _exact_rows(x, bits):
    """Rows of the cache in 64 bits: what each value's nearest grid midpoint is.  Only the grid is held in fewer
    bits, as the cache holds it."""
    x = x.double()
    if bits == 16:
        return x.to(torch.bfloat16).double()
    low, high = x.min(-1).values.unsqueeze(-1), x.max(-1).values.unsqueeze(-1)
    step, low = ((high - low) / 2 ** bits).half().double(), low.half().double()
    cell = ((x - low) / step).floor_().clamp_(0, 2 ** bits - 1)
    return torch.where(step > 0, low + (cell + 0.5) * step, low)


def _exact_cached(codes, grid, bits):
    """What the cache's bytes stand for, in 64 bits."""
    if bits == 16:
        return codes.view(torch.bfloat16).double()
    if bits == 4:
        low = codes % 16
        codes = torch.cat([low.unsqueeze(-1), ((codes - low) // 16).unsqueeze(-1)], -1).reshape(*codes.shape[:-1], -1)
    return (codes.double() + 0.5) * grid.double()[..., 0, None] + grid.double()[..., 1, None]


def _exact_attention(q, k, v, past):
    """One head's attention: q [n][dim], k and v [m][dim]; query i sees keys 0 .. past + i (all, where past is None)."""
    out = torch.empty_like(q)
    for at in range(0, len(q), 2048):
        a = (q[at:at + 2048] @ k.T) / math.sqrt(q.shape[1])
        if past is not None:
            a = a + torch.full_like(a, -math.inf).triu_(past + at + 1)
        out[at:at + 2048] = torch.softmax(a, 1) @ v
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == _CACHE:
        return [_exact_rows(s[w], c["bits"]) for w in ("k", "v")]
    q = s["q"].double()
    out = torch.empty_like(q)
    group = c["group"]
    if c["op"] == _DECODE:
        for b, n in enumerate(_lengths(c)):
            pages = s["pages"][b].long()
            for h in range(c["heads"]):
                k, v = (_exact_cached(s["pools"][i][pages, h].flatten(0, 1)[:n],
                                      s["pools"][2 + i][pages, h].flatten(0, 1)[:n] if c["bits"] < 16 else None,
                                      c["bits"]) for i in range(2))
                out[b, h * group:(h + 1) * group] = _exact_attention(q[b, h * group:(h + 1) * group], k, v, None)
        return out
    k, v = s["k"].double(), s["v"].double()
    at_q = at_k = 0
    for n in _lengths(c):
        m = n + c["past"]
        for h in range(q.shape[1]):
            out[at_q:at_q + n, h] = _exact_attention(q[at_q:at_q + n, h], k[at_k:at_k + m, h // group],
                                                     v[at_k:at_k + m, h // group], c["past"])
        at_q, at_k = at_q + n, at_k + m
    return out
