"""A decoder layer's further operators: what is timed and compared, their plain
forms in elementary torch operations, and their values in 64 bits.

Four operators, as a decoder runs them around the cache and the attention:

* "linear": a few tokens, or a prompt's, times a matrix of 4-bit weights whose
  groups of input channels have a scale and a zero point each, on the midpoint
  grid of the other weights, s * (q + 1/2) + z;
* "experts": the same product with ragged runs of rows, each run with its own
  expert's matrix; the rows may be gathered from the tokens on the way;
* "rope": norms of queries and keys for each head and the rotation by their
  positions in one pass, which also writes keys and values into the paged cache;
* "pages": what a step of a batch needs to know of the paged cache, from the
  requests' lengths: pages for the new tokens, their slots and positions, the
  new lengths and the ends of the packed sequences.
"""

import math

import torch

own = False

_LINEAR = "linear"
_EXPERTS = "experts"
_ROPE = "rope"
_PAGES = "pages"


def listed():
    return [
        # every decode step of a batch-1 program: the 8B shape's q and o projection, where latency counts
        {"name": "linear, 1 token, 4096 to 4096", "op": _LINEAR, "tokens": 1, "d_in": 4096, "d_out": 4096,
         "group": 128, "dtype": "bf16"},
        # its down projection, in a program that keeps activations in fp32, smaller groups
        {"name": "linear, 1 token, 14336 to 4096, groups of 64, fp32", "op": _LINEAR, "tokens": 1, "d_in": 14336,
         "d_out": 4096, "group": 64, "dtype": "f32"},
        # a small batch of conversations, up projection
        {"name": "linear, 13 tokens, 4096 to 14336", "op": _LINEAR, "tokens": 13, "d_in": 4096, "d_out": 14336,
         "group": 128, "dtype": "bf16"},
        # a prompt's up projection
        {"name": "linear, 2048 tokens, 4096 to 14336", "op": _LINEAR, "tokens": 2048, "d_in": 4096, "d_out": 14336,
         "group": 128, "dtype": "bf16"},
        # two tokens that go to eight of 64 experts each
        {"name": "experts, 16 rows to 64, 4096 to 1024", "op": _EXPERTS, "tokens": 2, "top": 8, "experts": 64,
         "d_in": 4096, "d_out": 1024, "group": 128, "gathered": True},
        # a batch of conversations: few rows for each of many experts, the smallest groups, an odd output size
        {"name": "experts, 516 rows to 64, 2048 to 2050, groups of 32", "op": _EXPERTS, "tokens": 129, "top": 4,
         "experts": 64, "d_in": 2048, "d_out": 2050, "group": 32, "gathered": True},
        # prompts, two of eight large experts for each token; the second product of an expert: its rows lie in order
        {"name": "experts, 4094 rows to 8, 4096 to 14336", "op": _EXPERTS, "tokens": 2047, "top": 2, "experts": 8,
         "d_in": 4096, "d_out": 14336, "group": 128, "gathered": False},
        # every decode step: one token, into a cache of bf16
        {"name": "rope, 1 token, 16 bit cache", "op": _ROPE, "tokens": 1, "heads": 8, "group": 4, "dim": 128,
         "turned": 128, "pairs": "halves", "norm": True, "dtype": "bf16", "bits": 16, "page": 64, "first": 20000},
        # a small model's prompt in fp32: no norm, half of each head turned, neighbouring channels paired, no cache
        {"name": "rope, 517 tokens, fp32, half turned", "op": _ROPE, "tokens": 517, "heads": 12, "group": 1, "dim": 64,
         "turned": 32, "pairs": "neighbours", "norm": False, "dtype": "f32", "bits": 0, "page": 0, "first": 0},
        # a long prompt far into a context, 70B heads, an 8-bit cache that is read back
        {"name": "rope, 16381 tokens, 8 bit cache", "op": _ROPE, "tokens": 16381, "heads": 8, "group": 8, "dim": 128,
         "turned": 128, "pairs": "halves", "norm": True, "dtype": "bf16", "bits": 8, "page": 128, "first": 114688},
        # a decode step of a batch of conversations
        {"name": "pages, 48 sequences, a token each", "op": _PAGES, "batch": 48, "longest": 8192, "new": 1, "page": 64,
         "short": False},
        # prompts of very different lengths that come in at once, some behind cached text
        {"name": "pages, 700 sequences, up to 1024 tokens each", "op": _PAGES, "batch": 700, "longest": 4096,
         "new": 1024, "page": 16, "short": False},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice([_LINEAR, _EXPERTS, _ROPE, _PAGES])
    group = rng.choice([32, 64, 128, 128])
    if op == _LINEAR:
        d_in, d_out = group * _spread(rng, 2, 14336 // group), _spread(rng, 16, 14336)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        # long prompts come in bf16, as the prefill product takes them
        most = 16 if dtype == "f32" else max(1, min(2048, 2048 * 4096 * 14336 // (d_in * d_out)))
        return {"op": op, "tokens": _spread(rng, 1, most), "d_in": d_in, "d_out": d_out, "group": group, "dtype": dtype}
    if op == _EXPERTS:
        experts = _spread(rng, 2, 128)
        d_in = group * _spread(rng, 2, 4096 // group)
        # weights at most those of the largest listed case, and so the products
        d_out = _spread(rng, 16, min(14336, 8 * 4096 * 14336 // (experts * d_in)))
        top = rng.randint(1, min(8, experts))
        most = max(1, min(4096, 4094 * 4096 * 14336 // (d_in * d_out)) // top)
        return {"op": op, "tokens": _spread(rng, 1, most), "top": top, "experts": experts, "d_in": d_in, "d_out": d_out,
                "group": group, "gathered": rng.random() < 0.5}
    if op == _ROPE:
        dim, heads, many = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 2, 4, 5, 7, 8])
        dtype, bits = rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, 8, 16])
        most = 16381 * 80 * 128 // (heads * (many + 2) * dim * (2 if dtype == "f32" else 1))
        return {"op": op, "tokens": _spread(rng, 1, min(most, 30000)), "heads": heads, "group": many, "dim": dim,
                "turned": rng.choice([dim, dim, dim // 2, dim // 4]), "pairs": rng.choice(["halves", "halves", "neighbours"]),
                "norm": rng.random() < 0.7, "dtype": dtype, "bits": bits, "page": rng.choice([16, 32, 64, 128, 256]),
                "first": rng.choice([0, rng.randint(1, 131072)])}
    return {"op": op, "batch": _spread(rng, 1, 700), "longest": _spread(rng, 16, 8192), "new": _spread(rng, 1, 1024),
            "page": rng.choice([16, 32, 64, 128, 256]), "short": rng.random() < 0.3}      # short: pages for half of them


# ------------------------------------------------------------------ inputs --

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _on_grid(w, bits):
    """Codes, scales and zero points of rows on the midpoint grid: all steps in 32 bits, the grid in fp16."""
    lo, hi = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
    s, z = ((hi - lo) * 2.0 ** -bits).half() + 0.0, lo.half() + 0.0
    step = s.float()
    q = torch.where(step == 0, 0.0, torch.floor((w - z.float()) / step).clamp(0, 2 ** bits - 1)).to(torch.uint8)
    return q, s[..., 0], z[..., 0]


def _weights(g, experts, d_in, d_out, group):
    """Codes [experts][d_out][d_in], scales and zero points [experts][d_out][groups] of normal weights with rows of
    different sizes, as trained ones have."""
    q = torch.empty(experts, d_out, d_in, dtype=torch.uint8, device="cuda")
    s, z = (torch.empty(experts, d_out, d_in // group, dtype=torch.float16, device="cuda") for _ in range(2))
    for e in range(experts):
        size = 0.02 * torch.exp(0.3 * torch.randn(d_out, 1, 1, generator=g, device="cuda"))
        w = (torch.randn(d_out, d_in // group, group, generator=g, device="cuda") * size).bfloat16().float()
        codes, s[e], z[e] = _on_grid(w, 4)
        q[e] = codes.view(d_out, d_in)
    return q, s, z


def _activations(g, tokens, width, dtype):
    """Unit normal rows with a few strong channels, as a layer's inputs have."""
    strong = torch.where(torch.rand(width, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    return (torch.randn(tokens, width, generator=g, device="cuda") * strong).to(dtype)


def _expert_counts(c, seed):
    """Rows of each expert: a router's choices, some experts far more liked than others; and the chosen ones, sorted."""
    g = torch.Generator().manual_seed(seed)
    liking = 0.7 * torch.randn(c["experts"], generator=g) + torch.empty(c["tokens"], c["experts"]).exponential_(generator=g).log().neg()
    chosen = liking.topk(c["top"], -1).indices                                      # [tokens][top]
    order = chosen.flatten().sort(stable=True).indices
    return torch.bincount(chosen.flatten(), minlength=c["experts"]), order // c["top"]


def _lengths(c):
    """Cached lengths and new tokens of each sequence; some have none of either."""
    g = torch.Generator().manual_seed(c["batch"])
    old = (torch.rand(c["batch"], generator=g) ** 2 * c["longest"]).long()
    new = torch.ones(c["batch"], dtype=torch.long) if c["new"] == 1 else (
        torch.rand(c["batch"], generator=g) ** 3 * (c["new"] + 1)).long()
    old[::5] = 0
    return old, new


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] in (_LINEAR, _EXPERTS):
        experts = c.get("experts", 1)
        s["q"], s["s"], s["z"] = _weights(g, experts, c["d_in"], c["d_out"], c["group"])
        if c["op"] == _LINEAR:
            s["x"] = _activations(g, c["tokens"], c["d_in"], _type(c["dtype"]))
        else:
            counts, tokens = _expert_counts(c, seed)
            s["most"] = int(counts.max())
            s["ends"] = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int().cuda()
            if c["gathered"]:
                s["x"], s["rows"] = _activations(g, c["tokens"], c["d_in"], torch.bfloat16), tokens.int().cuda()
            else:
                s["x"], s["rows"] = _activations(g, c["tokens"] * c["top"], c["d_in"], torch.bfloat16), None
        if own:
            import input_adaptive_bit_amd as G
            s["weight"] = G.fourbit_pack(s["q"], s["s"], s["z"])
    elif c["op"] == _ROPE:
        n_kv, dim, n = c["heads"], c["dim"], c["tokens"]
        n_q = n_kv * c["group"]
        rows = torch.randn(n, n_q + 2 * n_kv, dim, generator=g, device="cuda").to(_type(c["dtype"]))  # the fused projection's output
        s["q"], s["k"], s["v"] = rows[:, :n_q], rows[:, n_q:n_q + n_kv], rows[:, n_q + n_kv:]
        s["positions"] = torch.arange(c["first"], c["first"] + n, dtype=torch.int32, device="cuda")
        s["freqs"] = 10000.0 ** -(torch.arange(0, c["turned"], 2, dtype=torch.float64, device="cuda") / c["turned"])
        s["weights"] = [(1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(_type(c["dtype"])) if c["norm"] else None
                        for _ in range(2)]
        if c["bits"]:
            page = c["page"]
            n_pages = -(-n // page) + 3
            at = torch.arange(n, device="cuda")
            s["slots"] = torch.randperm(n_pages, generator=g, device="cuda")[at // page] * page + at % page
            shape = (n_pages, n_kv, page)
            s["pools"] = [torch.zeros(*shape, dim * c["bits"] // 8, dtype=torch.uint8, device="cuda") for _ in range(2)]
            s["pools"] += [torch.zeros(*shape, 2, dtype=torch.float16, device="cuda") if c["bits"] < 16 else None for _ in range(2)]
            if own:
                import input_adaptive_bit_amd as G
                s["cache"] = G.KVCache(G.grinqh_kv_layout_init(n_kv, dim, page, n_pages, c["bits"]), *s["pools"])
    else:
        old, new = _lengths(c)
        page = c["page"]
        held, total = -(-old // page), -(-(old + new) // page)
        n_pages = int(total.sum()) + 7
        order = torch.randperm(n_pages, generator=g, device="cuda").int()
        most = int(total.max()) + 2
        table = torch.full((c["batch"], most), -1, dtype=torch.int32, device="cuda")
        filled = torch.arange(most) < held[:, None]
        table[filled.cuda()] = order[:int(held.sum())]
        s["free"] = torch.cat([order[int(held.sum()):], torch.full((int(held.sum()),), -1, dtype=torch.int32, device="cuda")])
        free = n_pages - int(held.sum())
        s["n_free"] = torch.tensor([free // 2 if c["short"] else free], dtype=torch.int32, device="cuda")
        s["table"], s["lens"], s["new"] = table, old.int().cuda(), new.int().cuda()
        s["room"] = int(new.sum()) + 9                                              # a step's buffers are padded
    return s


# ------------------------------------------------------------- plain forms --

def _linear_plain(s):
    c = s["case"]
    q = s["q"][0].view(c["d_out"], -1, c["group"])
    w = s["s"][0].float().unsqueeze(-1) * (q.float() + 0.5) + s["z"][0].float().unsqueeze(-1)
    return torch.matmul(s["x"].float(), w.view(c["d_out"], -1).T).to(s["x"].dtype)


def _experts_plain(s):
    """The rows of each expert padded to the longest run, one batched product, the rows taken out again."""
    c, ends = s["case"], s["ends"].long()
    x = s["x"] if s["rows"] is None else s["x"][s["rows"].long()]
    q = s["q"].view(c["experts"], c["d_out"], -1, c["group"])
    w = (s["s"].float().unsqueeze(-1) * (q.float() + 0.5) + s["z"].float().unsqueeze(-1)).view(c["experts"], c["d_out"], -1)
    row = torch.arange(len(x), device="cuda")
    expert = torch.bucketize(row, ends[1:], right=True)
    at = row - ends[expert]
    padded = torch.zeros(c["experts"], s["most"], c["d_in"], device="cuda")
    padded[expert, at] = x.float()
    y = torch.matmul(padded, w.transpose(1, 2))
    return y[expert, at].to(torch.bfloat16)


def _turned(x, angle, turned, pairs):
    """x [tokens][heads][dim] with its first `turned` channels rotated in pairs by angle [tokens][turned / 2]."""
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    if pairs == "halves":
        a, b = x[..., :turned // 2], x[..., turned // 2:turned]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:turned:2], x[..., 1:turned:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., turned:]], -1)


def _values(codes, grid):
    """What rows of the 8-bit cache stand for, in 32 bits."""
    return grid[..., :1].float() * (codes.float() + 0.5) + grid[..., 1:].float()


def _kept(s, which):
    """A pool of bf16 rows as it stands."""
    return s["pools"][which].view(torch.bfloat16)


def _rope_plain(s):
    c = s["case"]
    angle = s["positions"].double().unsqueeze(1) * s["freqs"]                     # far positions need 64 bits
    out = []
    for x, weight in zip((s["q"], s["k"]), s["weights"]):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        out.append(_turned(x, angle, c["turned"], c["pairs"]).to(s["q"].dtype))
    if c["bits"]:
        at, row = s["slots"] // c["page"], s["slots"] % c["page"]
        for which, x in enumerate((out[1], s["v"])):
            if c["bits"] == 16:
                codes, grid = x.to(torch.bfloat16).view(torch.uint8), None
            else:
                codes, *grid = _on_grid(x.float(), c["bits"])
                s["pools"][2 + which][at, :, row] = torch.stack(grid, -1)
                grid = s["pools"][2 + which][at, :, row]
            s["pools"][which][at, :, row] = codes
            out.append(_values(s["pools"][which][at, :, row], grid).to(torch.bfloat16) if grid is not None else _kept(s, which))
    return out


def _pages_plain(s):
    page, old, new = s["case"]["page"], s["lens"].long(), s["new"].long()
    held, total = (old + page - 1) // page, (old + new + page - 1) // page
    need = total - held
    upto = need.cumsum(0)
    granted = (upto <= s["n_free"]) & (total <= s["table"].shape[1]) | (new == 0)
    lens = torch.where(granted, old + new, old)
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    cu_q, cu_k = torch.cat([zero, new.cumsum(0)]), torch.cat([zero, lens.cumsum(0)])
    # pages from the end of the free list, sequence after sequence
    column = torch.arange(s["table"].shape[1], device="cuda")
    taken = granted[:, None] & (column >= held[:, None]) & (column < total[:, None])
    given = torch.where(granted, need, 0)
    number = (given.cumsum(0) - given)[:, None] + column - held[:, None]
    table = torch.where(taken, s["free"][(s["n_free"] - 1 - number).clamp(0, len(s["free"]) - 1).long()], s["table"])
    s["table"].copy_(table)
    # slots and positions, padded
    token = torch.arange(s["room"], device="cuda")
    seq = torch.bucketize(token, cu_q[1:], right=True)
    there = seq < len(new)
    seq = seq.clamp(max=len(new) - 1)
    position = old[seq] + token - cu_q[seq]
    slot = table[seq, (position // page).clamp(0, table.shape[1] - 1)].long() * page + position % page
    slots = torch.where(there & granted[seq], slot, -1)
    positions = torch.where(there, position, 0)
    left = s["n_free"] - given.sum()
    return {"slots": slots, "positions": positions.int(), "lens": lens.int(), "cu_q": cu_q.int(), "cu_k": cu_k.int(),
            "table": s["table"], "n_free": left.int(), "refused": (~granted).sum().view(1).int()}


# ---------------------------------------------------------- the framework's --

def _linear_own(s):
    import input_adaptive_bit_amd as G
    return G.fourbit_linear(s["weight"], s["x"], out_dtype=s["x"].dtype)


def _experts_own(s):
    import input_adaptive_bit_amd as G
    return G.expert_linear(s["weight"], s["x"], s["ends"], s["rows"], out_dtype=torch.bfloat16)


def _rope_own(s):
    import input_adaptive_bit_amd as G
    c = s["case"]
    more = {"cache": s["cache"], "v": s["v"], "slots": s["slots"]} if c["bits"] else {}
    out = G.qk_rope(s["q"], s["k"], s["positions"], s["freqs"], *s["weights"], eps=1e-6,
                    neighbours=c["pairs"] == "neighbours", **more)
    if c["bits"] == 8:                               # a program that goes on from cached text reads it back
        out = [*out, *G.kv_read(s["cache"], s["slots"], torch.bfloat16)]
    elif c["bits"]:
        out = [*out, _kept(s, 0), _kept(s, 1)]
    return list(out)


def _pages_own(s):
    import input_adaptive_bit_amd as G
    step = G.kv_extend(s["table"], s["lens"], s["new"], s["free"], s["n_free"], s["case"]["page"], s["room"])
    return {"slots": step.slots, "positions": step.positions, "lens": step.seq_lens, "cu_q": step.cu_q, "cu_k": step.cu_k,
            "table": s["table"], "n_free": step.n_free, "refused": step.refused}


def run(state):
    op = state["case"]["op"]
    if own:
        return {_LINEAR: _linear_own, _EXPERTS: _experts_own, _ROPE: _rope_own, _PAGES: _pages_own}[op](state)
    return {_LINEAR: _linear_plain, _EXPERTS: _experts_plain, _ROPE: _rope_plain, _PAGES: _pages_plain}[op](state)


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] in (_LINEAR, _EXPERTS):
        weight = c["d_in"] * c["d_out"] // 2 + 4 * c["d_out"] * (c["d_in"] // c["group"])
        rows = c["tokens"] * c.get("top", 1)
        size = 4 if c.get("dtype") == "f32" else 2
        # the weights of the experts that are chosen at all
        chosen = c["experts"] * (1 - (1 - c["top"] / c["experts"]) ** c["tokens"]) if "experts" in c else 1
        return {"bytes": int(weight * chosen) + size * rows * c["d_out"]
                + size * c["d_in"] * (c["tokens"] if c.get("gathered") else rows), "flops": 2 * rows * c["d_in"] * c["d_out"]}
    if c["op"] == _ROPE:
        n_q, n_kv, dim = c["heads"] * c["group"], c["heads"], c["dim"]
        size = 2 if c["dtype"] == "bf16" else 4
        values = c["tokens"] * dim
        moved = 2 * size * values * (n_q + n_kv)                                    # queries and keys in and out
        if c["bits"] == 8:                                                          # values in, the cache out and in, its values out
            moved += n_kv * (size * values + 4 * (values + 4 * c["tokens"]) + 4 * values)
        elif c["bits"]:
            moved += n_kv * (size * values + 4 * values)
        return {"bytes": moved, "flops": 10 * values * (n_q + n_kv)}
    old, new = _lengths(c)
    total = int(new.sum())
    pages = int((-(-(old + new) // c["page"]) + (-old // c["page"])).sum())
    return {"bytes": 12 * total + 8 * pages + 20 * c["batch"], "flops": 4 * total + 10 * c["batch"]}


# ------------------------------------------------------- values in 64 bits --

def _exact_weights(s, e):
    """One expert's weights, group by group."""
    group = s["case"]["group"]
    half = s["q"][e].double().add_(0.5)
    return half.mul_(s["s"][e].double().repeat_interleave(group, 1)).add_(s["z"][e].double().repeat_interleave(group, 1))


def _exact_rows(x):
    """Rows read back from the 8-bit cache: each value's nearest midpoint, the grid held in fp16."""
    low, high = x.min(-1).values.unsqueeze(-1), x.max(-1).values.unsqueeze(-1)
    step, low = ((high - low) / 256).half().double(), low.half().double()
    cell = ((x - low) / step).floor().clamp(0, 255)
    return torch.where(step > 0, low + (cell + 0.5) * step, low)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == _LINEAR:
        return s["x"].double() @ _exact_weights(s, 0).T
    if c["op"] == _EXPERTS:
        ends = s["ends"].tolist()
        x = s["x"].double() if s["rows"] is None else s["x"].double().index_select(0, s["rows"])
        y = torch.empty(len(x), c["d_out"], dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            if ends[e] < ends[e + 1]:
                y[ends[e]:ends[e + 1]] = x[ends[e]:ends[e + 1]] @ _exact_weights(s, e).T
        return y
    if c["op"] == _PAGES:
        return None
    turned, n_kv, out = c["turned"], c["heads"], []
    turn = torch.polar(torch.ones_like(s["freqs"]).expand(c["tokens"], -1), torch.outer(s["positions"].double(), s["freqs"]))
    for x, weight in zip((s["q"], s["k"]), s["weights"]):
        x = x.double().clone()
        if weight is not None:
            x = x / (x.square().sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * weight.double()
        part = x[..., :turned]
        if c["pairs"] == "halves":
            part = part.unflatten(-1, (2, -1)).transpose(-1, -2)
        else:
            part = part.unflatten(-1, (-1, 2))
        part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn.unsqueeze(1))
        x[..., :turned] = part.transpose(-1, -2).flatten(-2) if c["pairs"] == "halves" else part.flatten(-2)
        out.append(x)
    if c["bits"] == 8:
        out += [_exact_rows(w.to(s["q"].dtype).double()) for w in (out[1], s["v"])]
    elif c["bits"]:
        for w in (out[1], s["v"]):
            pool = torch.zeros(len(s["pools"][0]), n_kv, c["page"], c["dim"], dtype=torch.float64, device="cuda")
            pool[s["slots"] // c["page"], :, s["slots"] % c["page"]] = w.double()
            out.append(pool)
    return out
