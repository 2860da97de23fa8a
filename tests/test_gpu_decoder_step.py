"""A decoder layer's operators run together, as a server uses them: pages for the
step, q|k|v product, norms and rotation into the cache, attention, o product,
experts' products; prompts first, then single tokens, some sequences leaving and
new ones coming.  Every stage is held against the fp64 oracle on what the stage
before it gave, with that stage's own bound (derived where its other tests are),
and the cache's contents against all keys and values so far."""

import numpy as np
import pytest

from oracle import attention_oracle as A
from oracle import decoder_oracle as O
from tests.attention_util import HALF, U, W_DECODE, W_PREFILL, head_bound, inside, to_type
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, MODEL, EXPERTS, TOP, GROUP, PAGE = 6, 2, 64, 256, 5, 2, 64, 16


@pytest.fixture(scope="module")
def dev():
    import input_adaptive_bit_amd as G
    G.load()
    return require_gpu()


def numbers(t):
    return t.float().cpu().numpy().astype(np.float64)


class Weights:
    def __init__(self, rng, experts, d_in, d_out, dev):
        import input_adaptive_bit_amd as G
        import torch
        groups = d_in // GROUP
        self.q = rng.integers(0, 16, (experts, d_out, d_in)).astype(np.uint8)
        self.s = (rng.random((experts, d_out, groups)) * 0.01 + 0.005).astype(np.float16)
        self.z = (-8 * self.s.astype(np.float32)).astype(np.float16)
        self.dev = G.fourbit_pack(*(torch.from_numpy(v).to(dev) for v in (self.q, self.s, self.z)))

    def check(self, got, x, ends=None, rows=None):
        if ends is None:
            want, size = O.linear(numbers(x), self.q[0], self.s[0], self.z[0], GROUP)
        else:
            want, size, written = O.experts(numbers(x), ends, rows, len(got), self.q, self.s, self.z, GROUP)
            assert written.all()
        d_in = self.q.shape[2]
        inside(numbers(got), want, (GROUP + 3 * (d_in // GROUP) + 32) * 2.0 ** -23 * size + HALF["bf16"] * np.abs(want) + 1e-30)


class Layer:
    def __init__(self, dev, bits):
        import input_adaptive_bit_amd as G
        import torch
        rng = np.random.default_rng(bits)
        self.dev, self.bits, self.batch, pages = dev, bits, 4, 60
        self.qkv = Weights(rng, 1, MODEL, (HEADS + 2 * KV) * DIM, dev)
        self.o = Weights(rng, 1, HEADS * DIM, MODEL, dev)
        self.experts = Weights(rng, EXPERTS, MODEL, MODEL, dev)
        self.norms = [to_type(A.bf16(1 + 0.2 * rng.standard_normal(DIM).astype(np.float32)), "bf16", dev) for _ in range(2)]
        self.freqs = torch.from_numpy(10000.0 ** -(np.arange(0, DIM, 2) / DIM)).to(dev)
        self.cache = G.new_kv_cache(KV, DIM, PAGE, pages, bits, dev)
        self.free, self.n_free = G.new_page_list(pages, dev)
        self.table = torch.full((self.batch, 12), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(self.batch, dtype=torch.int32, device=dev)
        self.ws = G.new_attention_workspace(self.cache.layout, HEADS, self.batch, 192, dev)
        self.seen = [([], []) for _ in range(self.batch)]                # the oracle's copy of what is cached

    def step(self, x, new):
        """x [tokens][MODEL] of the sequences' new tokens, packed."""
        import input_adaptive_bit_amd as G
        import torch
        lens = self.lens.cpu().numpy()
        single = max(new) == 1 and (lens + new > 0).all()
        plan = G.kv_extend(self.table, self.lens, torch.tensor(new, dtype=torch.int32, device=self.dev), self.free, self.n_free,
                           PAGE, len(x) + 3, in_place=True)
        n = len(x)
        qkv = G.fourbit_linear(self.qkv.dev, x).view(n, -1, DIM)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
        slots, positions = plan.slots[:n], plan.positions[:n]
        rq, rk = G.qk_rope(q, k, positions, self.freqs, *self.norms, cache=self.cache, v=v, slots=slots)
        if single:
            out = G.decode_attention(self.cache, rq, self.table, self.lens, 192, workspace=self.ws)
        elif lens.max() == 0:
            out = G.prefill_attention(rq, rk, v, plan.cu_q)
        else:                                                            # some sequences have a cached beginning
            page = torch.arange(int(plan.cu_k[-1]), device=self.dev)
            seq = torch.bucketize(page, plan.cu_k[1:].long(), right=True)
            at = page - plan.cu_k.long()[seq]
            every = self.table.long()[seq, at // PAGE] * PAGE + at % PAGE
            out = G.prefill_attention(rq, *G.kv_read(self.cache, every), plan.cu_q, plan.cu_k)
        y = G.fourbit_linear(self.o.dev, out.view(n, -1))
        chosen = torch.topk(y[:, :EXPERTS].float(), TOP, -1).indices     # a router of sorts
        flat, order = chosen.flatten().sort(stable=True)
        ends = torch.cat([torch.zeros(1, dtype=torch.long, device=self.dev), torch.bincount(flat, minlength=EXPERTS).cumsum(0)]).int()
        rows = (order // TOP).int()
        z = G.expert_linear(self.experts.dev, y, ends, rows)
        torch.cuda.synchronize()
        self.check(x, new, lens, plan, q, k, v, rq, rk, out, y, z, ends, rows, single)
        return z

    def check(self, x, new, lens, plan, q, k, v, rq, rk, out, y, z, ends, rows, single):
        n = len(x)
        assert int(plan.refused) == 0 and (plan.slots[n:] == -1).all()
        assert self.lens.tolist() == (lens + new).tolist()
        positions = np.concatenate([lens[b] + np.arange(new[b]) for b in range(self.batch)])
        assert plan.positions[:n].tolist() == positions.tolist()
        import torch
        qkv = torch.cat([q, k, v], 1).reshape(n, -1)
        self.qkv.check(qkv, x)
        for got, raw, weight in ((rq, q, self.norms[0]), (rk, k, self.norms[1])):
            want, size = O.rope(numbers(raw), positions, self.freqs.cpu().numpy(), numbers(weight), 1e-6)
            inside(numbers(got), want, (DIM / 2 + 20) * U * size + HALF["bf16"] * np.abs(want) + 1e-30)
        # what the cache stands for, of every sequence from its beginning
        begin = 0
        want, bound = np.zeros((n, HEADS, DIM)), np.zeros((n, HEADS, DIM))
        for b in range(self.batch):
            rows_b = slice(begin, begin + new[b])
            for kept, fresh in zip(self.seen[b], (rk, v)):
                kept.extend(numbers(fresh)[rows_b])
            begin += new[b]
            if new[b] == 0:
                continue
            keys, values = (np.array(kept) for kept in self.seen[b])
            if single or lens.max() > 0:
                keys, values = (A.row_values(*A.quantise_rows(w.astype(np.float32), self.bits), self.bits) for w in (keys, values))
                if not single:
                    keys, values = (A.bf16(w).astype(np.float64) for w in (keys, values))      # kv_read gives bf16
            mask = A.causal_mask(new[b], len(keys))
            for h in range(HEADS):
                kk, vv = keys[:, h // (HEADS // KV)], values[:, h // (HEADS // KV)]
                qq = numbers(rq)[rows_b, h]
                want[rows_b, h], _, p = A.attend(qq, kk, vv, DIM ** -0.5, mask)
                # codes enter as s c and s / 2 + z: at most three times the row's largest value each
                terms = (np.abs(kk), np.abs(vv)) if self.bits == 16 or not single else (
                    np.repeat(3 * np.abs(kk).max(1, keepdims=True), DIM, 1), np.repeat(3 * np.abs(vv).max(1, keepdims=True), DIM, 1))
                bound[rows_b, h], _ = head_bound(qq, terms[0], kk, terms[1], len(kk), p, DIM ** -0.5, W_DECODE if single else W_PREFILL,
                                                 want[rows_b, h], "bf16")
        inside(numbers(out), want, bound)
        self.o.check(y, out.reshape(n, -1))
        self.experts.check(z, y, ends.cpu().numpy(), rows.cpu().numpy())


@pytest.mark.parametrize("bits", [8, 16])
def test_prompts_tokens_and_sequences_that_come_and_go(dev, bits):
    import input_adaptive_bit_amd as G
    import torch
    layer = Layer(dev, bits)
    rng = np.random.default_rng(1)

    def tokens(n):
        return to_type(A.bf16(rng.standard_normal((n, MODEL)).astype(np.float32)), "bf16", dev)

    say(f"decoder step bits={bits}: prompts")
    layer.step(tokens(70), [33, 1, 20, 16])
    for turn in range(3):
        say(f"decoder step bits={bits}: token {turn}")
        layer.step(tokens(4), [1, 1, 1, 1])
    say(f"decoder step bits={bits}: a sequence leaves and another comes, a further prompt")
    done = torch.tensor([False, False, True, False], device=dev)
    G.kv_release(layer.table, layer.lens, done, layer.free, layer.n_free, PAGE)
    layer.seen[2] = ([], [])
    layer.step(tokens(45), [1, 18, 25, 1])
    layer.step(tokens(4), [1, 1, 1, 1])
    held = layer.table[layer.table >= 0].tolist()
    assert sorted(held + layer.free[:int(layer.n_free)].tolist()) == list(range(60))


def test_a_decode_step_in_a_graph(dev):
    """The whole step of single tokens is captured once and replayed: lengths, positions, slots and pages move on by
    themselves, and every replay gives what the same step gives eagerly."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(2)
    outs = {}
    for mode in ("eager", "graph"):
        layer = Layer(dev, 8)
        x = torch.empty(4, MODEL, dtype=torch.bfloat16, device=dev)
        new = torch.ones(4, dtype=torch.int32, device=dev)
        rng = np.random.default_rng(2)

        def step():
            plan = G.kv_extend(layer.table, layer.lens, new, layer.free, layer.n_free, PAGE, 4, in_place=True)
            qkv = G.fourbit_linear(layer.qkv.dev, x).view(4, -1, DIM)
            q, _ = G.qk_rope(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], plan.positions, layer.freqs, *layer.norms, cache=layer.cache,
                             v=qkv[:, HEADS + KV:], slots=plan.slots, keys=False)
            out = G.decode_attention(layer.cache, q, layer.table, layer.lens, 192, workspace=layer.ws)
            y = G.fourbit_linear(layer.o.dev, out.view(4, -1))
            return G.expert_linear(layer.experts.dev, y, ends, rows)

        ends = torch.tensor([0, 2, 2, 5, 7, 8], dtype=torch.int32, device=dev)
        rows = torch.tensor([0, 3, 1, 1, 2, 0, 3, 2], dtype=torch.int32, device=dev)
        got = []
        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                z = step()
        for turn in range(20):
            x.copy_(to_type(A.bf16(rng.standard_normal((4, MODEL)).astype(np.float32)), "bf16", dev))
            if mode == "graph":
                graph.replay()
            else:
                z = step()
            torch.cuda.synchronize()
            got.append(z.clone())
        assert layer.lens.tolist() == [20] * 4
        outs[mode] = got
    assert all(torch.equal(a, b) for a, b in zip(outs["eager"], outs["graph"]))
