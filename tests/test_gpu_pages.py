"""GPU parity of the page plan (grinqh_kv_extend, grinqh_kv_release) with the
oracle, number by number."""

import numpy as np
import pytest

from oracle import decoder_oracle as O
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import input_adaptive_bit_amd as G
    G.load()
    return require_gpu()


def pool(rng, lens, page, columns, spare, n_pages=None):
    """A table whose sequences hold their pages, and the list of the others."""
    held = [min(-(-max(int(n), 0) // page), columns) for n in lens]
    n_pages = n_pages or max(1, sum(held) + spare)
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), columns), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - at] = order[at:]
    return table, free, n_pages - at


def run(dev, table, lens, new, free, n_free, page, capacity, in_place=False, stride=0):
    import input_adaptive_bit_amd as G
    import torch
    wide = torch.full((table.shape[0], table.shape[1] + stride), 77, dtype=torch.int32, device=dev)
    t = wide[:, :table.shape[1]]
    t.copy_(torch.from_numpy(table))
    d = [torch.from_numpy(np.asarray(x, np.int32)).to(dev) for x in (lens, new, free, [n_free])]
    step = G.kv_extend(t, *d, page, capacity, in_place=in_place)
    torch.cuda.synchronize()
    if in_place:
        assert step.seq_lens is d[0] and step.n_free is d[3]
    else:
        assert np.array_equal(d[0].cpu().numpy(), lens) and int(d[3]) == n_free
    assert np.array_equal(d[2].cpu().numpy(), free) and (wide[:, table.shape[1]:] == 77).all()
    got = {k: getattr(step, k).cpu().numpy() for k in ("slots", "positions", "seq_lens", "cu_q", "cu_k")}
    return {**got, "table": t.cpu().numpy(), "n_free": int(step.n_free), "refused": int(step.refused)}


def same(got, want):
    for key, value in want.items():
        assert np.array_equal(got[key], value), (key, got[key], value)


@pytest.mark.parametrize("batch,longest,most,page", [(1, 0, 1, 16), (1, 100, 1, 64), (3, 50, 40, 16), (48, 800, 1, 32), (64, 300, 90, 256),
                                                     (65, 300, 200, 16), (700, 200, 30, 64), (1500, 40, 9, 16), (2, 10, 9000, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_steps_match_the_oracle(dev, batch, longest, most, page, in_place):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, longest + 1, batch)
    new = rng.integers(0, most + 1, batch) if most > 1 else np.ones(batch, np.int64)
    lens[::4], new[1::5] = 0, 0
    columns = int(max(-(-(lens + new) // page))) + 1
    need = int((-(-(lens + new) // page) + (-lens // page)).sum())
    for spare, pad in ((need, 0), (need + 5, 13), (need - 1, 3), (need // 2, 1), (0, 2)):
        table, free, n_free = pool(rng, lens, page, columns, max(spare, 0))
        capacity = int(new.sum()) + pad
        say(f"kv_extend batch={batch} new={int(new.sum())} page={page} free={n_free} of {need}")
        same(run(dev, table, lens, new, free, n_free, page, capacity, in_place, stride=pad),
             O.extend(table, lens, new, free, n_free, page, capacity))


def test_what_does_not_fit_is_refused_and_the_rest_served(dev):
    """Past the table's columns, past the capacity, and lengths and counts that are negative or very large."""
    rng = np.random.default_rng(0)
    lens = np.array([10, 16, 31, 0, -5, 33, 2 ** 31 - 1, 5, 0])
    new = np.array([1, 17, 1, 60, 3, -4, 2 ** 31 - 1, 0, 4])
    held = np.where(lens > 100, 0, lens)
    for columns, capacity in ((4, 200), (2, 200), (4, 20), (3, 0), (4, 5000)):
        table, free, n_free = pool(rng, held, 16, columns, 40)
        same(run(dev, table, lens, new, free, n_free, 16, capacity), O.extend(table, lens, new, free, n_free, 16, capacity))


@pytest.mark.parametrize("batch", [7, 300, 1500])
@pytest.mark.parametrize("capacity", [100, 9000])
def test_sums_past_the_types_end(dev, batch, capacity):
    """Lengths and counts whose sums pass 32 bits many times over: the ends stop at the largest number, and the sequences
    ahead of those counts are served as ever."""
    rng = np.random.default_rng(batch)
    lens, new = rng.integers(0, 40, batch), rng.integers(0, 3, batch)
    held = lens.copy()
    for at in (batch // 2, batch // 2 + 1, batch - 2, batch - 1):
        lens[at], new[at] = (2 ** 31 - 1, 0) if at % 2 else (3, 2 ** 31 - 1)
        held[at] = 0
    lens[batch // 2 + 2], new[batch // 2 + 2] = 0, 5
    held[batch // 2 + 2] = 0
    table, free, n_free = pool(rng, held, 16, 4, 2 * batch)
    for in_place in (False, True):
        say(f"kv_extend batch={batch} capacity={capacity} in place={in_place}")
        same(run(dev, table, lens, new, free, n_free, 16, capacity, in_place), O.extend(table, lens, new, free, n_free, 16, capacity))


def test_numbers_that_name_no_page(dev):
    """A table or list with entries outside the pool, and a count outside the list: no slot comes of them."""
    rng = np.random.default_rng(1)
    lens, new = np.array([20, 3, 0, 40]), np.array([5, 20, 40, 1])
    table, free, n_free = pool(rng, lens, 16, 5, 9)
    table[0, 1], table[3, 2] = 2 ** 30, -9
    free[n_free - 2], free[n_free - 3] = -1, 2 ** 31 - 1
    for count in (n_free, 0, -3, 2 ** 31 - 1):
        say(f"kv_extend n_free={count}")
        same(run(dev, table, lens, new, free, count, 16, 80), O.extend(table, lens, new, free, count, 16, 80))


def test_no_sequences_and_no_room(dev):
    import input_adaptive_bit_amd as G
    import torch
    free, n_free = G.new_page_list(5, dev)
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    for capacity in (0, 7, 5000):
        step = G.kv_extend(torch.zeros(0, 3, dtype=torch.int32, device=dev), none, none, free, n_free, 16, capacity)
        assert int(step.n_free) == 5 and int(step.refused) == 0 and step.cu_q.tolist() == [0] and step.cu_k.tolist() == [0]
        assert (step.slots == -1).all() and (step.positions == 0).all() and len(step.slots) == capacity


@pytest.mark.parametrize("batch,longest,page", [(1, 40, 16), (17, 100, 16), (40, 3000, 32), (1100, 60, 16), (2500, 20, 256)])
def test_pages_come_back(dev, batch, longest, page):
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, longest + 1, batch)
    columns = int(max(-(-lens // page))) + 2
    table, free, n_free = pool(rng, lens, page, columns, 6)
    for share in (0.0, 0.1, 0.5, 1.0):
        say(f"kv_release batch={batch} share={share}")
        finished = rng.random(batch) < share
        t, d, f, c = (torch.from_numpy(np.asarray(x, np.int32)).to(dev) for x in (table, lens, free, [n_free]))
        done = torch.from_numpy(finished).to(dev)
        G.kv_release(t, d, done if share < 0.3 else done.to(torch.uint8) * 3, f, c, page)
        want = O.release(table, lens, finished, free, n_free, page)
        for got, value in zip((t, d, f, c), (*want[:3], [want[3]])):
            assert np.array_equal(got.cpu().numpy(), value)


def test_release_passes_over_what_names_no_page_and_drops_what_the_list_cannot_hold(dev):
    import input_adaptive_bit_amd as G
    import torch
    table = np.array([[3, -1, 2 ** 30, 5], [1, 2, 0, 4], [9, 9, 9, 9]], np.int32)
    lens, finished = np.array([64, 2 ** 31 - 1, 33]), np.array([1, 1, 0], np.uint8)
    for n_free in (0, 5, 8, 10, -2, 99):
        free = np.full(10, -1, np.int32)
        t, d, f, c = (torch.from_numpy(np.asarray(x, np.int32)).to(dev) for x in (table, lens, free, [n_free]))
        G.kv_release(t, d, torch.from_numpy(finished).to(dev), f, c, 16)
        want = O.release(table, lens, finished, free, n_free, 16)
        for got, value in zip((t, d, f, c), (*want[:3], [want[3]])):
            assert np.array_equal(got.cpu().numpy(), value), n_free


def test_a_server_runs_for_many_steps(dev):
    """Sequences come, grow and go; no page is ever held twice, and none is lost."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(5)
    batch, page, n_pages = 24, 16, 90
    free, n_free = G.new_page_list(n_pages, dev)
    table = torch.full((batch, 12), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(batch, dtype=torch.int32, device=dev)
    served = 0
    for turn in range(40):
        new = np.where(lens.cpu().numpy() == 0, rng.integers(1, 90, batch), 1)
        before = lens.cpu().numpy()
        step = G.kv_extend(table, lens, torch.from_numpy(new.astype(np.int32)).to(dev), free, n_free, page, 2000, in_place=True)
        served += int((lens.cpu().numpy() - before).sum())
        held = table[table >= 0].tolist()
        spare = free[:int(n_free)].tolist()
        assert sorted(held + spare) == list(range(n_pages))
        assert np.array_equal((table >= 0).sum(1).cpu().numpy(), -(-lens.cpu().numpy() // page))
        got = step.slots[step.slots >= 0].tolist()
        assert len(set(got)) == len(got) == int((lens.cpu().numpy() - before).sum())
        done = torch.from_numpy(rng.random(batch) < 0.2).to(dev)
        G.kv_release(table, lens, done, free, n_free, page)
    assert served > 1000


def test_graph_replays_go_on_from_where_the_last_ended(dev):
    """A captured step in place: every replay adds a token to every sequence."""
    import input_adaptive_bit_amd as G
    import torch
    rng = np.random.default_rng(6)
    page, lens = 16, np.array([0, 15, 16, 40, 7])
    table, free, n_free = pool(rng, lens, page, 8, 60)
    t, d, f, c = (torch.from_numpy(np.asarray(x, np.int32)).to(dev) for x in (table, lens, free, [n_free]))
    new = torch.ones(5, dtype=torch.int32, device=dev)
    for capacity in (8, 6000):                                                        # one launch, and two
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step = G.kv_extend(t, d, new, f, c, page, capacity, in_place=True)
        for turn in range(4):
            new.copy_(torch.tensor([1, 1, 1, 1, 1], dtype=torch.int32) * (1 + turn % 2))
            want = O.extend(t.cpu().numpy(), d.cpu().numpy(), new.cpu().numpy(), free, int(c), page, capacity)
            graph.replay()
            torch.cuda.synchronize()
            got = {k: getattr(step, k).cpu().numpy() for k in ("slots", "positions", "seq_lens", "cu_q", "cu_k")}
            same({**got, "table": t.cpu().numpy(), "n_free": int(c), "refused": int(step.refused)}, want)
