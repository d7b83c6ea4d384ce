"""gptq_page_plan against the same plan made sequence by sequence in Python: whole numbers, all equal."""
import numpy as np
import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


def plan(cached, added, page, table, free, count, max_tokens):
    """(seq_lens, cu, positions, slots, table, free, count, status) by the definition."""
    table, free, status = table.copy(), free.copy(), 0
    B, width = table.shape
    most = width * page
    need = lambda n: -(-n // page)  # noqa: E731
    cut = max(0, min(count, len(free)))
    if cut != count:
        status |= g.DEV_NO_PAGE
    count = cut
    changes = []
    for a, d in zip(cached, added):
        c = max(0, min(a, most))
        n = c + d
        if c != a or n < 0 or n > most:
            status |= g.DEV_SEQ_LEN
        changes.append([c, None if n > most else max(0, n), max(0, d)])
    for b, (c, n, m) in enumerate(changes):
        for j in range(need(n), need(c)) if n is not None else ():
            if count < len(free):
                free[count] = table[b, j]
                count += 1
            else:
                status |= g.DEV_NO_PAGE
    short = False
    top = count
    for b, ch in enumerate(changes):
        c, n, m = ch
        take = max(0, need(n) - need(c)) if n is not None else 0
        if take == 0:
            continue
        short = short or take > top
        if short:
            status |= g.DEV_NO_PAGE
            ch[1] = None
            continue
        for j in range(take):
            top -= 1
            table[b, need(c) + j] = free[top]
    cu, positions, slots, lens = [0], [], [], []
    for b, (c, n, m) in enumerate(changes):
        for t in range(c, c + m):
            positions.append(t)
            slots.append(int(table[b, t // page]) * page + t % page if n is not None else -1)
        cu.append(cu[-1] + m)
        lens.append(c if n is None else n)
    if cu[-1] > max_tokens:
        status |= g.DEV_TOKEN_ROWS
    pad = max(0, max_tokens - len(slots))
    cu = np.minimum(cu, max_tokens)
    return lens, cu, (positions + [0] * pad)[:max_tokens], (slots + [-1] * pad)[:max_tokens], table, free, top, status


class Case:
    def __init__(self, cached, added, page, spare=0, width=None, room=0, seed=0, pad=0):
        rng = np.random.default_rng(seed)
        self.page, self.cached, self.added = page, list(cached), list(added)
        need = [-(-max(0, a) // page) for a in cached]
        most = max([1] + [-(-max(a, a + d) // page) for a, d in zip(cached, added)])
        width = width or most
        take = sum(max(0, -(-(a + d) // page) - n) for a, d, n in zip(cached, added, need))
        pages = sum(need) + max(0, take + spare)
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(cached), width), -9, np.int32)
        for b, n in enumerate(need):
            self.table[b, :min(n, width)] = order[:n][:width]
            order = order[n:]
        self.count = len(order)
        self.free = np.concatenate([order, np.full(sum(need) + room, -7, np.int32)])
        self.tokens = sum(max(0, d) for d in added) + pad

    def run(self, max_tokens=None, in_place=False, count=None, stream=None):
        d = lambda x: torch.from_numpy(np.asarray(x, np.int32).copy()).to(DEV)  # noqa: E731
        T = self.tokens if max_tokens is None else max_tokens
        count = self.count if count is None else count
        cached, table, free, n = d(self.cached), d(self.table), d(self.free), d([count])
        n_out = n if in_place else d([0])
        got = g.page_plan(cached, d(self.added), table, free, n, page_size=self.page, max_tokens=T, seq_lens=cached if in_place else None,
                          free_count_out=None if in_place else n_out, stream=stream)
        torch.cuda.synchronize()
        want = plan(self.cached, self.added, self.page, self.table, self.free, count, T)
        assert g.device_status() == want[7]
        for name, a, b in zip(("seq_lens", "cu", "positions", "slots", "table", "free", "count"), list(got) + [table, free, n_out],
                              list(want[:6]) + [[want[6]]]):
            assert np.array_equal(a.cpu().numpy(), np.asarray(b)), name
        if not in_place:
            assert int(n) == count and np.array_equal(cached.cpu().numpy(), self.cached)
        return want


def spread(B, most, seed):
    return np.random.default_rng(seed).integers(0, most + 1, B).tolist()


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("batch", [1, 2, 31, 33, 300, 513])
def test_steps_of_one_token(batch, page):
    Case(spread(batch, 200, batch), [1] * batch, page, spare=3, seed=page).run()


@pytest.mark.parametrize("page", [1, 13, 16])
@pytest.mark.parametrize("batch", [1, 5, 64, 700])
def test_chunks_waits_drops_and_ends(batch, page):
    cached = spread(batch, 300, batch + 1)
    added = [(40 * i) % 97 if i % 3 == 0 else (-a if i % 7 == 1 else -min(a, i % 20) if i % 5 == 2 else i % 2) for i, a in enumerate(cached)]
    w = Case(cached, added, page, spare=2, seed=page, pad=9).run()
    assert w[7] == 0
    Case(cached, added, page, spare=2, seed=page, pad=9).run(in_place=True)


def test_fresh_prompts_and_one_very_long_one():
    Case([0] * 6, [1, 16, 17, 0, 100000, 33], 16, spare=1).run()
    Case([0], [1], 16).run()
    Case([5], [0], 16).run()
    Case([100000, 3], [-100000, 60], 16, spare=0).run()


def test_pages_given_back_are_taken_in_the_same_step():
    c = Case([64, 0], [-64, 60], 16, spare=-4)    # nothing is free but what the first gives back
    assert c.count == 0
    assert c.run()[7] == 0


@pytest.mark.parametrize("spare", [-1, -5, -1000])
def test_too_few_pages(spare):
    cached = [10, 16, 0, 7, 30, 32, 5]
    added = [1, 1, 40, 2, 100, 1, -2]
    assert Case(cached, added, 16, spare=spare).run()[7] == g.DEV_NO_PAGE


def test_too_long_negative_and_too_many():
    c = Case([10, 20, 30], [5, 30, 1], 16, spare=3, width=3)      # the second would be 50 of 48
    assert c.run()[7] == g.DEV_SEQ_LEN
    c = Case([10, 20, 30], [2, -25, 1], 16, spare=3)
    assert c.run()[7] == g.DEV_SEQ_LEN
    c = Case([10, 20, 30], [10 ** 6, -2 ** 31, 1], 16, spare=-2 ** 40, width=4)
    assert c.run(max_tokens=50)[7] & (g.DEV_SEQ_LEN | g.DEV_TOKEN_ROWS)
    c = Case([10, 20, 30], [2, 3, 40], 16, spare=3)
    c.cached[0] = -4
    assert c.run()[7] == g.DEV_SEQ_LEN
    assert Case([10, 20, 30], [20, 30, 40], 16, spare=3).run(max_tokens=37)[7] == g.DEV_TOKEN_ROWS
    assert Case([10, 20], [1, 1], 16).run(max_tokens=0)[7] == g.DEV_TOKEN_ROWS


def test_a_list_without_room_and_a_wrong_count():
    c = Case([64, 40, 20], [-64, 0, -20], 16)
    c.free = c.free[:c.count + 3]                 # six pages come back
    assert c.run()[7] == g.DEV_NO_PAGE
    c = Case([64, 40], [1, 1], 16, spare=2)
    c.run(count=-3)
    c.run(count=10 ** 6)


def test_largest_batch():
    batch = 8192
    cached = spread(batch, 40, 3)
    added = [i % 3 - 1 if a else 1 for i, a in enumerate(cached)]
    Case(cached, added, 8, spare=5, pad=100).run()


def test_no_sequences():
    got = g.page_plan(*(torch.zeros(0, dtype=torch.int32, device=DEV) for _ in range(2)), torch.zeros((0, 4), dtype=torch.int32, device=DEV),
                      torch.zeros(3, dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV), page_size=16, max_tokens=5)
    assert got[0].shape == (0,) and got[1].tolist() == [0] and got[2].tolist() == [0] * 5 and got[3].tolist() == [-1] * 5


def test_steps_one_after_the_other_captured():
    # ten steps in place: the pages in use are always as many as the lengths need, each of them once
    batch, page, width = 50, 4, 12
    rng = np.random.default_rng(1)
    total = batch * width
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
    lens, added = i32(np.zeros(batch)), i32(np.zeros(batch))
    table, free, count = i32(np.full((batch, width), -1)), i32(rng.permutation(total)), i32([total])
    step = lambda: g.page_plan(lens, added, table, free, count, page_size=page, max_tokens=400, seq_lens=lens)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, cu, positions, slots = step()
    now = np.zeros(batch, int)
    for turn in range(10):
        d = rng.integers(-6, 9, batch)
        d = np.clip(now + d, 0, page * width) - now
        added.copy_(i32(d))
        graph.replay()
        torch.cuda.synchronize()
        now = now + d
        assert np.array_equal(lens.cpu().numpy(), now)
        t = table.cpu().numpy()
        used = np.concatenate([t[b, :-(-n // page)] for b, n in enumerate(now)])
        rest = free.cpu().numpy()[:int(count)]
        assert len(set(used.tolist())) == len(used) and sorted(np.concatenate([used, rest]).tolist()) == list(range(total))
        at = 0
        for b, m in enumerate(np.maximum(d, 0)):
            for x in range(now[b] - m, now[b]):
                assert int(positions[at]) == x and int(slots[at]) == t[b, x // page] * page + x % page
                at += 1
        assert int(cu[-1]) == at and bool((slots[at:] == -1).all())
    assert g.device_status() == 0


def test_on_another_stream():
    Case([10, 64, 31], [7, -64, 1], 16, spare=2).run(stream=torch.cuda.Stream())


def test_wrong_tensors_are_refused():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    a = dict(cached=i32(2), added=i32(2), block_table=i32(2, 3), free_pages=i32(5), free_count=i32(1), page_size=16, max_tokens=4)
    for kw in (dict(cached=i32(2).cpu()), dict(added=i32(3)), dict(block_table=i32(3, 3)), dict(free_pages=i32(5, 1)), dict(free_count=i32(2)),
               dict(max_tokens=-1), dict(seq_lens=i32(3)), dict(added=i32(4)[::2])):
        with pytest.raises(ValueError):
            g.page_plan(**dict(a, **kw))
    for kw in (dict(cached=i32(2).long()), dict(free_count=i32(1).long())):
        with pytest.raises(TypeError):
            g.page_plan(**dict(a, **kw))
    with pytest.raises(g.GPTQError) as e:
        g.page_plan(**dict(a, page_size=0))
    assert e.value.code == -2
