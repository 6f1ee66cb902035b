"""Pages handed out and taken back on the GPU, against the same on lists."""
import random

import pytest
import torch

import paged8_ref as R8

pytestmark = pytest.mark.gpu

INVALID, CAPACITY = -1, -7


@pytest.fixture(autouse=True)
def fp32_default():
    """The files of a run share torch's default type."""
    old = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(old)


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_nvfp4_block_gb300 as M
    assert torch.cuda.is_available()
    return M


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    """A pool and its sequences, on lists and on the GPU."""

    def __init__(self, M, lens, ps, width, free, seed=0, waste=3, held=None):
        r = random.Random(seed)
        self.M, self.ps, self.lens = M, ps, list(lens)
        self.held = [-(-max(n, 0) // ps) for n in lens] if held is None else list(held)
        need = [max(0, min(h, width)) for h in self.held]
        ids = list(range(sum(need) + free + waste))
        r.shuffle(ids)
        self.table, at = [], 0
        for h in need:
            self.table.append(ids[at:at + h] + [-1] * (width - h))
            at += h
        self.free = ids[at:at + free] + [-1] * (len(ids) - free)
        self.n_free = free
        self.up()

    def up(self):
        self.d = dict(table=ints(self.table), held=ints(self.held), free=ints(self.free), n_free=ints([self.n_free]),
                      len=ints(self.lens))
        self.pool = self.M.PagePool(self.d["table"], self.d["held"], self.d["free"], self.d["n_free"], self.ps)
        self.ws = self.M.pool_workspace()

    def same(self):
        d = self.d
        assert d["table"].tolist() == self.table and d["held"].tolist() == self.held
        assert d["n_free"].tolist() == [self.n_free]
        assert d["free"].tolist()[:max(0, self.n_free)] == self.free[:max(0, self.n_free)]

    def reserve(self, rows, n_rows, with_slots=True, granted=True):
        n = len(self.lens)
        full = lambda k: torch.full((k,), -77, dtype=torch.int32, device="cuda")
        start, slot, pos, ok = full(n + 1), full(n_rows), full(n_rows), full(n)
        self.M.moe_paged_reserve(self.pool, self.d["len"], ints(rows), start, self.ws, slot=slot if with_slots else None,
                                 pos=pos if with_slots else None, granted=ok if granted else None)
        self.table, self.held, self.n_free, *want = R8.reserve(self.table, self.held, self.free, self.n_free, self.lens,
                                                               rows, self.ps, n_rows if with_slots else 0)
        assert start.tolist() == want[0]
        if with_slots:
            assert slot.tolist() == want[1] and pos.tolist() == want[2]
        if granted:
            assert ok.tolist() == want[3]
        self.same()
        return start, slot, pos

    def release(self, keep, shared=None):
        self.M.moe_paged_release(self.pool, ints(keep), self.ws, shared=None if shared is None else ints(shared))
        self.table, self.held, self.free, self.n_free = R8.release(self.table, self.held, self.free, self.n_free, keep,
                                                                   shared, self.ps)
        self.same()

    def error(self):
        return self.M.moe_workspace_error(self.ws)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 37, 255, 256, 257, 1024])
def test_rounds_of_reserve_and_release(M, ps, n):
    r = random.Random(n * ps)
    lens = [r.choice([0, 1, ps - 1, ps, ps + 1, r.randint(0, 700)]) for _ in range(n)]
    s = Server(M, lens, ps, 1000 // ps + 30, 20 * n + 5, seed=n)
    for step in range(4):
        rows = [r.choice([0, 1, 2, 16, r.randint(0, ps)]) for _ in range(n)]
        s.reserve(rows, sum(rows) + 5 if step != 1 else 1, with_slots=step != 2)
        assert s.error() == (CAPACITY if step == 1 and sum(rows) > 1 else 0)
        s.lens = [x + r.randint(0, k) for x, k in zip(s.lens, rows)]
        s.d["len"].copy_(ints(s.lens))
        s.release([x if r.random() < 0.8 else 0 for x in s.lens])
        for b, h in enumerate(s.held):  # ended sequences begin again
            if h == 0:
                s.lens[b] = 0
        s.d["len"].copy_(ints(s.lens))
        assert s.error() == 0


def test_long_prompts_over_many_ctas(M):
    lens = [0, 5000, 17, 0, 40000]
    s = Server(M, lens, 16, 6000, 9000, seed=3)
    s.reserve([50001, 3, 0, 16000, 30007], 96011 + 13)
    assert s.error() == 0
    s.release(lens)
    assert s.error() == 0


def test_many_pages_and_no_slots(M):
    s = Server(M, [0] * 700, 16, 100, 60000)
    s.reserve([1599] * 700, 0, with_slots=False, granted=False)
    assert s.error() == CAPACITY  # 70,000 pages are wanted
    assert s.n_free == 0 and sum(s.held) == 60000
    s.release([0] * 700)
    assert s.error() == 0


@pytest.mark.parametrize("free", [0, 1, 4, 5, 9, 10])
def test_a_pool_that_runs_short(M, free):
    # pages wanted: 2, 0, 3, 5 -- the first that do not fit end the granting of pages, not of rows in pages held
    s = Server(M, [16, 3, 0, 40], 16, 20, free)
    s.reserve([20, 5, 33, 80], 150)
    assert s.error() == (0 if free == 10 else CAPACITY)


def test_sequences_past_their_tables(M):
    s = Server(M, [60, 64, 10], 16, 4, 50)
    s.reserve([4, 1, 30], 40)  # the second needs a fifth page; the third is served all the same
    assert s.error() == CAPACITY
    assert s.held == [4, 4, 3]


@pytest.mark.parametrize("what", ["len", "rows", "held", "held2"])
def test_bad_sequences_are_skipped(M, what):
    s = Server(M, [20, 30, 40], 16, 6, 20, held=[2, 2, 3])
    rows = [20, 20, 20]
    if what == "len":
        s.lens[1] = -(2 ** 31)
    if what == "rows":
        rows[1] = -3
    if what.startswith("held"):
        s.held[1] = -1 if what == "held" else 7
    s.up()
    s.reserve(rows, 64)
    assert s.error() == INVALID
    if what.startswith("held"):
        s.release([0, 0, 0])
        assert s.error() == INVALID


@pytest.mark.parametrize("n_free", [-1, -(2 ** 31), 10 ** 6, 2 ** 31 - 1])
def test_a_bad_count_of_free_pages_is_none(M, n_free):
    s = Server(M, [20, 30], 16, 6, 20)
    s.n_free = n_free
    s.up()
    s.reserve([1, 100], 101)  # only the rows that fit held pages
    assert s.error() == INVALID
    s.release([0, 0])
    assert s.error() == INVALID


def test_lengths_and_rows_at_the_end_of_their_type(M):
    top = 2 ** 31 - 1
    s = Server(M, [top, 5, 7], 16, 6, 20, held=[0, 1, 1])
    s.reserve([top, top, top], 50)
    assert s.error() == CAPACITY


def test_bad_pages_on_the_stack_get_no_slot(M):
    s = Server(M, [0, 0], 16, 4, 6)
    s.free[5], s.free[3] = -5, 10 ** 6
    s.up()
    s.reserve([16, 50], 70)
    assert s.error() == INVALID


def test_a_stack_without_room_keeps_the_pages(M):
    s = Server(M, [40, 40, 0], 16, 4, 2, waste=0)
    s.n_free = 7  # the first sequence's pages are said to be free already
    s.up()
    s.release([0, 0, 0])
    assert s.error() == INVALID
    s.n_free = 5
    s.up()
    s.release([0, 0, 0])  # room for the first one's three only
    assert s.error() == INVALID


def test_shared_pages_stay(M):
    s = Server(M, [100, 100, 100], 16, 8, 3)
    s.release([0, 50, 100], shared=[2, 5, 100])
    assert s.error() == 0 and s.held == [2, 5, 7]
    s.release([0, 0, 0], shared=[-1, 0, 7])
    assert s.error() == 0 and s.held == [0, 0, 7]


def test_a_release_undoes_a_reserve(M):
    lens = [31 * i % 200 for i in range(300)]
    s = Server(M, lens, 16, 40, 2000, seed=5)
    before = {n: t.clone() for n, t in s.d.items()}
    s.reserve([i % 19 for i in range(300)], 3000)
    s.release(lens)
    assert all(torch.equal(before[n], t) for n, t in s.d.items()) and s.error() == 0


def test_captured_and_replayed(M):
    """A graph of reserve and release whose inputs change between replays."""
    lens = [10 * i for i in range(40)]
    s = Server(M, lens, 16, 60, 500, seed=9)
    rows, start = ints([0] * 40), torch.zeros(41, dtype=torch.int32, device="cuda")
    slot = torch.zeros(800, dtype=torch.int32, device="cuda")
    keep = ints(lens)
    M.moe_paged_reserve(s.pool, s.d["len"], rows, start, s.ws, slot=slot)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_paged_reserve(s.pool, s.d["len"], rows, start, s.ws, slot=slot)
        M.moe_paged_release(s.pool, keep, s.ws)
    for step in range(5):
        r = [(7 * i + step) % 18 for i in range(40)]
        rows.copy_(ints(r))
        keep.copy_(ints([n + k // 2 for n, k in zip(lens, r)]))
        g.replay()
        s.table, s.held, s.n_free, st, sl, _, _ = R8.reserve(s.table, s.held, s.free, s.n_free, lens, r, 16, 800)
        assert start.tolist() == st and slot.tolist() == sl
        s.table, s.held, s.free, s.n_free = R8.release(s.table, s.held, s.free, s.n_free, keep.tolist(), None, 16)
        s.same()
    assert s.error() == 0


def test_on_another_stream(M):
    s = Server(M, [5, 50], 16, 8, 9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    rows = ints([20, 20])
    torch.cuda.synchronize()
    M.moe_paged_reserve(s.pool, s.d["len"], rows, start, s.ws, stream=side)
    side.synchronize()
    s.table, s.held, s.n_free, *_ = R8.reserve(s.table, s.held, s.free, s.n_free, s.lens, [20, 20], 16, 0)
    s.same()


@pytest.mark.parametrize("n", [64, 65, 300, 1024])
def test_pages_without_slots_over_many_ctas(M, n):
    """Rounds of one graph, a few pages a sequence up to hundreds, more asked for than there are in some."""
    s = Server(M, [0] * n, 16, 300, 40 * n, seed=n)
    rows, start = ints([0] * n), torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    M.moe_paged_reserve(s.pool, s.d["len"], rows, start, s.ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_paged_reserve(s.pool, s.d["len"], rows, start, s.ws)
    r = random.Random(n)
    for step in range(4):
        want = [r.choice([0, 1, 17, 16 * r.randint(0, 80), 4800 if step == 2 else 3]) for _ in range(n)]
        rows.copy_(ints(want))
        g.replay()
        s.table, s.held, s.n_free, st, *_ = R8.reserve(s.table, s.held, s.free, s.n_free, s.lens, want, 16, 0)
        assert start.tolist() == st
        s.same()
        s.release([0] * n if step == 2 else [min(16 * h, 40) for h in s.held])
    assert s.error() in (0, CAPACITY)


@pytest.mark.parametrize("bad", [-1, -5, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [2, 90])
def test_bad_pages_in_the_table_go_back_as_they_stand(M, n, bad):
    """A release that meets them records it; so does the reserve that hands them out again, to nobody's slot."""
    s = Server(M, [40] * n, 16, 40, 5, seed=n)
    s.table[1][2] = bad
    s.up()
    s.release([40, 20] + [40] * (n - 2))
    assert s.error() == INVALID and s.free[5] == bad and s.n_free == 6 and s.held[1] == 2
    s.lens[1] = 20
    s.d["len"].copy_(ints(s.lens))
    _, slot, _ = s.reserve([0, 20] + [0] * (n - 2), 23)
    assert s.error() == INVALID and s.table[1][2] == bad
    assert (slot[:12] >= 0).all() and (slot[12:] == -1).all()
    s.release([0] * n)
    assert s.error() == INVALID and s.n_free == 5 + 3 * n and s.free.count(bad) == 1 + (bad == -1) * (len(s.free) - s.n_free)
