"""GPU: pages given to new tokens (chain_page_plan) and taken back (chain_page_trim), against a plain loop over
sequences and pages.  Whole numbers: every result is compared for equality."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cg():
    import chain_gb300
    chain_gb300.lib()
    return chain_gb300


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32)


class State:
    """Sequences of a pool with their pages, the rest on the stack; unused entries hold nonsense."""

    def __init__(self, lens, page, max_pages, spare, seed=0, extra=3):
        rng = random.Random(seed)
        need = [-(-L // page) for L in lens]
        self.pool = sum(need) + spare
        ids = list(range(self.pool))
        rng.shuffle(ids)
        self.page, self.max_pages, self.lens, self.count = page, max_pages, list(lens), spare
        self.table = [[-9 - b] * max_pages for b in range(len(lens))]
        for b, m in enumerate(need):
            for k in range(m):
                self.table[b][k] = ids.pop()
        self.free = ids + [-77] * (sum(need) + extra)
        assert len(ids) == spare

    def cuda(self, wide=0):
        t = torch.full((max(len(self.lens), 1), self.max_pages + wide), -5, dtype=torch.int32)
        if self.lens:
            t[:, :self.max_pages] = ints(self.table)
        self.tabled = t.cuda()[:len(self.lens), :self.max_pages]
        self.freed, self.countd, self.lensd = ints(self.free).cuda(), ints([self.count]).cuda(), ints(self.lens).cuda()
        return self

    def plan(self, news, rows):
        """The definition; returns (cu, positions, slots) and keeps the new state."""
        cu, positions, slots = [0], [], []
        for b, n in enumerate(news):
            n = max(0, min(n, rows - cu[-1]))
            L = self.lens[b]
            for k in range(-(-L // self.page), min(-(-(L + n) // self.page), self.max_pages)):
                self.count -= 1
                self.table[b][k] = self.free[self.count] if self.count >= 0 else -1
            for p in range(L, L + n):
                k = p // self.page
                e = self.table[b][k] if k < self.max_pages else -1
                positions.append(p)
                slots.append(-1 if e < 0 else e * self.page + p % self.page)
            cu.append(cu[-1] + n)
            self.lens[b] = L + n
        self.count = max(self.count, 0)
        rest = [-1] * (rows - len(positions))
        return cu, positions + rest, slots + rest

    def trim(self, keeps):
        for b, keep in enumerate(keeps):
            L, left = self.lens[b], max(0, min(self.lens[b], keep))
            for k in range(-(-left // self.page), -(-L // self.page)):
                e = self.table[b][k]
                if 0 <= e < self.pool:
                    if self.count < len(self.free):
                        self.free[self.count] = e
                    self.count += 1
            self.lens[b] = left
        self.count = min(self.count, len(self.free))

    def same(self, kv, count, table=None, free=None):
        assert kv.tolist() == self.lens and count.tolist() == [self.count]
        if table is not None:
            assert table.tolist() == self.table
        if free is not None:
            assert free.tolist() == self.free


# lens, new tokens, page, rows behind the last
PLANS = {
    "one token, new page": ([64], [1], 64, 0),
    "one token, same page": ([63], [1], 64, 0),
    "first token": ([0], [1], 16, 3),
    "nothing new": ([5, 0, 16], [0, 0, 0], 16, 2),
    "single tokens": ([(37 * i) % 300 for i in range(90)], [1] * 90, 16, 7),
    "some without": ([(37 * i) % 300 for i in range(100)], [i % 3 for i in range(100)], 32, 0),
    "prompts": ([0] * 9, [700, 1, 16, 17, 15, 0, 32, 33, 64], 16, 5),
    "chunks": ([10, 100, 31, 32, 33], [200, 0, 1, 64, 3000], 32, 1),
    "large pages": ([1000, 0, 1024, 1025], [30, 2000, 1, 0], 1024, 0),
    "most of one block": ([7 * i % 40 for i in range(1024)], [8] * 1024, 16, 0),
    "more rows than one block": ([5, 0, 77], [8000, 300, 1], 16, 200),
    "more sequences than one block": ([(11 * i) % 70 for i in range(1025)], [1 + i % 3 for i in range(1025)], 16, 9),
    "largest batch": ([(11 * i) % 70 for i in range(8192)], [i % 2 for i in range(8192)], 16, 100),
    "long rows": ([100000, 3, 0, 16], [70001, 0, 0, 131072], 64, 0),
}


def plan(cg, s, news, rows, **kw):
    return cg.page_plan(ints(news).cuda(), s.lensd, s.tabled, s.freed, s.countd, s.page, rows, **kw)


@pytest.mark.parametrize("name", PLANS)
def test_plan(cg, name):
    lens, news, page, pad = PLANS[name]
    most = max(-(-(L + n) // page) for L, n in zip(lens, news)) + 2
    need = sum(-(-(L + n) // page) + -(-L // page) * -1 for L, n in zip(lens, news))
    s = State(lens, page, most, need + 4, len(name)).cuda(wide=len(name) % 4)
    rows = sum(news) + pad
    cu, kv, count, positions, slots = plan(cg, s, news, rows)
    assert cg.chain_check()[0] == 0
    rc, rp, rs = s.plan(news, rows)
    assert cu.tolist() == rc and positions.tolist() == rp and slots.tolist() == rs
    s.same(kv, count, s.tabled, s.freed)


@pytest.mark.parametrize("news,rows", [([40, 1, 0, 300], 341), ([40, 0, 0, 9000], 9100)])
def test_plan_in_place_step_after_step(cg, news, rows):
    s = State([10, 0, 33, 900], 16, 2000, 1600, 5).cuda()
    out = (torch.empty(5, dtype=torch.int32, device="cuda"), s.lensd, s.countd,
           torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int64, device="cuda"))
    ws = torch.full((cg.chain_page_plan_workspace_size(4),), 255, dtype=torch.uint8, device="cuda")
    for step in range(2):
        cu, kv, count, positions, slots = plan(cg, s, news, rows, out=out, workspace=ws)
        assert kv is s.lensd and cg.chain_check()[0] == 0
        rc, rp, rs = s.plan(news, rows)
        assert cu.tolist() == rc and positions.tolist() == rp and slots.tolist() == rs
        s.same(s.lensd, s.countd, s.tabled)


@pytest.mark.parametrize("pad", [0, 9000])  # both forms
def test_what_a_plan_reports(cg, pad):
    base = ([20, 40, 5], 16, 6, 9)
    # the stack runs out: entries and slots of -1
    s = State(*base, seed=3).cuda()
    s.countd.fill_(2)
    s.count = 2
    news, rows = [30, 20, 10], 60 + pad
    cu, kv, count, positions, slots = plan(cg, s, news, rows)
    assert cg.chain_check()[0] == cg.ERR_ARG and cg.chain_check()[0] == 0
    rc, rp, rs = s.plan(news, rows)
    assert -1 in rs[:60]
    assert cu.tolist() == rc and positions.tolist() == rp and slots.tolist() == rs
    s.same(kv, count, s.tabled)
    # a full table: nothing is written beyond it
    s = State(*base, seed=4).cuda(wide=3)
    news = [90, 0, 1]
    cu, kv, count, positions, slots = plan(cg, s, news, 91 + pad)
    assert cg.chain_check()[0] == cg.ERR_ARG
    rc, rp, rs = s.plan(news, 91 + pad)
    assert cu.tolist() == rc and positions.tolist() == rp and slots.tolist() == rs
    s.same(kv, count, s.tabled)
    assert bool((s.tabled._base[:, 6:] == -5).all()) if s.tabled._base is not None else True
    # lengths that cannot be, counts that cannot be
    s = State(*base, seed=5).cuda()
    bad = s.lensd.clone()
    bad[1] = -4
    s.lens[1], first = 0, s.lensd
    s.lensd = bad
    cu, kv, count, positions, slots = plan(cg, s, [1, 2, -7], 3 + pad)
    assert cg.chain_check()[0] == cg.ERR_ARG
    rc, rp, rs = s.plan([1, 2, 0], 3 + pad)
    assert cu.tolist() == rc and positions.tolist() == rp and slots.tolist() == rs
    s.same(kv, count, s.tabled)
    for wrong, taken in ((-3, 0), (10 ** 6, None)):
        s = State(*base, seed=6).cuda()
        s.countd.fill_(wrong)
        s.count = len(s.free) if taken is None else taken
        kv, count = plan(cg, s, [0, 0, 0], pad)[1:3]
        assert cg.chain_check()[0] == cg.ERR_ARG
        s.same(kv, count, s.tabled)


@pytest.mark.parametrize("rows", [25, 8200])
def test_tokens_beyond_the_rows_are_left_out(cg, rows):
    s = State([3, 40, 0], 16, 1000, 900, 7).cuda()
    news = [20, rows - 15, 30]
    cu, kv, count, positions, slots = plan(cg, s, news, rows)
    assert cg.chain_check()[0] == cg.ERR_ARG
    rc, rp, rs = s.plan(news, rows)
    assert rc[-1] == rows
    assert cu.tolist() == rc and positions.tolist() == rp and slots.tolist() == rs
    s.same(kv, count, s.tabled)


TRIMS = {
    "one token": ([33], [32], 16),
    "nothing": ([33, 0, 16], [33, 5, 100], 16),
    "everything": ([33, 0, 16, 1], [0, 0, 0, 0], 16),
    "rejected tokens": ([(37 * i) % 900 + 8 for i in range(300)], [(37 * i) % 900 + 8 - i % 9 for i in range(300)], 16),
    "done ones": ([(337 * i) % 5000 for i in range(70)], [0 if i % 3 else 5000 for i in range(70)], 16),
    "long ones": ([130000, 40, 262144], [5, 40, 100000], 16),
    "most of one block": ([40] * 1024, [7] * 1024, 32),
    "largest batch": ([(11 * i) % 70 for i in range(8192)], [(7 * i) % 70 - 5 for i in range(8192)], 16),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", TRIMS)
def test_trim(cg, name, in_place):
    lens, keeps, page = TRIMS[name]
    s = State(lens, page, max(-(-L // page) for L in lens) + 1, 3, len(name)).cuda(wide=len(name) % 3)
    before = s.tabled.clone()
    out = (s.lensd, s.countd) if in_place else None
    kv, count = cg.page_trim(ints(keeps).cuda(), s.lensd, s.tabled, s.freed, s.countd, page, s.pool, out=out)
    assert cg.chain_check()[0] == 0
    s.trim(keeps)
    s.same(kv, count, s.tabled, s.freed)
    assert torch.equal(s.tabled, before)


@pytest.mark.parametrize("max_pages", [8, 50000])  # both forms
def test_what_a_trim_reports(cg, max_pages):
    # entries that name no page are not put on the stack
    for bad in (-1, 2 ** 31 - 1, -2 ** 31):
        s = State([100, 70, 20], 16, max_pages, 2, 8)
        s.table[0][3] = bad
        s.table[1][4] = s.pool
        s.cuda()
        kv, count = cg.page_trim(ints([10, 0, 20]).cuda(), s.lensd, s.tabled, s.freed, s.countd, 16, s.pool)
        assert cg.chain_check()[0] == cg.ERR_ARG and cg.chain_check()[0] == 0
        s.trim([10, 0, 20])
        s.same(kv, count, s.tabled, s.freed)
    # a stack that overflows
    s = State([100, 70, 20], 16, max_pages, 2, 9, extra=0)
    s.free = s.free[:6]
    s.cuda()
    guard = torch.full((20,), 123, dtype=torch.int32, device="cuda")
    guard[:6] = s.freed
    s.freed = guard[:6]
    kv, count = cg.page_trim(ints([0, 0, 0]).cuda(), s.lensd, s.tabled, s.freed, s.countd, 16, s.pool)
    assert cg.chain_check()[0] == cg.ERR_ARG
    s.trim([0, 0, 0])
    s.same(kv, count, s.tabled, s.freed)
    assert bool((guard[6:] == 123).all())
    # a length past the table's end counts as that
    s = State([100, 16 * 7], 16, 7, 2, 10).cuda()
    s.lensd[1] = 16 * 7 + 1
    kv, count = cg.page_trim(ints([100, 16]).cuda(), s.lensd, s.tabled, s.freed, s.countd, 16, s.pool)
    assert cg.chain_check()[0] == cg.ERR_ARG
    s.trim([100, 16])
    s.same(kv, count, s.tabled, s.freed)


LARGE_TRIMS = {
    "one sequence, all of it": ([700000], [0], 16, 43760),
    "one sequence, one page": ([700000], [699990], 16, 43760),
    "every sequence, all of it": ([(331 * i) % 1100 for i in range(1024)], [0] * 1024, 16, 70),
    "every sequence, some of it": ([(331 * i) % 1100 for i in range(1023)], [(77 * i) % 1100 for i in range(1023)], 16, 70),
    "a long one among short ones": ([5] * 200 + [300000] + [17] * 300, [1] * 200 + [40] + [3] * 300, 16, 18800),
    "one token each": ([16 * i + 1 for i in range(300)], [16 * i for i in range(300)], 16, 350),
}


@pytest.mark.parametrize("missing", [0, 7])
@pytest.mark.parametrize("name", LARGE_TRIMS)
def test_trim_of_a_large_table(cg, name, missing):
    lens, keeps, page, max_pages = LARGE_TRIMS[name]
    s = State(lens, page, max_pages, 3, len(name))
    lost, k = 0, 0
    for b, (L, keep) in enumerate(zip(lens, keeps)):  # every so often an entry that names no page
        for e in range(-(-min(L, keep) // page), -(-L // page)):
            k += 1
            if missing and k % missing == 0:
                s.table[b][e] = -1 if k % 2 else s.pool
                lost += 1
    s.cuda()
    out = (s.lensd, s.countd)
    kv, count = cg.page_trim(ints(keeps).cuda(), s.lensd, s.tabled, s.freed, s.countd, page, s.pool, out=out)
    assert cg.chain_check()[0] == (cg.ERR_ARG if lost else 0)
    s.trim(keeps)
    s.same(kv, count, s.tabled, s.freed)


def test_nothing_to_do(cg):
    s = State([], 16, 4, 5).cuda()
    cu, kv, count, positions, slots = plan(cg, s, [], 6)
    assert cu.tolist() == [0] and kv.numel() == 0 and count.tolist() == [5]
    assert positions.tolist() == slots.tolist() == [-1] * 6
    kv, count = cg.page_trim(ints([]).cuda(), s.lensd, s.tabled, s.freed, s.countd, 16, s.pool)
    assert kv.numel() == 0 and count.tolist() == [5] and cg.chain_check()[0] == 0


def test_refusals(cg):
    s = State([5, 6], 16, 4, 5).cuda()
    with pytest.raises(ValueError):
        cg.page_plan(ints([1, 1]), s.lensd, s.tabled, s.freed, s.countd, 16, 4)
    with pytest.raises(ValueError):
        plan(cg, s, [1, 1, 1], 4)
    with pytest.raises(ValueError):
        cg.page_plan(ints([1, 1]).cuda(), s.lensd.long(), s.tabled, s.freed, s.countd, 16, 4)
    with pytest.raises(cg.ChainError):
        cg.page_plan(ints([1, 1]).cuda(), s.lensd, s.tabled, s.freed, s.countd, 24, 4)
    with pytest.raises(cg.ChainError):
        plan(cg, s, [1, 1], 4, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        plan(cg, s, [1, 1], 4, out=cg.page_plan(ints([1, 1]).cuda(), s.lensd, s.tabled.clone(), s.freed, s.countd, 16, 5))
    assert cg.chain_check()[0] == 0


def test_steps_captured_in_a_graph(cg):
    # plan and trim of a state kept in place, replayed: as many steps as replays
    s = State([16 * i for i in range(40)], 16, 64, 400, 11).cuda()
    rows = 130
    news, keeps = ints([3] * 40).cuda(), ints([10 ** 6] * 39 + [5]).cuda()
    out = (torch.empty(41, dtype=torch.int32, device="cuda"), s.lensd, s.countd,
           torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int64, device="cuda"))
    ws = torch.empty(max(cg.chain_page_plan_workspace_size(40), cg.chain_page_trim_workspace_size(40)),
                     dtype=torch.uint8, device="cuda")

    def step(stream=None):
        cg.page_plan(news, s.lensd, s.tabled, s.freed, s.countd, 16, rows, out=out, workspace=ws, stream=stream)
        cg.page_trim(keeps, s.lensd, s.tabled, s.freed, s.countd, 16, s.pool, out=(s.lensd, s.countd), workspace=ws,
                     stream=stream)

    def ref():
        got = s.plan([3] * 40, rows)
        s.trim([10 ** 6] * 39 + [5])
        return got

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    ref()
    s.same(s.lensd, s.countd, s.tabled, s.freed)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(5):
        g.replay()
        cu, positions, slots = ref()
        assert out[0].tolist() == cu and out[3].tolist() == positions and out[4].tolist() == slots
        s.same(s.lensd, s.countd, s.tabled, s.freed)
    assert cg.chain_check()[0] == 0


def test_the_slots_are_where_the_cache_is_written(cg):
    # plan, write by the plan's arrays, read back by its slot map
    Hkv, d, page = 2, 64, 32
    s = State([30, 0, 64], page, 8, 12, 13).cuda()
    news, rows = [5, 70, 1], 80
    cu, kv, count, positions, slots = plan(cg, s, news, rows)
    x = torch.randn(rows, Hkv, d, device="cuda").bfloat16()
    kc, vc = (torch.zeros(s.pool, page, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cg.chain_paged_append(x, 2 * x, cu, kv, s.tabled, kc, vc)
    assert cg.chain_check()[0] == 0
    there = slots[:76]
    assert torch.equal(kc.view(-1, Hkv, d)[there], x[:76]) and torch.equal(vc.view(-1, Hkv, d)[there], 2 * x[:76])
    kc.view(-1, Hkv, d)[there] = 0
    assert not bool(kc.any()) and slots[76:].tolist() == [-1] * 4
