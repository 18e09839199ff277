"""GPU: page trim (chain_page_trim) in each of its three forms -- one block, a cluster of blocks, two launches, which the
table's entries choose (up to 8,192, up to 131,072, more) -- against a plain loop over sequences and pages.  Whole
numbers: every result is compared for equality."""
import pytest
import torch

from test_gpu_page_plan import State, cg, ints  # noqa: F401  (cg: the fixture)

pytestmark = pytest.mark.gpu


def trim(cg, s, keeps, out=None, **kw):
    return cg.page_trim(ints(keeps).cuda(), s.lensd, s.tabled, s.freed, s.countd, s.page, s.pool, out=out, **kw)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch", [1, 2, 5, 7, 8, 9, 31, 32, 33, 65])
def test_few_sequences_of_a_cluster(cg, batch, in_place):
    # lanes of a warp without a sequence beside lanes that read one
    max_pages = 60000 // batch
    lens = [(16 * max_pages * (i + 1)) // batch - 5 * i for i in range(batch)]
    assert 1 << 13 < batch * max_pages <= 1 << 17 and min(lens) > 0 and max(lens) <= 16 * max_pages
    keeps = [0 if i % 3 == 0 else L - 40 * (i % 5) for i, L in enumerate(lens)]
    s = State(lens, 16, max_pages, 3, batch).cuda()
    before = s.tabled.clone()
    kv, count = trim(cg, s, keeps, (s.lensd, s.countd) if in_place else None)
    assert cg.chain_check()[0] == 0
    s.trim(keeps)
    s.same(kv, count, s.tabled, s.freed)
    assert bool((s.tabled == before).all())


# More than 65,536 entries that go back through one cluster: a warp's piece is more than it holds at a time, so it counts in
# rounds and loads again to put.  lens, keeps, max_pages
LONG_PIECES = {
    "one sequence": ([16 * 130000 - 3], [20], 131072),
    "one sequence, just more than is held": ([16 * 65600], [0], 70000),
    "one sequence, just as much as is held": ([16 * 65536], [0], 70000),
    "two long ones": ([16 * 60000, 16 * 65000 + 1], [16 * 100 + 5, 0], 65536),
    "a thousand": ([16 * (110 + i % 18) for i in range(1000)], [16 * (i % 7) for i in range(1000)], 128),
    "a thousand, many without": ([16 * 128 * (i % 3 > 0) for i in range(1024)], [5 * (i % 2) for i in range(1024)], 128),
    "long ones among short ones": ([17, 0, 1] + [16 * 14500 - 7] * 6, [16 * (i % 2) for i in range(9)], 14500),
    "long ones": ([16 * 10900 - 7 - i for i in range(12)], [700 * i for i in range(12)], 10900),
}


@pytest.mark.parametrize("missing", [0, 7, 1])
@pytest.mark.parametrize("name", LONG_PIECES)
def test_long_pieces_of_a_cluster(cg, name, missing):
    lens, keeps, max_pages = LONG_PIECES[name]
    assert 1 << 13 < len(lens) * max_pages <= 1 << 17 and len(lens) <= 1024
    s = State(lens, 16, max_pages, 3, len(name))
    back = lost = 0
    for b, (L, keep) in enumerate(zip(lens, keeps)):
        for e in range(-(-min(L, keep) // 16), -(-L // 16)):
            back += 1
            if missing and back % missing == 0:
                s.table[b][e] = -1 if back % 2 else s.pool
                lost += 1
    assert back >= 65536
    s.cuda(wide=len(name) % 3)
    kv, count = trim(cg, s, keeps, (s.lensd, s.countd))
    assert cg.chain_check()[0] == (cg.ERR_ARG if lost else 0)
    s.trim(keeps)
    s.same(kv, count, s.tabled, s.freed)


FORMS = {"one block": 8, "a cluster": 5000, "two launches": 50000}  # of three sequences, by the table's columns


@pytest.mark.parametrize("form", FORMS)
def test_what_each_form_reports(cg, form):
    max_pages = FORMS[form]
    # a stack that overflows: what does not fit is lost, and nothing is written behind it
    for fits in (0, 1, 4, 14):
        s = State([100, 70, 20], 16, max_pages, 2, 9, extra=0)
        s.free = s.free[:2 + fits]
        s.cuda()
        guard = torch.full((40,), 123, dtype=torch.int32, device="cuda")
        guard[:2 + fits] = s.freed
        s.freed = guard[:2 + fits]
        kv, count = trim(cg, s, [0, 0, 0])
        assert cg.chain_check()[0] == (0 if fits == 14 else cg.ERR_ARG)
        s.trim([0, 0, 0])
        s.same(kv, count, s.tabled, s.freed)
        assert bool((guard[2 + fits:] == 123).all())
    # entries that name no page
    for bad in (-1, 2 ** 31 - 1, -2 ** 31):
        s = State([100, 70, 20], 16, max_pages, 2, 8)
        s.table[0][3], s.table[1][4] = bad, s.pool
        s.cuda()
        kv, count = trim(cg, s, [10, 0, 20])
        assert cg.chain_check()[0] == cg.ERR_ARG and cg.chain_check()[0] == 0
        s.trim([10, 0, 20])
        s.same(kv, count, s.tabled, s.freed)
    # a length past the table's end counts as that, one below zero as none
    s = State([100, 16 * max_pages, 70], 16, max_pages, 2, 10).cuda(wide=3)
    s.lensd[1], s.lensd[2], s.lens[2] = 16 * max_pages + 1, -1, 0
    kv, count = trim(cg, s, [100, 16, 5])
    assert cg.chain_check()[0] == cg.ERR_ARG
    s.trim([100, 16, 5])
    s.same(kv, count, None, s.freed)
    # a stack's count out of range
    for wrong in (-3, -2 ** 31, 10 ** 6, 2 ** 31 - 1):
        s = State([100, 70, 20], 16, max_pages, 2, 11).cuda()
        s.countd.fill_(wrong)
        s.count = 0 if wrong < 0 else len(s.free)
        kv, count = trim(cg, s, [50, 0, 30])
        assert cg.chain_check()[0] == cg.ERR_ARG
        s.trim([50, 0, 30])
        s.same(kv, count, s.tabled, s.freed)


@pytest.mark.parametrize("form", FORMS)
def test_each_form_captured_and_replayed(cg, form):
    # one step after another on a state kept in place: each replay cuts and plans again
    max_pages, rows = FORMS[form], 5000  # more rows than one block plans
    s = State([100, 70, 20], 16, max_pages, 90, 12).cuda()
    news, keeps = [20, 40, 30], [30, 10 ** 9, 0]
    newsd, keepsd = ints(news).cuda(), ints(keeps).cuda()
    out = (torch.empty(4, dtype=torch.int32, device="cuda"), s.lensd, s.countd,
           torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int64, device="cuda"))
    ws = torch.full((max(cg.chain_page_plan_workspace_size(3), cg.chain_page_trim_workspace_size(3)),), 255,
                    dtype=torch.uint8, device="cuda")

    def step():
        cg.page_trim(keepsd, s.lensd, s.tabled, s.freed, s.countd, 16, s.pool, out=(s.lensd, s.countd), workspace=ws)
        cg.page_plan(newsd, s.lensd, s.tabled, s.freed, s.countd, 16, rows, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        if i:
            g.replay()
        fits = s.lens[1] + 40 <= 16 * max_pages
        s.trim(keeps)
        cu, positions, slots = s.plan(news, rows)
        assert cg.chain_check()[0] == (0 if fits else cg.ERR_ARG)
        assert out[0].tolist() == cu and out[3].tolist() == positions and out[4].tolist() == slots
        s.same(s.lensd, s.countd, s.tabled)
        if not fits:
            break


@pytest.mark.parametrize("form", FORMS)
def test_two_states_on_two_streams(cg, form):
    states = [State([300 + i, 70, 16 * 20 - i], 16, max(FORMS[form], 24), 60, 13 + i).cuda() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for keep in (250, 130, 17, 1):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                trim(cg, s, [keep] * 3, (s.lensd, s.countd))
            s.trim([keep] * 3)
    torch.cuda.synchronize()
    assert cg.chain_check()[0] == 0
    for s in states:
        s.same(s.lensd, s.countd, s.tabled, s.freed)
