"""GPU: page trim (chain_page_trim) in each of its three forms -- one block, a cluster of blocks, two launches, which the
table's entries choose (up to 8,192, up to 131,072, more) -- against a plain loop over sequences and pages.  Whole
numbers: every result is compared for equality."""
import pytest

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
