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
