"""GPU: page plan (chain_page_plan) on both sides of what one block takes, 1,024 sequences and 4,096 rows, against a plain
loop over sequences and pages.  Whole numbers: every result is compared for equality."""
import pytest

from test_gpu_page_plan import State, cg, plan  # noqa: F401  (cg: the fixture)

pytestmark = pytest.mark.gpu

# sequences, new tokens of sequence i, rows behind the last
SIZES = {
    "all that one block takes": (1024, lambda i: 4, 0),
    "all of its sequences, some without tokens": (1024, lambda i: (0, 1, 7)[i % 3], 900),
    "one row more": (1024, lambda i: 4, 1),
    "one row more, a token": (1024, lambda i: 4 + (i == 700), 0),
    "one sequence more": (1025, lambda i: 1 + i % 3, 4),
    "one sequence more, without tokens": (1025, lambda i: 3 * (i < 1024), 0),
    "one sequence, all of its rows": (1, lambda i: 4096, 0),
    "one sequence, one row more": (1, lambda i: 4097, 0),
    "the last sequence alone": (1024, lambda i: 900 * (i == 1023), 5),
    "no rows": (1024, lambda i: 0, 0),
}


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("name", SIZES)
def test_plan(cg, name, page):
    count, new, pad = SIZES[name]
    lens, news = [(7 * i) % 90 for i in range(count)], [new(i) for i in range(count)]
    need = sum(-(-(L + n) // page) - -(-L // page) for L, n in zip(lens, news))
    s = State(lens, page, max(-(-(L + n) // page) for L, n in zip(lens, news)) + 1, need + 2, len(name)).cuda(wide=1)
    rows = sum(news) + pad
    cu, kv, left, positions, slots = plan(cg, s, news, rows)
    assert cg.chain_check()[0] == 0
    rc, rp, rs = s.plan(news, rows)
    assert cu.tolist() == rc and positions.tolist() == rp and slots.tolist() == rs
    s.same(kv, left, s.tabled, s.freed)


@pytest.mark.parametrize("pad", [0, 5000])
def test_a_full_table_and_a_stack_that_runs_out(cg, pad):
    # a full table takes what it can from the stack, whose count is what is left; a stack that runs out is left with none
    s = State([20, 40, 5], 16, 6, 9, 4).cuda()
    count = plan(cg, s, [90, 0, 1], 91 + pad)[2]
    assert cg.chain_check()[0] == cg.ERR_ARG
    s.plan([90, 0, 1], 91 + pad)
    assert count.tolist() == [s.count] == [5]
    s = State([20, 40, 5], 16, 6, 2, 4).cuda()
    count = plan(cg, s, [50, 0, 1], 51 + pad)[2]
    assert cg.chain_check()[0] == cg.ERR_ARG and count.tolist() == [0]
