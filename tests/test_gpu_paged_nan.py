"""GPU: a query that is not a number.  Its row of O and of the LSE is NaN, as the definition's; every other row
has the bits that it has without it."""
import math

import pytest
import torch

import chain_synth as cs
from test_gpu_paged import Cache, cg  # noqa: F401  (cg: the fixture)
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu

# lens, news, H, Hkv, d, page.  A unit of work is whole (short caches) or cut and joined (long ones).
CASES = {
    "single tokens": ([20, 300, 7], [1, 1, 1], 8, 2, 128, 16),
    "single tokens, long": ([9000, 4001], [1, 1], 8, 2, 128, 64),
    "single tokens, long, d 64": ([9000, 4001], [1, 1], 8, 2, 64, 64),
    "chunks": ([90, 300, 130], [90, 20, 5], 8, 2, 128, 16),
    "chunks, long": ([9000, 4001], [70, 33], 8, 2, 128, 64),
    "chunks, long, d 64": ([9000, 4001], [70, 33], 6, 6, 64, 64),
    "33 heads on one": ([5000, 64], [1, 1], 33, 1, 64, 64),
}


def ascending(c):
    """Keys whose product with an infinity at element 7 is one."""
    for x in c.k:
        x[..., 7] = x[..., 7].abs() + 1
    return c


def spoiled(q, news, value):
    """A row of each sequence, and which rows these are."""
    bad, at, lo = q.clone(), torch.zeros(q.shape[:2], dtype=torch.bool), 0
    for b, n in enumerate(news):
        t, h = lo + (5 * b + 2) % n, (3 * b + 1) % q.shape[1]
        bad[t, h, 7] = value
        at[t, h] = True
        lo += n
    return bad, at


def same_but(at, got, clean):
    (o, lse), (ro, rl) = got, clean
    assert bool(o.cpu()[at].isnan().all()), "O of the row"
    assert bool(lse.cpu().t()[at].isnan().all()), "LSE of the row"
    assert torch.equal(o.cpu()[~at], ro.cpu()[~at]) and torch.equal(lse.cpu().t()[~at], rl.cpu().t()[~at])


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_paged(cg, name, causal, value):
    lens, news, H, Hkv, d, page = CASES[name]
    c = ascending(Cache(lens, news, Hkv, d, page, 80)).fill().cuda()
    q = cs.normal((c.total, H, d), 81)
    bad, at = spoiled(q, news, value)
    run = lambda x: cg.attention_fwd_paged(x.cuda(), c.kcd, c.vcd, *c.args, causal=causal)
    same_but(at, run(bad), run(q))
    assert cg.chain_check()[0] == 0


PREFIXES = {
    "single tokens": ([(5, 512)], [512 + 9 * i + 1 for i in range(5)], [1] * 5, 8, 2, 128, 16),
    "single tokens, long": ([(4, 9984)], [9984 + 64 * i + 1 for i in range(4)], [1] * 4, 8, 2, 128, 64),
    "single tokens, long, d 64": ([(2, 9984), (3, 4096)], [9985, 9990, 4100, 4097, 7000], [1] * 5, 15, 5, 64, 16),
    "many rows": ([(40, 9984)], [9984 + 3 * i + 1 for i in range(40)], [1] * 40, 8, 2, 128, 64),
    "chunks, long": ([(3, 4096)], [4096 + 200, 4096 + 65, 4096 + 9], [150, 64, 9], 8, 2, 128, 64),
    "chunks, d 64": ([(3, 4096)], [4096 + 200, 4096 + 65, 4096 + 9], [150, 64, 9], 6, 6, 64, 64),
}


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("name", PREFIXES)
def test_prefix(cg, name, wide, value):
    groups, lens, news, H, Hkv, d, page = PREFIXES[name]
    c = ascending(Shared(groups, lens, news, Hkv, d, page, 82)).fill().cuda(wide)
    q = cs.normal((c.total, H, d), 83)
    bad, at = spoiled(q, news, value)
    run = lambda x: cg.attention_fwd_paged_prefix(x.cuda(), c.kcd, c.vcd, *c.args, causal=True)
    same_but(at, run(bad), run(q))
    assert cg.chain_check()[0] == 0


def test_rows_that_see_nothing_stay_zero(cg):
    # more new tokens than cached ones
    c = Cache([5, 130], [9, 200], 2, 128, 16, 84).fill().cuda()
    q = cs.normal((c.total, 4, 128), 85)
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=True)
    assert cg.chain_check()[0] == 0
    for lo, n in ((0, 4), (9, 70)):
        assert not bool(o[lo:lo + n].any()) and bool((lse[:, lo:lo + n] == -math.inf).all())
