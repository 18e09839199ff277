"""GPU: the page plan, the page trim and the attention behind shared prefixes write nothing outside their outputs and the
workspace that they ask for: each is a view into a larger buffer whose guards hold a pattern."""
import pytest
import torch

import chain_synth as cs
from test_gpu_page_plan import State, cg, ints  # noqa: F401  (cg: the fixture)
from test_gpu_paged import check
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu
GUARD = 1 << 16  # bytes on each side


class Guarded:
    def __init__(self):
        self.all = []

    def bytes(self, n):
        whole = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((whole, n))
        return whole[GUARD:GUARD + n]

    def tensor(self, dtype, *shape):
        n = torch.empty(shape, dtype=dtype, device="meta").nbytes
        return self.bytes(n).view(dtype).view(*shape)

    def intact(self):
        torch.cuda.synchronize()
        return all(bool((w[:GUARD] == 0xA5).all()) and bool((w[GUARD + n:] == 0xA5).all()) for w, n in self.all)


# groups, lens, news, H, Hkv, d, page
PREFIXES = {
    "single tokens": ([(20, 1024)], [1024 + 17 * i + 1 for i in range(20)], [1] * 20, 8, 2, 128, 16),
    "single tokens, d 64": ([(20, 1024)], [1024 + 17 * i + 1 for i in range(20)], [1] * 20, 15, 5, 64, 16),
    "long, few rows": ([(2, 9088)], [9089, 9300], [1, 1], 8, 1, 128, 64),
    "long, many rows": ([(40, 4096)], [4097 + i for i in range(40)], [1] * 40, 8, 2, 128, 64),
    "chunks": ([(3, 4096), (2, 640)], [4300, 4161, 4105, 700, 641], [150, 64, 9, 33, 1], 8, 2, 128, 64),
    "chunks, d 64": ([(3, 4096), (2, 640)], [4300, 4161, 4105, 700, 641], [150, 64, 9, 33, 1], 6, 6, 64, 64),
    "one token": ([(1, 128)], [129], [1], 1, 1, 64, 16),
}


@pytest.mark.parametrize("groups", [True, False])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("name", PREFIXES)
def test_prefix(cg, name, wide, groups):
    shared, lens, news, H, Hkv, d, page = PREFIXES[name]
    c = Shared(shared, lens, news, Hkv, d, page, 91).fill().cuda(wide)
    q = cs.normal((c.total, H, d), 92)
    g = Guarded()
    o, lse = g.tensor(torch.bfloat16, c.total, H, d), g.tensor(torch.float32, H, c.total)
    size = cg.chain_fwd_paged_prefix_workspace_size if groups else cg.chain_fwd_paged_workspace_size
    ws = g.bytes(size(q.cuda(), c.kcd))
    pre = (c.gcu, c.glens) if groups else (c.gcu[:1], c.glens[:0])
    cg.chain_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args[:3], *pre, cg.MASK_CAUSAL, d ** -0.5, o, lse, ws)
    assert cg.chain_check()[0] == 0 and g.intact()
    check(c, q, o, lse, True, d ** -0.5)


@pytest.mark.parametrize("count,max_pages,rows", [(1, 8, 5), (3, 5000, 5000), (3, 50000, 40), (1024, 8, 3000),
                                                  (1025, 8, 3000), (8192, 8, 9000)])
def test_plan_and_trim(cg, count, max_pages, rows):
    lens, news = [(11 * i) % 90 for i in range(count)], [i % 2 for i in range(count)]
    s = State(lens, 16, max_pages, count + 5, 93)
    g = Guarded()
    table, free = g.tensor(torch.int32, count, max_pages), g.tensor(torch.int32, len(s.free))
    table.copy_(ints(s.table)), free.copy_(ints(s.free))
    s.tabled, s.freed, s.countd, s.lensd = table, free, g.tensor(torch.int32, 1), g.tensor(torch.int32, count)
    s.countd.fill_(s.count), s.lensd.copy_(ints(s.lens))
    out = (g.tensor(torch.int32, count + 1), s.lensd, s.countd, g.tensor(torch.int32, rows), g.tensor(torch.int64, rows))
    cg.page_plan(ints(news).cuda(), s.lensd, table, free, s.countd, 16, rows, out=out,
                 workspace=g.bytes(cg.chain_page_plan_workspace_size(count)))
    assert cg.chain_check()[0] == 0 and g.intact()
    cu, positions, slots = s.plan(news, rows)
    assert out[0].tolist() == cu and out[3].tolist() == positions and out[4].tolist() == slots
    s.same(s.lensd, s.countd, table, free)
    keeps = [L // 2 for L in s.lens]
    cg.page_trim(ints(keeps).cuda(), s.lensd, table, free, s.countd, 16, s.pool, out=(s.lensd, s.countd),
                 workspace=g.bytes(cg.chain_page_trim_workspace_size(count)))
    assert cg.chain_check()[0] == 0 and g.intact()
    s.trim(keeps)
    s.same(s.lensd, s.countd, table, free)
