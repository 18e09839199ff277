"""GPU: attention over a paged cache behind shared prefixes, where nothing is left behind the prefix and where a page
ends behind it.  Tolerances: those of test_gpu_prefix, by the same check."""
import pytest
import torch

import chain_synth as cs
from test_gpu_paged import cg, check  # noqa: F401  (cg: the fixture)
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu

# heads, K/V heads, new tokens: the 128-row kernel for chunks, and for groups of heads that do not fit 16 rows; the 16-row one
FORMS = {"a chunk": (8, 2, [9, 1, 1]), "33 heads on one": (66, 2, [1, 1, 1]), "full tiles": (4, 4, [200, 130, 3]),
         "single tokens": (8, 2, [1, 1, 1])}


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("lens", [[384, 384, 384], [384, 384, 500], [384, 400, 384]])
@pytest.mark.parametrize("page", [64, 128, 256, 1024])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_a_prefix_that_is_all_and_ends_inside_a_page(cg, form, d, page, lens, wide):
    # without a mask; the slots behind the 384 positions are NaN where no sequence has written
    H, Hkv, news = FORMS[form]
    if page < 256 and lens != [384] * 3:  # their 384 positions end with a page
        lens = [384, 384 + page + 3, 384]
    c = Shared([(3, 384)], lens, news, Hkv, d, page, 71).fill().cuda(wide)
    q = cs.normal((c.total, H, d), 72)
    o, lse = cg.attention_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args, causal=False)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, False, d ** -0.5)


@pytest.mark.parametrize("P", [128, 256, 640, 896])
def test_several_groups_whose_prefix_is_all(cg, P):
    c = Shared([(2, P), (3, 384)], [P, P, 384, 384, 384], [5, 1, 40, 1, 0], 2, 128, 1024, 73).fill().cuda()
    q = cs.normal((c.total, 8, 128), 74)
    o, lse = cg.attention_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args, causal=False)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, False, 128 ** -0.5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("news", [[1, 1, 1], [20, 1, 33]])
def test_without_groups_it_is_the_plain_call(cg, news, causal):
    c = Shared([], [300, 5000, 64], news, 2, 128, 64, 75).fill().cuda()
    q = cs.normal((c.total, 8, 128), 76).cuda()
    ref = cg.attention_fwd_paged(q, c.kcd, c.vcd, *c.args[:3], causal=causal)
    ws = torch.empty(cg.chain_fwd_paged_workspace_size(q, c.kcd), dtype=torch.uint8, device="cuda")
    for given in (ws, None):
        got = cg.attention_fwd_paged_prefix(q, c.kcd, c.vcd, *c.args, causal=causal, workspace=given)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert cg.chain_check()[0] == 0
