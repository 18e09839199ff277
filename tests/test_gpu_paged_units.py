"""GPU: the 128-row kernel of attention over a paged cache where a block's warps pass from one
unit of work to the next: many short units to a block, and units of one and of two query tiles in
turn.  Against the definition in 64 bits, and bit for bit from call to call."""
import pytest
import torch

import chain_synth as cs
from test_gpu_paged import Cache, cg, check  # noqa: F401  (cg: the fixture)

pytestmark = pytest.mark.gpu


def run(cg, lens, news, H, Hkv, d, page, times=20):
    assert sum(news) > len(news)  # not a call of single tokens
    c = Cache(lens, news, Hkv, d, page, 900 + d).fill().cuda()
    q = cs.normal((c.total, H, d), 11)
    ref, rl = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=True)
    assert cg.chain_check()[0] == 0
    check(c, q, ref, rl, True, d ** -0.5)
    for _ in range(times):
        o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=True)
        assert torch.equal(o, ref) and torch.equal(lse, rl)
    assert cg.chain_check()[0] == 0


@pytest.mark.parametrize("d", [64, 128])
def test_many_units_to_a_block(cg, d):
    run(cg, [1 + (37 * i) % 300 for i in range(400)], [1 + i % 2 for i in range(400)], 6, 3, d, 16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_units_of_one_and_two_query_tiles_in_turn(cg, d, page):
    # 32 tokens of four heads fill a query tile: a chunk of 33 to 64 takes two, a token one of the two buffers
    news = [(1, 40, 3, 64, 33, 2, 1, 1, 50)[i % 9] for i in range(90)]
    run(cg, [n + (53 * i) % 200 for i, n in enumerate(news)], news, 8, 2, d, page)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,news", [(256, {5: 200, 6: 1, 90: 1, 91: 9, 255: 1}), (40, {0: 1, 7: 30, 39: 2}),
                                        (64, {i: 1 for i in range(0, 64, 3)}), (300, {150: 299})])
def test_a_batch_padded_with_empty_sequences(cg, d, batch, news):
    # fewer new tokens than sequences: single tokens, chunks and sequences without any, some of them with a
    # cache, rows behind the last sequence, and the same bits from a captured call
    lens = [(13 * b) % 90 if b % 4 == 0 else 0 for b in range(batch)]
    for b, n in news.items():
        lens[b] = n + (71 * b) % 700
    news = [news.get(b, 0) for b in range(batch)]
    assert sum(news) < batch
    H = 8
    c = Cache(lens, news, 2, d, 16, 950 + batch, pad_rows=min(3, batch - sum(news))).fill().cuda()
    q = cs.normal((c.total, H, d), 12).cuda()
    o = torch.full_like(q, 7.0)
    lse = torch.full((H, c.total), 9.0, device="cuda")
    ws = torch.empty(cg.chain_fwd_paged_workspace_size(q, c.kcd), dtype=torch.uint8, device="cuda")
    call = lambda: cg.chain_fwd_paged(q, c.kcd, c.vcd, *c.args, cg.MASK_CAUSAL, d ** -0.5, o, lse, ws)
    call()
    assert cg.chain_check()[0] == 0
    check(c, q.cpu(), o, lse, True, d ** -0.5)
    n = sum(news)
    assert bool((o[n:] == 7).all()) and bool((lse[:, n:] == 9).all())
    ref, rl = o.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        o.zero_()
        lse.zero_()
        g.replay()
        assert torch.equal(o[:n], ref[:n]) and torch.equal(lse[:, :n], rl[:, :n])
    assert cg.chain_check()[0] == 0
