"""GPU: the kernels of the norm + rotation calls each for itself.  Which kernel runs follows from the
bytes of a token's heads, so the head counts here stand on both sides of that choice.  Tolerances
of test_gpu_qk_norm_rope."""
import pytest
import torch

import chain_synth as cs
import test_gpu_qk_norm_rope as base
from test_gpu_paged import Cache
from test_gpu_qk_norm_rope import EPS, cg, freqs  # noqa: F401  (cg: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv", [(2, 1), (20, 4)])
@pytest.mark.parametrize("neighbour", [False, True])
def test_a_frequency_that_is_not_finite_shows(cg, H, Hkv, neighbour):
    T, d = 5, 128
    x = cs.normal((T, H + 2 * Hkv, d), 3).cuda()
    q, k, v = x.split((H, Hkv, Hkv), 1)
    g, w = torch.ones(d, device="cuda"), freqs(d).cuda()
    bad = w.clone()
    bad[3], bad[40], bad[63] = float("nan"), float("inf"), -float("inf")
    at = torch.tensor([3, 40, 63])
    pairs = torch.cat([2 * at, 2 * at + 1] if neighbour else [at, at + d // 2])
    rest = torch.ones(d, dtype=torch.bool)
    rest[pairs] = False

    def check(got, ref):
        assert bool(got[..., pairs].isnan().all()) and torch.equal(got[..., rest], ref[..., rest])

    for got, ref in zip(*(cg.qk_norm_rope(q, k, g, g, f, eps=EPS, interleaved=neighbour) for f in (bad, w))):
        check(got, ref)
    c = Cache([T], [T], Hkv, d, 16, 4).cuda()
    outs = []
    for f in (bad, w):
        pool = torch.zeros_like(c.kcd)
        qo = cg.qk_norm_rope_append(q, k, v, g, g, f, pool, torch.zeros_like(pool), *c.args, interleaved=neighbour)
        outs.append((qo, pool[c.table[0, 0], :T]))
    for got, ref in zip(*outs):
        check(got, ref)
    # a row's gradient runs through its mean, a weight's does not
    dq, dk, *bad_g = cg.qk_norm_rope_bwd(q, k, q, k, g, g, bad, eps=EPS, interleaved=neighbour)
    assert bool(dq.isnan().all()) and bool(dk.isnan().all())
    for got, ref in zip(bad_g, cg.qk_norm_rope_bwd(q, k, q, k, g, g, w, eps=EPS, interleaved=neighbour)[2:]):
        check(got, ref)


# (tokens, H, Hkv, d, rot, neighbour, type)
BY_TOKENS = [(300, 24, 8, 64, 64, False, "bf16"), (77, 33, 2, 64, 32, False, "bf16"), (130, 20, 4, 64, 64, True, "bf16"),
             (5000, 12, 6, 64, 64, False, "bf16"), (300, 12, 4, 64, 64, False, "f32"), (65, 15, 5, 64, 32, True, "f32"),
             (129, 9, 3, 128, 128, True, "f32"), (40, 10, 2, 128, 96, False, "f32"), (4001, 12, 4, 64, 64, True, "f32")]
BY_ROWS = [(50, 2, 1, 64, 64, True, "f32"), (33, 3, 1, 128, 128, True, "f32"), (31, 3, 1, 128, 64, False, "f32"),
           (65, 3, 1, 128, 64, True, "bf16"), (64, 4, 1, 128, 128, False, "bf16"), (70, 7, 3, 64, 16, True, "bf16")]
BOTH = [(60, 5, 2, 128, 64, False, "f32"), (61, 6, 2, 128, 128, True, "bf16")]  # forward by tokens, backward by rows


@pytest.mark.parametrize("case", BY_TOKENS + BY_ROWS + BOTH)
def test_forward_and_backward(cg, case):
    base.test_forward_and_backward(cg, *case)


@pytest.mark.parametrize("neighbour", [False, True])
@pytest.mark.parametrize("H,Hkv,d", [(6, 1, 128), (1, 4, 128), (3, 1, 128), (12, 4, 128), (12, 1, 64), (2, 8, 64),
                                     (4, 1, 64), (20, 4, 64), (33, 3, 64)])
@pytest.mark.parametrize("rot", [1.0, 0.5])
def test_the_fused_write_has_the_bits_of_the_two_calls(cg, H, Hkv, d, neighbour, rot):
    # the two choices of kernel go by different bytes: (6, 1, 128) and (12, 1, 64) norm by tokens alone and
    # by rows in the fused call, (1, 4, 128) and (2, 8, 64) the other way round
    lens, news = [70, 300, 40, 900], [70, 1, 33, 500]
    c = Cache(lens, news, Hkv, d, 16, 21).cuda()
    q, k, v = cs.normal((c.total, H + 2 * Hkv, d), 22).cuda().split((H, Hkv, Hkv), 1)
    gq, gk = ((1 + 0.2 * cs.normal((d,), s, dtype=torch.float32)).cuda() for s in (1, 2))
    w = freqs(int(d * rot)).cuda()
    pos = torch.cat([torch.arange(L - n, L) for L, n in zip(lens, news)]).int().cuda()
    rq, rk = cg.qk_norm_rope(q, k, gq, gk, w, pos, interleaved=neighbour)
    pools = [torch.zeros_like(c.kcd) for _ in range(4)]
    cg.chain_paged_append(rk, v, *c.args, *pools[:2])
    qo = cg.qk_norm_rope_append(q, k, v, gq, gk, w, *pools[2:], *c.args, interleaved=neighbour)
    assert cg.chain_check()[0] == 0
    assert torch.equal(qo, rq) and torch.equal(pools[2], pools[0]) and torch.equal(pools[3], pools[1])
    assert bool(pools[0].any()) and bool(pools[1].any())
