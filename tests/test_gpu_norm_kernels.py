"""GPU: the kernels of the norm + rotation calls each for itself.  Which kernel runs follows from the
bytes of a token's heads, so the head counts here stand on both sides of that choice.  Tolerances
of test_gpu_qk_norm_rope."""
import pytest
import torch

import chain_synth as cs
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
