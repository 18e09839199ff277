"""GPU: attention over a paged cache within the bounds that every forward of the
library holds (tol.py): max and mean error of O against the definition in 64 bits,
and the LSE.  The rounding of O alone takes 1.41e-3 of the mean bound of 2e-3 on
normally distributed values, and a P of one bf16 takes it to 2.1e-3 to 2.3e-3."""
import pytest
import torch

import chain_synth as cs
from test_gpu_paged import Cache, cg, reference  # noqa: F401  (cg: the fixture)
from tol import assert_fwd_close, assert_lse_close

pytestmark = pytest.mark.gpu

# lens, news, H, Hkv, d, page
TOKENS = {
    "one token over 100": ([100], [1], 32, 8, 128, 16),
    "one token over 8192": ([8192], [1], 32, 8, 128, 64),
    "one token over 8192, d 64": ([8192], [1], 32, 8, 64, 64),
    "eight sequences": ([100, 2000, 333, 1024, 4000, 65, 700, 1500], [1] * 8, 32, 8, 128, 64),
    "many sequences, d 64": ([(53 * i) % 900 + 40 for i in range(40)], [1] * 40, 15, 5, 64, 16),
    "sixteen heads to a key head": ([900, 3000], [1, 1], 32, 2, 128, 128),
    "whole sequences to a block": ([1500 - 7 * i for i in range(64)], [1] * 64, 32, 8, 128, 64),
    "whole sequences to a block, d 64": ([1500 - 7 * i for i in range(64)], [1] * 64, 24, 8, 64, 64),
    "four tokens of one sequence": ([1700], [4], 16, 4, 64, 32),
}


def run(cg, case, causal=True):
    lens, news, H, Hkv, d, page = case
    c = Cache(lens, news, Hkv, d, page, 4000 + len(lens)).fill().cuda()
    q = cs.normal((c.total, H, d), 7)
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=causal)
    assert cg.chain_check()[0] == 0
    ref = [reference(c, q, b, causal, d ** -0.5) for b in range(len(lens)) if news[b]]
    assert_fwd_close(o, torch.cat([r[0] for r in ref]))
    assert_lse_close(lse, torch.cat([r[2] for r in ref], 1))


@pytest.mark.parametrize("name", TOKENS)
def test_single_tokens(cg, name):
    run(cg, TOKENS[name])


CHUNKS = {
    "a chunk over 2000": ([2000], [200], 16, 4, 128, 128),
    "a chunk over 2000, d 64": ([2000], [200], 16, 4, 64, 64),
    "mixed, odd group": ([700, 33, 1500, 70, 900], [60, 1, 1, 70, 300], 14, 2, 128, 16),
    "mixed, odd group, d 64": ([700, 33, 1500, 70, 900], [60, 1, 1, 70, 300], 15, 5, 64, 16),
    "whole sequences to a block": ([700 - 3 * i for i in range(64)], [3] * 64, 16, 8, 128, 64),
    "whole sequences to a block, d 64": ([700 - 3 * i for i in range(64)], [3] * 64, 16, 8, 64, 64),
    "no grouped heads, d 64": ([900, 600], [130, 257], 4, 4, 64, 32),
    "more query heads than a small tile takes": ([3000, 900], [1, 1], 64, 2, 128, 128),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", CHUNKS)
def test_chunks(cg, name, causal):
    run(cg, CHUNKS[name], causal)
