"""The workspace that the attention with shared prefixes asks for without groups, when it is chain_fwd_paged: on the
CPU, with dummy addresses that are never dereferenced.  Run only where no GPU is visible."""
import pytest

torch = pytest.importorskip("torch")

from test_abi_args import D, R, cg, no_device  # noqa: F401  (cg: the fixture)
from test_prefix_args import prefix

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-side argument checks only; never run with a device present")


@pytest.mark.parametrize("total,d", [(10, 128), (10, 64), (32768, 128)])
def test_without_groups(cg, total, d):
    q, pool = D(cg, (total, 4, d)), D(cg, (20, 16, 2, d))
    tensors = dict(Q=q, Kc=pool, Vc=pool, O=D(cg, (total, 4, d)), L=D(cg, (4, total), cg.F32))
    size = cg.lib().chain_fwd_paged_workspace_size(R(q), R(pool))
    assert 0 < size < cg.lib().chain_fwd_paged_prefix_workspace_size(R(q), R(pool))
    none = dict(groups=0, gcu=None, glens=None)
    assert prefix(cg, **tensors, **none, size=size) in no_device(cg)
    assert prefix(cg, **tensors, **none, size=size - 1) == cg.ERR_ARG
    assert prefix(cg, **tensors, size=size) == cg.ERR_ARG
