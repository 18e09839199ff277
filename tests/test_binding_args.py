"""The native module's own checks, on the CPU: a call that passes them gets as far as the
device query.  Run only where no GPU is visible: host tensors stand in for device tensors."""
import pytest

torch = pytest.importorskip("torch")

import chain_gb300 as cg

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-side argument checks only; never run with a device present")


def attention(workspace, n_bytes=None):
    q, pool = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16)
    cu, lens, table = (torch.zeros(s, dtype=torch.int32) for s in ((2,), (1,), (1, 4)))
    n = cg._bytes(workspace) if n_bytes is None else n_bytes
    cg._small().fwd_paged(q, pool, pool, cu, lens, table, 1, 0.1, torch.empty_like(q), torch.zeros(4, 3), workspace, n,
                          -1, 0)


def backward(workspace):
    q, k, g = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), torch.zeros(64)
    cg._small().qk_norm_rope_bwd(q, k, q, k, g, g, None, None, 1e-6, 0, torch.empty_like(q), torch.empty_like(k),
                                 torch.empty_like(g), torch.empty_like(g), workspace, cg._bytes(workspace), -1, 0)


@pytest.mark.parametrize("call", [attention, backward])
def test_a_workspace_is_memory_of_its_own(call):
    # a view's elements times their size say nothing about the bytes behind its address
    need = 1 << 26
    with pytest.raises(cg.ChainError):  # no device: every check before it passed
        call(torch.empty(need, dtype=torch.uint8))
    for bad in (torch.empty(1, dtype=torch.uint8).expand(need), torch.empty(4, need // 2, dtype=torch.uint8)[:, ::2]):
        with pytest.raises(ValueError):
            call(bad)
