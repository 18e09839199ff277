"""Host-side argument checks of the attention with shared prefixes, on the CPU: dummy addresses that are
never dereferenced.  Run only where no GPU is visible."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_abi_args import D, R, cg, no_device  # noqa: F401  (cg: the fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-side argument checks only; never run with a device present")
PTR = 0x50000000


def prefix(cg, **over):
    a = dict(Q=D(cg, (10, 4, 128)), Kc=D(cg, (20, 16, 2, 128)), Vc=D(cg, (20, 16, 2, 128)), cu=PTR, lens=PTR, table=PTR,
             stride=7, batch=3, max_pages=7, gcu=PTR, glens=PTR, groups=2, mask=1, scale=0.1, O=D(cg, (10, 4, 128)),
             L=D(cg, (4, 10), cg.F32), ws=PTR)
    a["size"] = cg.lib().chain_fwd_paged_prefix_workspace_size(R(a["Q"]), R(a["Kc"]))
    assert a["size"] > cg.lib().chain_fwd_paged_workspace_size(R(a["Q"]), R(a["Kc"]))
    a.update(over)
    return cg.lib().chain_fwd_paged_prefix(R(a["Q"]), R(a["Kc"]), R(a["Vc"]), a["cu"], a["lens"], a["table"], a["stride"],
                                           a["batch"], a["max_pages"], a["gcu"], a["glens"], a["groups"], a["mask"],
                                           ctypes.c_float(a["scale"]), R(a["O"]), R(a["L"]), a["ws"], a["size"], None)


def test_prefix(cg):
    for ok in (dict(), dict(groups=0, gcu=None, glens=None), dict(groups=8192), dict(mask=0), dict(batch=1, stride=0),
               dict(gcu=PTR + 4)):
        assert prefix(cg, **ok) in no_device(cg), ok
    for name in ("Q", "Kc", "Vc", "cu", "lens", "table", "gcu", "glens", "O", "L", "ws"):
        assert prefix(cg, **{name: None}) == cg.ERR_ARG, name
    for bad in (dict(groups=-1), dict(gcu=PTR + 2), dict(glens=PTR + 1), dict(mask=2), dict(scale=0.0),
                dict(batch=-1), dict(stride=6), dict(max_pages=0), dict(size=64), dict(ws=PTR + 8),
                dict(size=cg.lib().chain_fwd_paged_workspace_size(R(D(cg, (10, 4, 128))), R(D(cg, (20, 16, 2, 128))))),
                dict(O=D(cg, (10, 5, 128))), dict(L=D(cg, (4, 11), cg.F32)), dict(Vc=D(cg, (21, 16, 2, 128)))):
        assert prefix(cg, **bad) == cg.ERR_ARG, bad
    for bad in (dict(groups=8193), dict(batch=8193)):
        assert prefix(cg, **bad) == cg.ERR_UNSUPPORTED, bad
    assert prefix(cg, L=D(cg, (4, 10))) == cg.ERR_DTYPE
    assert prefix(cg, Q=D(cg, (10, 4, 128), cg.F32)) == cg.ERR_DTYPE
    # nothing to do: done without a device
    e, l = D(cg, (0, 4, 128), ptr=0), D(cg, (4, 0), cg.F32, ptr=0)
    assert prefix(cg, Q=e, O=e, L=l) == cg.OK
    assert prefix(cg, batch=0) == cg.OK


def test_workspace_size(cg):
    size = cg.lib().chain_fwd_paged_prefix_workspace_size
    q, pool = D(cg, (10, 4, 128)), D(cg, (20, 16, 2, 128))
    assert size(R(D(cg, (1000, 4, 128))), R(pool)) > size(R(q), R(pool)) > 0
    for a, b in ((None, pool), (q, None), (D(cg, (10, 4, 64)), pool), (D(cg, (10, 3, 128)), pool),
                 (q, D(cg, (20, 24, 2, 128))), (D(cg, (10, 4, 128), cg.F32), pool)):
        assert size(R(a), R(b)) == 0


def test_the_native_modules_own_checks(cg):
    def call(**over):
        q, pool = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16)
        i = lambda *s: torch.zeros(*s, dtype=torch.int32)
        a = dict(q=q, kc=pool, vc=pool, cu=i(3), lens=i(2), table=i(2, 4), gcu=i(2), glens=i(1), mask=1, scale=0.1,
                 o=torch.empty_like(q), lse=torch.zeros(4, 3), ws=torch.empty(1 << 27, dtype=torch.uint8))
        a.update(over)
        cg._small().fwd_paged_prefix(*a.values(), cg._bytes(a["ws"]), -1, 0)

    with pytest.raises(cg.ChainError):  # no device: every check before it passed
        call()
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for bad in (dict(gcu=i(1)), dict(gcu=i(3)), dict(glens=i(2)), dict(gcu=i(2).long()), dict(glens=i(1, 1)),
                dict(gcu=i(4)[::2]), dict(cu=i(2)), dict(ws=torch.empty(1, dtype=torch.uint8).expand(1 << 27))):
        with pytest.raises(ValueError):
            call(**bad)
