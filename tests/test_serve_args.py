"""Host-side argument checks of the norm + rotation and paged-cache entry
points, on the CPU: descriptors hold dummy addresses that are never
dereferenced, a bad argument returns its status, and a valid call gets past
every check and fails only at the device query.  Run only where no GPU is
visible."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from test_abi_args import D, R, cg, no_device  # noqa: F401  (cg: the fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-side argument checks only; never run with a device present")
PTR = 0x50000000


def rope(cg, **over):
    T, H, Hkv, d, dt = over.get("T", 10), 4, 2, over.get("d", 128), over.get("dt", cg.BF16)
    a = dict(Q=D(cg, (T, H, d), dt), K=D(cg, (T, Hkv, d), dt), gq=D(cg, (d,), cg.F32), gk=D(cg, (d,)),
             w=D(cg, (d // 2,), cg.F32), pos=PTR, eps=1e-6, pairs=0, Qo=D(cg, (T, H, d), dt),
             Ko=D(cg, (T, Hkv, d), dt))
    a.update({k: v for k, v in over.items() if k in a})
    return cg.lib().chain_qk_norm_rope(R(a["Q"]), R(a["K"]), R(a["gq"]), R(a["gk"]), R(a["w"]), a["pos"], a["eps"],
                                       a["pairs"], R(a["Qo"]), R(a["Ko"]), None)


def test_qk_norm_rope(cg):
    B, F = cg.BF16, cg.F32
    for ok in (dict(), dict(d=64), dict(dt=F), dict(w=None), dict(pos=None), dict(pairs=1),
               dict(w=D(cg, (24,), F)), dict(Q=D(cg, (10, 4, 128), strides=(1024, 128, 1))),
               dict(Q=D(cg, (10, 4, 128), strides=(128, 1280, 1)))):
        assert rope(cg, **ok) in no_device(cg), ok
    for name in ("Q", "K", "gq", "gk", "Qo", "Ko"):
        assert rope(cg, **{name: None}) == cg.ERR_ARG
    for bad in (0.0, -1.0, math.nan, math.inf):
        assert rope(cg, eps=bad) == cg.ERR_ARG
    for bad in (dict(pairs=2), dict(pairs=-1), dict(pos=PTR + 2), dict(d=96), dict(w=D(cg, (72,), F)),
                dict(w=D(cg, (12,), F)), dict(w=D(cg, (0,), F)), dict(w=D(cg, (32,), F, strides=(2,))),
                dict(gq=D(cg, (64,), F)), dict(gq=D(cg, (128,), F, ptr=PTR + 4)), dict(gk=D(cg, (1, 128), F)),
                dict(Qo=D(cg, (10, 5, 128))), dict(Ko=D(cg, (9, 2, 128))), dict(K=D(cg, (10, 2, 64))),
                dict(Q=D(cg, (10, 4, 128), ptr=PTR + 8)), dict(Q=D(cg, (10, 4, 128), strides=(516, 128, 1))),
                dict(Q=D(cg, (10, 4, 128), strides=(0, 128, 1))), dict(Q=D(cg, (10, 4, 128), strides=(1024, 256, 2))),
                dict(Q=D(cg, (1, 10, 4, 128))), dict(Q=D(cg, (40, 128)))):
        assert rope(cg, **bad) == cg.ERR_ARG, bad
    for bad in (dict(w=D(cg, (64,), B)), dict(Q=D(cg, (10, 4, 128), F)), dict(Ko=D(cg, (10, 2, 128), F)),
                dict(gq=D(cg, (128,), cg.E4M3)), dict(dt=cg.E4M3)):
        assert rope(cg, **bad) == cg.ERR_DTYPE, bad
    # [B][n][heads][d], with any strides; a batch of another size
    q4, k4 = D(cg, (3, 5, 4, 128), strides=(4096, 128, 640, 1)), D(cg, (3, 5, 2, 128))
    assert rope(cg, Q=q4, K=k4, Qo=q4, Ko=k4) in no_device(cg)
    assert rope(cg, Q=q4, K=D(cg, (5, 3, 2, 128)), Qo=q4, Ko=k4) == cg.ERR_ARG
    # no tokens: done without a device, the pointers may be null
    e4, e2 = D(cg, (0, 4, 128), ptr=0), D(cg, (0, 2, 128), ptr=0)
    assert rope(cg, Q=e4, K=e2, Qo=e4, Ko=e2) == cg.OK


def rope_bwd(cg, **over):
    q, k = (lambda: D(cg, (10, 4, 128))), (lambda: D(cg, (10, 2, 128)))
    a = dict(dQo=q(), dKo=k(), Q=q(), K=k(), gq=D(cg, (128,)), gk=D(cg, (128,)), w=D(cg, (64,), cg.F32), dQ=q(),
             dK=k(), dgq=D(cg, (128,), cg.F32), dgk=D(cg, (128,), cg.F32), ws=PTR)
    need = cg.lib().chain_qk_norm_rope_bwd_workspace_size(R(a["Q"]))
    assert need > 0
    a["size"] = need
    a.update(over)
    return cg.lib().chain_qk_norm_rope_bwd(R(a["dQo"]), R(a["dKo"]), R(a["Q"]), R(a["K"]), R(a["gq"]), R(a["gk"]),
                                           R(a["w"]), None, 1e-6, 0, R(a["dQ"]), R(a["dK"]), R(a["dgq"]),
                                           R(a["dgk"]), a["ws"], a["size"], None)


def test_qk_norm_rope_bwd(cg):
    assert rope_bwd(cg) in no_device(cg)
    for name in ("dQo", "dKo", "Q", "K", "gq", "gk", "dQ", "dK", "dgq", "dgk", "ws"):
        assert rope_bwd(cg, **{name: None}) == cg.ERR_ARG, name
    assert rope_bwd(cg, size=100) == cg.ERR_ARG
    assert rope_bwd(cg, ws=PTR + 8) == cg.ERR_ARG
    assert rope_bwd(cg, dgq=D(cg, (64,), cg.F32)) == cg.ERR_ARG
    assert rope_bwd(cg, dgk=D(cg, (128,))) == cg.ERR_DTYPE
    assert rope_bwd(cg, dQo=D(cg, (11, 4, 128))) == cg.ERR_ARG
    assert rope_bwd(cg, dK=D(cg, (10, 2, 128), cg.F32)) == cg.ERR_DTYPE
    assert cg.lib().chain_qk_norm_rope_bwd_workspace_size(None) == 0
    assert cg.lib().chain_qk_norm_rope_bwd_workspace_size(R(D(cg, (10, 4, 96)))) == 0


def paged(cg, call, **over):
    a = dict(Q=D(cg, (10, 4, 128)), K=D(cg, (10, 2, 128)), V=D(cg, (10, 2, 128)), gq=D(cg, (128,)),
             gk=D(cg, (128,)), w=D(cg, (64,), cg.F32), eps=1e-6, pairs=0, cu=PTR, lens=PTR, table=PTR, stride=7,
             batch=3, max_pages=7, Kc=D(cg, (20, 16, 2, 128)), Vc=D(cg, (20, 16, 2, 128)), Qo=D(cg, (10, 4, 128)),
             mask=1, scale=0.1, O=D(cg, (10, 4, 128)), L=D(cg, (4, 10), cg.F32), ws=PTR)
    a["size"] = cg.lib().chain_fwd_paged_workspace_size(R(a["Q"]), R(a["Kc"]))
    assert a["size"] > 0
    a.update(over)
    seqs = (a["cu"], a["lens"], a["table"], a["stride"], a["batch"], a["max_pages"])
    lib = cg.lib()
    if call == "append":
        return lib.chain_paged_append(R(a["K"]), R(a["V"]), *seqs, R(a["Kc"]), R(a["Vc"]), None)
    if call == "norm_append":
        return lib.chain_qk_norm_rope_append(R(a["Q"]), R(a["K"]), R(a["V"]), R(a["gq"]), R(a["gk"]), R(a["w"]),
                                             a["eps"], a["pairs"], *seqs, R(a["Kc"]), R(a["Vc"]), R(a["Qo"]), None)
    return lib.chain_fwd_paged(R(a["Q"]), R(a["Kc"]), R(a["Vc"]), *seqs, a["mask"], ctypes.c_float(a["scale"]),
                               R(a["O"]), R(a["L"]), a["ws"], a["size"], None)


USES = {"append": ("K", "V"), "norm_append": ("Q", "K", "V", "gq", "gk", "Qo"), "attn": ("Q", "O", "L", "ws")}


@pytest.mark.parametrize("call", USES)
def test_paged(cg, call):
    big = lambda page: dict(Kc=D(cg, (20, page, 2, 128)), Vc=D(cg, (20, page, 2, 128)))
    for ok in (dict(), big(64), big(1024), dict(Kc=D(cg, (20, 16, 2, 128), strides=(4096, 128, 2048, 1))),
               dict(batch=1, stride=0)):
        assert paged(cg, call, **ok) in no_device(cg), ok
    for name in USES[call] + ("cu", "lens", "table", "Kc", "Vc"):
        assert paged(cg, call, **{name: None}) == cg.ERR_ARG, name
    for bad in (dict(batch=-1), dict(batch=2 ** 21), dict(max_pages=0), dict(max_pages=-4), dict(stride=6),
                dict(max_pages=2 ** 27, stride=2 ** 27), dict(cu=PTR + 1), dict(lens=PTR + 2), dict(table=PTR + 3),
                dict(Vc=D(cg, (21, 16, 2, 128))), dict(Kc=D(cg, (20, 16, 128))),
                dict(Kc=D(cg, (20, 16, 2, 128), ptr=PTR + 8)),
                dict(Kc=D(cg, (20, 16, 2, 128), strides=(4096, 260, 128, 1))),
                dict(Kc=D(cg, (20, 16, 2, 128), strides=(0, 256, 128, 1)))):
        assert paged(cg, call, **bad) == cg.ERR_ARG, bad
    for page in (8, 24, 96, 2048):
        assert paged(cg, call, **big(page)) == cg.ERR_UNSUPPORTED, page
    f = D(cg, (20, 16, 2, 128), cg.F32)
    assert paged(cg, call, Kc=f, Vc=f) == cg.ERR_DTYPE
    assert paged(cg, call, batch=0) == cg.OK
    x = USES[call][0]
    shape = tuple(D(cg, (10, 4 if x == "Q" else 2, 128)).shape[:3])
    assert paged(cg, call, **{x: D(cg, shape, cg.F32)}) == cg.ERR_DTYPE
    assert paged(cg, call, **{x: D(cg, (10, 3, 128))}) == cg.ERR_ARG      # heads
    assert paged(cg, call, **{x: D(cg, shape[:2] + (64,))}) == cg.ERR_ARG


def test_norm_append_only(cg):
    for bad in (dict(eps=0.0), dict(pairs=3), dict(w=D(cg, (68,), cg.F32)), dict(Qo=D(cg, (10, 5, 128))),
                dict(V=D(cg, (9, 2, 128))), dict(gk=D(cg, (64,)))):
        assert paged(cg, "norm_append", **bad) == cg.ERR_ARG, bad
    assert paged(cg, "norm_append", w=None) in no_device(cg)


def test_attention_only(cg):
    for bad in (dict(mask=2), dict(scale=0.0), dict(scale=math.nan), dict(size=8), dict(ws=PTR + 4),
                dict(O=D(cg, (10, 5, 128))), dict(L=D(cg, (4, 11), cg.F32)),
                dict(L=D(cg, (4, 10), cg.F32, strides=(9, 1)))):
        assert paged(cg, "attn", **bad) == cg.ERR_ARG, bad
    assert paged(cg, "attn", L=D(cg, (4, 10))) == cg.ERR_DTYPE
    assert paged(cg, "attn", batch=8193) == cg.ERR_UNSUPPORTED
    wide = dict(Q=D(cg, (10, 258, 128)), O=D(cg, (10, 258, 128)), L=D(cg, (258, 10), cg.F32))
    assert paged(cg, "attn", **wide) == cg.ERR_UNSUPPORTED  # 129 query heads to a key head
    size = cg.lib().chain_fwd_paged_workspace_size
    q, pool = D(cg, (10, 4, 128)), D(cg, (20, 16, 2, 128))
    assert size(R(q), R(pool)) > 0
    for a, b in ((None, pool), (q, None), (D(cg, (10, 4, 64)), pool), (D(cg, (10, 3, 128)), pool),
                 (q, D(cg, (20, 24, 2, 128))), (D(cg, (10, 4, 128), cg.F32), pool)):
        assert size(R(a), R(b)) == 0
    # no tokens: done without a device
    e, l = D(cg, (0, 4, 128), ptr=0), D(cg, (4, 0), cg.F32, ptr=0)
    assert paged(cg, "attn", Q=e, O=e, L=l) == cg.OK


def test_strides_out_of_reach(cg):
    # no tensor spans 2^40 bytes: refused before a copy is described with such a stride
    for far in (2 ** 39, 2 ** 61, 2 ** 63 - 8):
        assert rope(cg, Q=D(cg, (10, 4, 128), strides=(far, 128, 1))) == cg.ERR_ARG
        assert paged(cg, "attn", Q=D(cg, (10, 4, 128), strides=(far, 128, 1))) == cg.ERR_ARG
        assert paged(cg, "append", Kc=D(cg, (20, 16, 2, 128), strides=(far, 256, 128, 1))) == cg.ERR_ARG
