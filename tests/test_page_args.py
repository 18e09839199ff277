"""Host-side argument checks of the page plan and page trim, on the CPU: dummy addresses that are never
dereferenced, a bad argument returns its status, and a valid call gets past every check and fails only
at the device query.  Run only where no GPU is visible."""
import pytest

torch = pytest.importorskip("torch")

from test_abi_args import cg, no_device  # noqa: F401  (cg: the fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-side argument checks only; never run with a device present")
PTR = 0x50000000


def plan(cg, **over):
    a = dict(new=PTR, kv=PTR, table=PTR, stride=9, batch=5, max_pages=9, page=16, free=PTR, capacity=40, count=PTR,
             cu=PTR, kv_out=PTR, count_out=PTR, positions=PTR, slots=PTR, rows=30, ws=PTR)
    a["size"] = cg.chain_page_plan_workspace_size(over.get("batch", 5)) if over.get("batch", 5) > 0 else 64
    a.update(over)
    return cg.lib().chain_page_plan(*(a[k] for k in (
        "new", "kv", "table", "stride", "batch", "max_pages", "page", "free", "capacity", "count", "cu", "kv_out",
        "count_out", "positions", "slots", "rows", "ws", "size")), None)


def trim(cg, **over):
    a = dict(keep=PTR, kv=PTR, table=PTR, stride=9, batch=5, max_pages=9, page=16, pool=50, free=PTR, capacity=40,
             count=PTR, kv_out=PTR, count_out=PTR, ws=PTR)
    a["size"] = cg.chain_page_trim_workspace_size(over.get("batch", 5)) if over.get("batch", 5) > 0 else 64
    a.update(over)
    return cg.lib().chain_page_trim(*(a[k] for k in (
        "keep", "kv", "table", "stride", "batch", "max_pages", "page", "pool", "free", "capacity", "count", "kv_out",
        "count_out", "ws", "size")), None)


@pytest.mark.parametrize("call", [plan, trim])
def test_shared_arguments(cg, call):
    for ok in (dict(), dict(page=1024), dict(batch=1, stride=0), dict(batch=8192), dict(capacity=0, free=None),
               dict(batch=0, kv=None, table=None, kv_out=None), dict(stride=1 << 40)):
        assert call(cg, **ok) in no_device(cg), ok
    for name in ("kv", "table", "free", "count", "kv_out", "count_out", "ws"):
        assert call(cg, **{name: None}) == cg.ERR_ARG, name
        assert call(cg, **{name: PTR + 2}) == cg.ERR_ARG, name
    for bad in (dict(batch=-1), dict(max_pages=0), dict(max_pages=-3), dict(stride=8), dict(stride=-9, batch=1),
                dict(capacity=-1), dict(capacity=2 ** 31), dict(ws=PTR + 8), dict(size=8),
                dict(max_pages=2 ** 26 + 1, stride=2 ** 27)):
        assert call(cg, **bad) == cg.ERR_ARG, bad
    for bad in (dict(page=8), dict(page=24), dict(page=0), dict(page=-16), dict(page=2048), dict(batch=8193, size=1 << 30)):
        assert call(cg, **bad) == cg.ERR_UNSUPPORTED, bad


def test_plan_only(cg):
    for ok in (dict(rows=0, positions=None, slots=None), dict(rows=2 ** 30 - 1), dict(positions=PTR + 4)):
        assert plan(cg, **ok) in no_device(cg), ok
    for bad in (dict(new=None), dict(cu=None), dict(rows=-1), dict(rows=2 ** 30), dict(positions=None), dict(slots=None),
                dict(slots=PTR + 4), dict(positions=PTR + 1)):
        assert plan(cg, **bad) == cg.ERR_ARG, bad


def test_trim_only(cg):
    for bad in (dict(keep=None), dict(pool=-1), dict(pool=2 ** 31 - 1)):
        assert trim(cg, **bad) == cg.ERR_ARG, bad
    assert trim(cg, pool=0) in no_device(cg)


def test_workspace_sizes(cg):
    for size in (cg.chain_page_plan_workspace_size, cg.chain_page_trim_workspace_size):
        assert size(0) > 0 and size(8192) > size(1) > 0
        assert size(-1) == 0 and size(8193) == 0


def ints(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def test_the_native_modules_own_checks(cg):
    # host tensors stand in for device tensors, "on the current device" being -1
    def call(**over):
        a = dict(new=ints(3), kv=ints(3), table=ints(3, 4), free=ints(8), count=ints(1), page=16, cu=ints(4),
                 kv_out=ints(3), count_out=ints(1), positions=ints(6), slots=ints(6, dtype=torch.int64),
                 ws=torch.empty(256, dtype=torch.uint8))
        a.update(over)
        cg._small().page_plan(*a.values(), cg._bytes(a["ws"]), -1, 0)

    with pytest.raises(cg.ChainError):  # no device: every check before it passed
        call()
    for bad in (dict(new=ints(2)), dict(kv=ints(4)), dict(table=ints(4, 4)), dict(table=ints(12)), dict(cu=ints(3)),
                dict(count=ints(2)), dict(positions=ints(5)), dict(slots=ints(6)), dict(kv_out=ints(2)),
                dict(new=ints(3, dtype=torch.int64)), dict(free=ints(16)[::2]), dict(table=ints(3, 8)[:, ::2]),
                dict(ws=torch.empty(1, dtype=torch.uint8).expand(256))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(cg.ChainError):  # a row stride below max_pages
        call(table=ints(1, 4).expand(3, 4))
    for page in (2 ** 32 + 16, -16, 0):
        with pytest.raises(cg.ChainError) as e:
            call(page=page)
        assert e.value.status == cg.ERR_UNSUPPORTED

    def trim_call(**over):
        a = dict(keep=ints(3), kv=ints(3), table=ints(3, 4), free=ints(8), count=ints(1), page=16, pool=9,
                 kv_out=ints(3), count_out=ints(1), ws=torch.empty(256, dtype=torch.uint8))
        a.update(over)
        cg._small().page_trim(*a.values(), cg._bytes(a["ws"]), -1, 0)

    with pytest.raises(cg.ChainError):
        trim_call()
    for bad in (dict(keep=ints(2)), dict(kv_out=ints(4)), dict(free=ints(2, 4)), dict(count_out=ints(0))):
        with pytest.raises(ValueError):
            trim_call(**bad)
