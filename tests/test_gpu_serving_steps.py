"""GPU: a server's steps with the calls in the order in which they are used: pages planned, norm + rotation into the
cache, attention behind a shared prompt, rejected tokens and finished requests trimmed.  The state is kept in place.
Attention is checked against the definition in 64 bits on what the cache holds, with the tolerances of
test_gpu_paged; the bookkeeping for whole numbers."""
import types

import pytest
import torch

import chain_synth as cs
from test_gpu_paged import cg, check  # noqa: F401  (cg: the fixture)
from test_gpu_qk_norm_rope import EPS, freqs

pytestmark = pytest.mark.gpu

H, HKV, D, PAGE, POOL = 8, 2, 128, 32, 160


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, cg, batch, max_pages, rows, seed=0):
        self.cg, self.rows = cg, rows
        self.kc, self.vc = (torch.full((POOL, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        g = torch.Generator().manual_seed(seed)
        self.free, self.count = torch.randperm(POOL, generator=g).int().cuda(), ints([POOL])
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.w, self.gq, self.gk = freqs(D).cuda(), *((1 + 0.1 * cs.normal((D,), s, dtype=torch.float32)).cuda() for s in (1, 2))
        self.out = (torch.empty(batch + 1, dtype=torch.int32, device="cuda"), self.lens, self.count,
                    torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int64, device="cuda"))
        self.ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")

    def write(self, news, qkv):
        """Plans the new tokens and writes them; returns (cu_seqlens, rotated queries)."""
        cg = self.cg
        cu = cg.page_plan(news, self.lens, self.table, self.free, self.count, PAGE, self.rows, out=self.out,
                          workspace=self.ws)[0]
        q = cg.qk_norm_rope_append(qkv[:, :H], qkv[:, H:H + HKV], qkv[:, H + HKV:], self.gq, self.gk, self.w, self.kc,
                                   self.vc, cu, self.lens, self.table, eps=EPS)
        return cu, q

    def trim(self, keep):
        self.cg.page_trim(keep, self.lens, self.table, self.free, self.count, PAGE, POOL, out=(self.lens, self.count),
                          workspace=self.ws)

    def held(self, b):
        n = -(-int(self.lens[b]) // PAGE)
        return self.table[b, :n].tolist()

    def view(self, cu):
        """The sequences as the checks of the attention take them."""
        c = types.SimpleNamespace(cu=cu.cpu(), lens=self.lens.tolist(), Hkv=HKV, d=D, k=[], v=[])
        for b, L in enumerate(c.lens):
            pages = torch.tensor(self.held(b), dtype=torch.long, device="cuda")
            c.k.append(self.kc[pages].reshape(-1, HKV, D)[:L].cpu())
            c.v.append(self.vc[pages].reshape(-1, HKV, D)[:L].cpu())
        return c


def shared_prompt(cg, batch, prompt, max_pages, rows):
    """A server whose `batch` sequences all begin with the prompt, written once."""
    s = Server(cg, batch, max_pages, rows)
    s.write(ints([prompt] + [0] * (batch - 1)), cs.normal((rows, H + 2 * HKV, D), 3).cuda())
    assert cg.chain_check()[0] == 0
    m = prompt // PAGE
    s.table[1:, :m] = s.table[0, :m]
    s.lens.fill_(prompt)
    return s


def test_steps_of_a_batch_behind_a_shared_prompt(cg):
    B, prompt, rows = 6, 288, 300  # nine whole pages, rows enough for the prompt
    s = shared_prompt(cg, B, prompt, 20000, rows)  # a table so wide that the prefix is taken by itself
    assert int(s.count) == POOL - prompt // PAGE
    gcu, glens = ints([0, B]), ints([prompt])
    for step, (news, rejected) in enumerate([([1] * 6, [0] * 6), ([3, 1, 5, 1, 40, 4], [2, 0, 4, 1, 9, 0]),
                                             ([1, 0, 1, 1, 0, 1], [0] * 6), ([4] * 6, [3, 0, 2, 4, 1, 3]), ([33] * 6, [0] * 6)]):
        qkv = cs.normal((rows, H + 2 * HKV, D), 10 + step).cuda()
        before = s.lens.tolist()
        cu, q = s.write(ints(news), qkv)
        o, lse = cg.attention_fwd_paged_prefix(q, s.kc, s.vc, cu, s.lens, s.table, gcu, glens, causal=True)
        assert cg.chain_check()[0] == 0
        assert s.lens.tolist() == [a + b for a, b in zip(before, news)]
        n = sum(news)
        # the plan's slot map names what was written, its positions the rotation
        pos = torch.cat([torch.arange(a, a + m) for a, m in zip(before, news)]).int().cuda()
        assert torch.equal(s.out[3][:n], pos) and s.out[3][n:].tolist() == [-1] * (rows - n)
        rq, rk = cg.qk_norm_rope(qkv[:n, :H], qkv[:n, H:H + HKV], s.gq, s.gk, s.w, pos, eps=EPS)
        slots = s.out[4][:n]
        assert torch.equal(q[:n], rq) and torch.equal(s.kc.view(-1, HKV, D)[slots], rk)
        assert torch.equal(s.vc.view(-1, HKV, D)[slots], qkv[:n, H + HKV:])
        check(s.view(cu), q.cpu(), o, lse, True, D ** -0.5)
        s.trim(s.lens - ints(rejected))
        assert cg.chain_check()[0] == 0
        # every page is in one place, but for the prompt's
        own = [p for b in range(B) for p in s.held(b)[prompt // PAGE:]]
        free = s.free[:int(s.count)].tolist()
        assert sorted(own + free + s.held(0)[:prompt // PAGE]) == list(range(POOL))
    s.trim(ints([prompt] * (B - 1) + [0]))  # the last one returns the prompt
    assert int(s.count) == POOL and sorted(s.free.tolist()) == list(range(POOL))
    assert s.lens.tolist() == [prompt] * (B - 1) + [0] and cg.chain_check()[0] == 0


def test_a_step_captured_and_replayed(cg):
    # plan, write, attention and trim in one graph, the state in place, a batch padded with idle sequences
    B, prompt, rows = 8, 256, 260
    s = shared_prompt(cg, B, prompt, 16000, rows)
    s.lens[6:] = 0
    rows_step = 10
    s.rows, s.out = rows_step, (*s.out[:3], s.out[3][:rows_step], s.out[4][:rows_step])
    gcu, glens, news, keep = ints([0, B]), ints([prompt]), ints([1] * 6 + [0, 0]), ints([10 ** 6] * B)
    qkv = torch.empty(rows_step, H + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
    ws = None

    def step():
        cu, q = s.write(news, qkv)
        o, lse = cg.attention_fwd_paged_prefix(q, s.kc, s.vc, cu, s.lens, s.table, gcu, glens, causal=True, workspace=ws)
        s.trim(keep)
        return cu, q, o, lse

    qkv.copy_(cs.normal(tuple(qkv.shape), 20))
    ws = torch.empty(cg.chain_fwd_paged_prefix_workspace_size(qkv[:, :H], s.kc), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cu, q, o, lse = step()
    for i in range(1, 5):
        qkv.copy_(cs.normal(tuple(qkv.shape), 20 + i))
        g.replay()
        assert cg.chain_check()[0] == 0
        assert s.lens.tolist() == [prompt + 1 + i] * 6 + [0, 0]
        check(s.view(cu), q.cpu(), o, lse, True, D ** -0.5)


@pytest.mark.parametrize("name", ["plan", "trim", "prefix"])
def test_outputs_belong_to_the_stream_given(cg, name):
    # memory that the current stream has freed but still writes must not become another stream's output
    s = shared_prompt(cg, 5, 256, 20000, 300)
    cu, q = s.write(ints([1, 7, 30, 1, 1]), cs.normal((300, H + 2 * HKV, D), 5).cuda())
    news, keep, gcu, glens = ints([3, 1, 60, 0, 2]), ints([256] * 5), ints([0, 5]), ints([256])
    table, free = s.table.clone(), s.free.clone()
    f = {"plan": lambda st: cg.page_plan(news, s.lens, table, s.free, s.count, PAGE, 70, stream=st),
         "trim": lambda st: cg.page_trim(keep, s.lens, s.table, free, s.count, PAGE, POOL, stream=st),
         "prefix": lambda st: tuple(x[:40] for x in cg.attention_fwd_paged_prefix(
             q, s.kc, s.vc, cu, s.lens, s.table, gcu, glens, causal=True, stream=st)[:1])}[name]
    ref = [x.clone() for x in f(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (side, side.cuda_stream):
        torch.cuda._sleep(200_000_000)
        junk = [torch.empty_like(x) for x in ref for _ in range(3)]
        for x in junk:
            x.fill_(7)
        del junk
        out = f(st)
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
    assert cg.chain_check()[0] == 0


@pytest.mark.parametrize("news", [[1, 1], [40, 3]])
def test_prefix_with_offsets_past_32_bits(cg, news):
    # pages, queries and outputs further apart than 2^31 elements
    far, page, Hkv, heads = 2 ** 31 + 512, 256, 1, 2
    n = sum(news)
    store = torch.empty(3 * far + 2 ** 21, dtype=torch.bfloat16, device="cuda")
    pool = lambda at: store.as_strided((4, page, Hkv, D), (far, D, D, 1), at)
    kc, vc = pool(0), pool(page * D)
    lens, prefix = [256 + 50, 256 + 20], 256
    k = [cs.normal((L, Hkv, D), 30 + b) for b, L in enumerate(lens)]
    v = [cs.normal((L, Hkv, D), 40 + b) for b, L in enumerate(lens)]
    k[1][:prefix], v[1][:prefix] = k[0][:prefix], v[0][:prefix]
    for c, x in ((kc, k), (vc, v)):
        c[3] = x[0][:prefix].cuda()
        c[1, :50], c[0, :20] = x[0][prefix:].cuda(), x[1][prefix:].cuda()
    table = torch.full((2, 600), -1, dtype=torch.int32)
    table[:, 0] = 3
    table[0, 1], table[1, 1] = 1, 0
    q = cs.normal((n, heads, D), 50)
    qf = store.as_strided((3, heads, D), (far, D, 1), 2 ** 20)[:n] if n <= 3 else q.cuda()
    qf.copy_(q)
    cu = ints([0, news[0], n])
    o, lse = cg.attention_fwd_paged_prefix(qf, kc, vc, cu, ints(lens), table.cuda(), ints([0, 2]), ints([prefix]), causal=True)
    assert cg.chain_check()[0] == 0
    check(types.SimpleNamespace(cu=cu.cpu(), lens=lens, Hkv=Hkv, d=D, k=k, v=v), q, o, lse, True, D ** -0.5)
