"""GPU: the paged K/V cache -- its writes (chain_paged_append,
chain_qk_norm_rope_append) and the attention of a chunk of new tokens over it
(chain_fwd_paged) -- against the definition in 64 bits.

Tolerances of the attention.  O is rounded to bf16 (2^-8 of its value) and P
enters the second product as bf16 (2^-8 of each weight, so 2^-8 of the
weighted sum of |v|).  A score's fp32 error e, at most d 2^-24 of the sum of
|q_i k_i| times the scale, moves each weight by a factor 1 +- 2 e, and so do the
exponentials' 2^-20.  The LSE moves by e and 2^-20 of itself."""
import math

import pytest
import torch

import chain_synth as cs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cg():
    import chain_gb300
    chain_gb300.lib()
    return chain_gb300


class Cache:
    """A pool whose free slots hold NaN, and a table whose unused entries hold nonsense."""

    def __init__(self, lens, news, Hkv, d, page, seed, heads_first=False, spare=3, pad_rows=0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(L, 0) // page) for L in lens]
        pool = sum(need) + spare
        order = torch.randperm(pool, generator=g)
        self.table = torch.full((len(lens), max(1, max(need))), -7, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m].int()
            at += m
        self.lens, self.news, self.page, self.Hkv, self.d = lens, news, page, Hkv, d
        self.k = [cs.normal((L, Hkv, d), seed + 10 + b) for b, L in enumerate(lens)]
        self.v = [cs.normal((L, Hkv, d), seed + 500 + b) for b, L in enumerate(lens)]
        shape = (pool, Hkv, page, d) if heads_first else (pool, page, Hkv, d)
        kc, vc = (torch.full(shape, float("nan"), dtype=torch.bfloat16) for _ in range(2))
        self.kc, self.vc = (x.transpose(1, 2) if heads_first else x for x in (kc, vc))
        self.cu = torch.tensor([0] + news, dtype=torch.int32).cumsum(0).int()
        self.total = int(self.cu[-1]) + pad_rows

    def fill(self):
        for b, L in enumerate(self.lens):
            p = torch.arange(L)
            pages, slots = self.table[b].long()[p // self.page], p % self.page
            self.kc[pages, slots], self.vc[pages, slots] = self.k[b], self.v[b]
        return self

    def cuda(self):
        self.kcd, self.vcd = self.kc.cuda(), self.vc.cuda()  # strides kept
        self.cud, self.tabled = self.cu.cuda(), self.table.cuda()
        self.lensd = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return self

    @property
    def args(self):
        return self.cud, self.lensd, self.tabled


def reference(c, q, b, causal, scale):
    """O [n, H, d], its bound, LSE [H, n], its bound of sequence b, in 64 bits."""
    lo, hi, L = int(c.cu[b]), int(c.cu[b + 1]), c.lens[b]
    n, H = hi - lo, q.shape[1]
    G = H // c.Hkv
    x = q[lo:hi].double().transpose(0, 1)                                       # [H, n, d]
    k = c.k[b].double().transpose(0, 1).repeat_interleave(G, 0)
    v = c.v[b].double().transpose(0, 1).repeat_interleave(G, 0)
    z = x @ k.transpose(1, 2) * scale
    e = (x.abs() @ k.abs().transpose(1, 2) * scale).amax(-1) * c.d * 2.0 ** -24 if L else torch.zeros(H, n).double()
    if causal:
        z.masked_fill_(torch.arange(L)[None, :] > (L - n + torch.arange(n))[:, None], -math.inf)
    lse = torch.logsumexp(z, -1) if L else torch.full((H, n), -math.inf, dtype=torch.float64)
    p = torch.exp(z - lse[..., None])
    p = torch.where(torch.isfinite(lse)[..., None], p, torch.zeros((), dtype=torch.float64))
    o, size = p @ v, p @ v.abs()
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -19 + 4 * e[..., None]) * size
    ltol = e + 2.0 ** -20 * (1 + lse.abs())
    return o.transpose(0, 1), tol.transpose(0, 1), lse, ltol


def check(c, q, o, lse, causal, scale):
    o, lse = o.cpu().double(), lse.cpu().double()
    for b in range(len(c.lens)):
        lo, hi = int(c.cu[b]), int(c.cu[b + 1])
        if lo == hi:
            continue
        ro, tol, rl, ltol = reference(c, q, b, causal, scale)
        err = (o[lo:hi] - ro).abs()
        assert bool((err <= tol).all()), \
            f"sequence {b}: O off by {(err / tol.clamp_min(1e-300)).max():.3f} of its tolerance"
        got = lse[:, lo:hi]
        none = torch.isinf(rl)
        assert torch.equal(got[none], rl[none]), f"sequence {b}: rows that see nothing"
        assert bool(((got - rl)[~none].abs() <= ltol[~none]).all()), f"sequence {b}: LSE"


# lens, news, H, Hkv, d, page, heads first
CASES = {
    "one token, one key": ([1], [1], 8, 2, 128, 16, False),
    "single tokens": ([1, 15, 16, 17, 127, 128, 129, 500], [1] * 8, 8, 1, 128, 16, False),
    "single tokens, d 64": ([2000, 3, 640, 128, 129], [1] * 5, 15, 5, 64, 64, True),
    "long caches": ([5000, 3001], [1, 1], 32, 8, 128, 64, False),
    "chunks": ([300, 256, 130, 1000], [300, 100, 129, 257], 4, 2, 128, 32, True),
    "chunks, d 64": ([300, 64, 511], [299, 64, 200], 6, 6, 64, 128, False),
    "mixed, odd group": ([400, 0, 33, 1500, 70, 12], [60, 0, 1, 1, 70, 5], 14, 2, 128, 16, False),
    "more new than cached": ([5, 0, 130], [9, 3, 200], 6, 3, 64, 16, False),
    "large pages": ([1030, 2049, 90], [40, 1, 90], 8, 4, 128, 1024, False),
    "all heads on one key head": ([700, 129], [3, 1], 128, 1, 64, 256, False),
    "group of 33": ([260, 90], [20, 1], 66, 2, 128, 64, True),
    "many short": ([(7 * i) % 90 + 1 for i in range(200)], [1 + i % 2 if (7 * i) % 90 else 1 for i in range(200)],
                   4, 4, 64, 16, False),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_attention(cg, name, causal):
    lens, news, H, Hkv, d, page, heads_first = CASES[name]
    c = Cache(lens, news, Hkv, d, page, 700 + len(name), heads_first).fill().cuda()
    q = cs.normal((c.total, H, d), 3)
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=causal)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, causal, d ** -0.5)


def test_strided_tensors_and_rows_behind_the_last_sequence(cg):
    c = Cache([200, 90], [33, 1], 2, 128, 16, 41, pad_rows=6).fill().cuda()
    H, d = 6, 128
    qkv = cs.normal((c.total, H + 4, d), 5)
    o = torch.full((c.total, 2 * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, c.total + 3), 9.0, device="cuda")
    ws = torch.full((cg.chain_fwd_paged_workspace_size(qkv[:, :H], c.kcd),), 255, dtype=torch.uint8, device="cuda")
    ov, lv = o[:, H:], lse[:, :c.total]
    cg.chain_fwd_paged(qkv.cuda()[:, :H], c.kcd, c.vcd, *c.args, cg.MASK_CAUSAL, 0.3, ov, lv, ws)
    assert cg.chain_check()[0] == 0
    check(c, qkv[:, :H], ov, lv, True, 0.3)
    n = int(c.cu[-1])
    assert bool((o[:, :H] == 7).all()) and bool((o[n:] == 7).all())
    assert bool((lse[:, n:] == 9).all())


def test_large_scores(cg):
    # scores of hundreds, rising along the keys: the running maximum moves at every tile
    c = Cache([700], [130], 1, 128, 64, 51)
    c.k[0] = (c.k[0].float() * torch.linspace(0.1, 20, 700)[:, None, None]).bfloat16()
    c.fill().cuda()
    q = cs.normal((130, 2, 128), 6) * 3
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=True, scale=0.5)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, True, 0.5)


def test_repeated_calls_and_graph(cg):
    # the same bits from call to call, eager and replayed, with new lengths between replays
    c = Cache([900, 40, 333], [1, 20, 1], 2, 128, 64, 61).fill().cuda()
    q = cs.normal((c.total, 8, 128), 8)
    qd = q.cuda()
    ref, rl = cg.attention_fwd_paged(qd, c.kcd, c.vcd, *c.args, causal=True)
    o, lse = torch.empty_like(ref), torch.empty_like(rl)
    ws = torch.empty(cg.chain_fwd_paged_workspace_size(qd, c.kcd), dtype=torch.uint8, device="cuda")
    call = lambda: cg.chain_fwd_paged(qd, c.kcd, c.vcd, *c.args, cg.MASK_CAUSAL, 128 ** -0.5, o, lse, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        o.zero_()
        g.replay()
        assert torch.equal(o, ref) and torch.equal(lse, rl)
    c.lensd.copy_(torch.tensor([700, 25, 3], dtype=torch.int32))
    c.lens = [700, 25, 3]
    c.k, c.v = ([x[:L] for x, L in zip(t, c.lens)] for t in (c.k, c.v))
    g.replay()
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, True, 128 ** -0.5)


@pytest.mark.parametrize("page,heads_first,d", [(16, False, 128), (64, True, 64)])
def test_append(cg, page, heads_first, d):
    lens, news, H, Hkv = [40, 3, 1, 0, 257, 100], [40, 2, 1, 0, 130, 1], 5, 3
    c = Cache(lens, news, Hkv, d, page, 71, heads_first, pad_rows=4).cuda()
    qkv = cs.normal((c.total, H + 2 * Hkv, d), 9)
    qd, kd, vd = (x for x in qkv.cuda().split((H, Hkv, Hkv), 1))
    pos = torch.cat([torch.arange(L - n, L) for L, n in zip(lens, news)]).int()
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(news)])
    pages, slots = c.table.long()[seq, pos.long() // page], pos.long() % page
    n = len(pos)

    def untouched(pool, old):
        pool, old = pool.cpu().clone(), old.clone()
        pool[pages, slots] = 0
        old[pages, slots] = 0
        assert torch.equal(pool.contiguous().view(torch.int16), old.contiguous().view(torch.int16))

    cg.chain_paged_append(kd, vd, *c.args, c.kcd, c.vcd)
    assert cg.chain_check()[0] == 0
    for pool, x, old in ((c.kcd, kd, c.kc), (c.vcd, vd, c.vc)):
        assert torch.equal(pool.cpu()[pages, slots], x.cpu()[:n])
        untouched(pool, old)
    # norm and rotation at the cache positions: the two calls' results, bit for bit
    gq, gk = ((1 + 0.2 * cs.normal((d,), s, dtype=torch.float32)).cuda() for s in (1, 2))
    w = (10000.0 ** (-torch.arange(0, d, 2) / d)).float().cuda()
    for neighbour in (False, True):
        rq, rk = cg.qk_norm_rope(qd[:n], kd[:n], gq, gk, w, pos.cuda(), interleaved=neighbour)
        k2, v2 = c.kc.cuda(), c.vc.cuda()
        qo = torch.full((c.total, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
        cg.chain_qk_norm_rope_append(qd, kd, vd, gq, gk, w, 1e-6, int(neighbour), *c.args, k2, v2, qo)
        assert cg.chain_check()[0] == 0
        assert torch.equal(qo[:n], rq) and bool((qo[n:] == 3).all())
        assert torch.equal(k2.cpu()[pages, slots], rk.cpu())
        assert torch.equal(v2.cpu()[pages, slots], vd.cpu()[:n])
        untouched(k2, c.kc)
        untouched(v2, c.vc)


def test_missing_pages_and_lengths_are_reported(cg):
    # a page index outside the pool, a length above the table, a position below 0: reported, not accessed
    c = Cache([100, 40], [3, 2], 2, 128, 16, 81).fill().cuda()
    q = cs.normal((5, 4, 128), 1).cuda()
    ok = cg.attention_fwd_paged(q, c.kcd, c.vcd, *c.args, causal=True)[0]
    assert cg.chain_check()[0] == 0
    for bad in (-1, c.kcd.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = c.tabled.clone()
        t[1, 0] = bad
        o, _ = cg.attention_fwd_paged(q, c.kcd, c.vcd, c.cud, c.lensd, t, causal=True)
        assert cg.chain_check()[0] == cg.ERR_ARG
        assert cg.chain_check()[0] == 0
        assert torch.equal(o[:3], ok[:3])  # the other sequence is right
        k2 = c.kcd.clone()
        t[1, 2] = bad  # the new tokens' page
        cg.chain_paged_append(q[:, :2], q[:, 2:], c.cud, c.lensd, t, k2, c.vcd.clone())
        assert cg.chain_check()[0] == cg.ERR_ARG
    for lens in ([100, 1000], [100, -3]):
        o, _ = cg.attention_fwd_paged(q, c.kcd, c.vcd, c.cud, torch.tensor(lens, dtype=torch.int32).cuda(),
                                      c.tabled, causal=True)
        assert cg.chain_check()[0] == cg.ERR_ARG
        assert torch.equal(o[:3], ok[:3])
        cg.chain_paged_append(q[:, :2], q[:, 2:], c.cud, torch.tensor(lens, dtype=torch.int32).cuda(), c.tabled,
                              c.kcd.clone(), c.vcd.clone())
        assert cg.chain_check()[0] == cg.ERR_ARG


def test_nothing_to_do(cg):
    c = Cache([5, 6], [0, 0], 2, 64, 16, 91).cuda()
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = cg.attention_fwd_paged(q, c.kcd, c.vcd, *c.args, causal=True)
    cg.chain_paged_append(q[:, :2], q[:, :2], *c.args, c.kcd, c.vcd)
    assert o.numel() == 0 and cg.chain_check()[0] == 0
    # tokens, but none of them in a sequence
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    cg.attention_fwd_paged(q, c.kcd, c.vcd, *c.args, causal=True)
    cg.chain_paged_append(q[:, :2], q[:, :2], *c.args, c.kcd, c.vcd)
    assert cg.chain_check()[0] == 0
    assert torch.equal(c.kcd.cpu().view(torch.int16), c.kc.view(torch.int16))


def test_refusals(cg):
    c = Cache([5, 6], [1, 1], 2, 64, 16, 92).fill().cuda()
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        cg.attention_fwd_paged(q.half(), c.kcd, c.vcd, *c.args, causal=True)
    with pytest.raises(ValueError):
        cg.attention_fwd_paged(q, c.kcd.cpu(), c.vcd, *c.args, causal=True)
    with pytest.raises(ValueError):
        cg.attention_fwd_paged(q, c.kcd, c.vcd, c.cud[:2], c.lensd, c.tabled, causal=True)
    with pytest.raises(ValueError):
        cg.attention_fwd_paged(q, c.kcd, c.vcd, c.cud, c.lensd.long(), c.tabled, causal=True)
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(cg.ChainError):  # 3 query heads over 2
        cg.attention_fwd_paged(q[:, :3], c.kcd, c.vcd, *c.args, causal=True, workspace=ws)
    with pytest.raises(cg.ChainError):  # short workspace
        cg.attention_fwd_paged(q, c.kcd, c.vcd, *c.args, causal=True, workspace=ws)
    with pytest.raises(cg.ChainError):  # page of 24
        k24 = torch.zeros(4, 24, 2, 64, dtype=torch.bfloat16, device="cuda")
        cg.chain_paged_append(q[:, :2], q[:, :2], *c.args, k24, k24)
    with pytest.raises(cg.ChainError):  # f32 pool
        cg.chain_paged_append(q[:, :2], q[:, :2], *c.args, c.kcd.float(), c.vcd.float())


def test_prompt_in_chunks_then_tokens_matches_whole_attention(cg):
    # norm + rotation into the cache and attention over it, chunk by chunk and then token by token,
    # against the packed attention of the whole sequences
    H, Hkv, d, page = 8, 2, 128, 32
    lens = [200, 77]
    steps = [[100, 40], [97, 30], [1, 1], [1, 1], [1, 5]]
    full = torch.tensor([0, 200, 277], dtype=torch.int32)
    qkv = cs.normal((277, H + 2 * Hkv, d), 12).cuda()
    gq, gk = ((1 + 0.2 * cs.normal((d,), s, dtype=torch.float32)).cuda() for s in (1, 2))
    w = (10000.0 ** (-torch.arange(0, d, 2) / d)).float().cuda()
    pos = torch.cat([torch.arange(L) for L in lens]).int().cuda()
    q, k = cg.qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hkv], gq, gk, w, pos)
    ro, rl = cg.attention_fwd_varlen(q, k, qkv[:, H + Hkv:].contiguous(), full.cuda(), 200, True)
    c = Cache(lens, [0, 0], Hkv, d, page, 99).cuda()
    o, lse = torch.empty_like(ro), torch.empty_like(rl)
    done = [0, 0]
    for news in steps:
        rows = torch.cat([torch.arange(int(full[b]) + done[b], int(full[b]) + done[b] + n)
                          for b, n in enumerate(news)]).cuda()
        done = [x + n for x, n in zip(done, news)]
        cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32).cuda()
        kv = torch.tensor(done, dtype=torch.int32).cuda()
        part = qkv[rows]
        qo = cg.qk_norm_rope_append(part[:, :H], part[:, H:H + Hkv], part[:, H + Hkv:], gq, gk, w, c.kcd, c.vcd,
                                    cu, kv, c.tabled)
        assert torch.equal(qo, q[rows])
        o[rows], l = cg.attention_fwd_paged(qo, c.kcd, c.vcd, cu, kv, c.tabled, causal=True)
        lse[:, rows] = l
    assert done == lens and cg.chain_check()[0] == 0
    # both are within their rounding of the same values: 2^-8 of O each, and P's 2^-8 of sum p |v|
    size = cg.attention_fwd_varlen(q, k, qkv[:, H + Hkv:].abs().contiguous(), full.cuda(), 200, True)[0].float()
    err = (o.float() - ro.float()).abs()
    assert bool((err <= 2.0 ** -7 * ro.float().abs() + 2.0 ** -7 * size).all())
    assert bool(((lse - rl).abs() <= 1e-4).all())
