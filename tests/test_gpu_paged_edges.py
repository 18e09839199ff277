"""GPU: the norm + rotation and paged-cache calls where they could go wrong --
other streams and two calls at once, captured graphs, offsets past 32 bits,
the largest batch, shared pages and rows behind what is packed.  Attention is
checked against the definition in 64 bits with the tolerances of
test_gpu_paged; the rest bit for bit against the same call made plainly."""
import pytest
import torch

import chain_synth as cs
from test_gpu_paged import Cache, cg, check  # noqa: F401  (cg: the fixture)
from test_gpu_qk_norm_rope import EPS, freqs

pytestmark = pytest.mark.gpu


def calls(cg, d=128):
    """Each call on inputs of its own, as f(stream) -> outputs."""
    c = Cache([300, 1, 77], [130, 1, 5], 2, d, 32, 31).fill().cuda()
    q, k, v = (cs.normal((c.total, h, d), 60 + h).cuda() for h in (8, 2, 2))
    g, w = (1 + 0.1 * cs.normal((d,), 64, dtype=torch.float32)).cuda(), freqs(d).cuda()
    return {
        "forward": lambda s: cg.qk_norm_rope(q, k, g, g, w, stream=s),
        "backward": lambda s: cg.qk_norm_rope_bwd(q, k, q, v, g, g, w, stream=s),
        "append": lambda s: (cg.qk_norm_rope_append(q, k, v, g, g, w, c.kcd.clone(), c.vcd.clone(), *c.args,
                                                    stream=s),),
        "attention": lambda s: cg.attention_fwd_paged(q, c.kcd, c.vcd, *c.args, causal=True, stream=s),
    }


@pytest.mark.parametrize("name", ["forward", "backward", "append", "attention"])
def test_outputs_belong_to_the_stream_given(cg, name):
    # memory that the current stream has freed but still writes must not become another stream's output
    f = calls(cg)[name]
    ref = [x.clone() for x in f(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        torch.cuda._sleep(200_000_000)
        junk = [torch.empty_like(x) for x in ref for _ in range(2)]
        for x in junk:
            x.fill_(7)
        del junk
        out = f(s)
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b)


def test_two_calls_at_once(cg):
    # two streams, their launches interleaved: every result as alone
    H, d = 16, 64
    cases = [Cache(lens, news, 2, d, 16, 80 + i).fill().cuda()
             for i, (lens, news) in enumerate([([3000, 20, 700], [1, 1, 90]), ([1900, 1900], [1, 1])])]
    qs = [cs.normal((c.total, H, d), 85 + i).cuda() for i, c in enumerate(cases)]
    ws = [torch.empty(cg.chain_fwd_paged_workspace_size(q, c.kcd), dtype=torch.uint8, device="cuda")
          for q, c in zip(qs, cases)]
    g, w = torch.ones(d, device="cuda"), freqs(d).cuda()
    both = lambda i, s: (*cg.attention_fwd_paged(qs[i], cases[i].kcd, cases[i].vcd, *cases[i].args, causal=True,
                                                 workspace=ws[i], stream=s),
                         *cg.qk_norm_rope_bwd(qs[i], qs[i], qs[i], qs[i], g, g, w, stream=s))
    ref = [[x.clone() for x in both(i, None)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            outs[i].append(both(i, streams[i]))
    torch.cuda.synchronize()
    assert cg.chain_check()[0] == 0
    for i in range(2):
        for out in outs[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, ref[i]))


def test_a_layer_captured(cg):
    # append, attention, norm forward and backward in one graph: replays give the eager bits
    H, Hkv, d = 8, 2, 128
    c = Cache([260, 40, 1], [4, 40, 1], Hkv, d, 16, 90).fill().cuda()
    q, k, v = (cs.normal((c.total, h, d), 91 + h).cuda() for h in (H, Hkv, Hkv))
    g, w = torch.ones(d, device="cuda"), freqs(d).cuda()
    ws = torch.empty(cg.chain_fwd_paged_workspace_size(q, c.kcd), dtype=torch.uint8, device="cuda")

    def layer():
        qo = cg.qk_norm_rope_append(q, k, v, g, g, w, c.kcd, c.vcd, *c.args, eps=EPS)
        o, lse = cg.attention_fwd_paged(qo, c.kcd, c.vcd, *c.args, causal=True, workspace=ws)
        return (qo, o, lse, *cg.qk_norm_rope(q, k, g, g, w, eps=EPS), *cg.qk_norm_rope_bwd(o, v, q, k, g, g, w, eps=EPS))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ref = [x.clone() for x in layer()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for _ in range(3):
        for x in out:
            x.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert cg.chain_check()[0] == 0


def test_offsets_past_32_bits(cg):
    # pages, tokens and heads further apart than 2^31 elements
    far, d, page, Hkv, H = 2 ** 31 + 512, 128, 16, 1, 2
    store = torch.empty(2 * far + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    pool = lambda at: store.as_strided((3, page, Hkv, d), (far, d, d, 1), at)
    kc, vc = pool(0), pool(4096)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    old = cs.normal((2, 37, Hkv, d), 95)
    q, k, v = cs.normal((3, H, d), 96), cs.normal((3, Hkv, d), 97), cs.normal((3, Hkv, d), 98)
    qf = store.as_strided((3, H, d), (far, d, 1), 2 ** 17)
    kf = store.as_strided((3, Hkv, d), (far, d, 1), 2 ** 18)
    vf = store.as_strided((3, Hkv, d), (far, d, 1), 2 ** 18 + 512)
    for x, y in ((qf, q), (kf, k), (vf, v)):
        x.copy_(y)
    first = torch.tensor([0, 37], dtype=torch.int32, device="cuda")
    cg.chain_paged_append(old[0].cuda(), old[1].cuda(), first, torch.tensor([37], dtype=torch.int32, device="cuda"),
                          table, kc, vc)
    cg.chain_paged_append(kf, vf, cu, lens, table, kc, vc)
    assert cg.chain_check()[0] == 0
    keys, vals = torch.cat((old[0], k)), torch.cat((old[1], v))
    for i, p in enumerate((2, 0, 1)):
        n = min(page, 40 - i * page)
        assert torch.equal(kc[p, :n].cpu(), keys[i * page:i * page + n])
        assert torch.equal(vc[p, :n].cpu(), vals[i * page:i * page + n])
    o, lse = cg.attention_fwd_paged(qf, kc, vc, cu, lens, table, causal=True)
    c = Cache([40], [3], Hkv, d, page, 99)
    c.k, c.v = [keys], [vals]
    check(c, q, o, lse, True, d ** -0.5)
    g, w = torch.ones(d, device="cuda"), freqs(d).cuda()
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    ref = cg.qk_norm_rope(q.cuda(), k.cuda(), g, g, w, pos)
    bwd = cg.qk_norm_rope_bwd(q.cuda(), k.cuda(), q.cuda(), k.cuda(), g, g, w, pos)
    assert all(torch.equal(a, b) for a, b in zip(cg.qk_norm_rope(qf, kf, g, g, w, pos), ref))
    assert all(torch.equal(a, b) for a, b in zip(cg.qk_norm_rope_bwd(qf, kf, qf, kf, g, g, w, pos), bwd))
    cg.chain_qk_norm_rope(qf, kf, g, g, w, pos, 1e-6, 0, qf, kf)
    assert torch.equal(qf, ref[0]) and torch.equal(kf, ref[1])


def test_rows_beyond_the_packed_ones(cg):
    # cu_seqlens past the packed rows counts only those: the writes and the attention agree on the positions
    d, Hkv, H = 64, 2, 4
    c = Cache([50], [8], Hkv, d, 16, 101).cuda()
    k, v, q = cs.normal((8, Hkv, d), 102).cuda(), cs.normal((8, Hkv, d), 103).cuda(), cs.normal((8, H, d), 104).cuda()
    g, w = torch.ones(d, device="cuda"), freqs(d).cuda()
    over = torch.tensor([0, 11], dtype=torch.int32, device="cuda")
    pools = [[c.kc.cuda(), c.vc.cuda()] for _ in range(2)]
    for p, cu in zip(pools, (c.cud, over)):
        cg.chain_paged_append(k, v, cu, c.lensd, c.tabled, *p)
        p.append(cg.qk_norm_rope_append(q, k, v, g, g, w, *(x.clone() for x in p), cu, c.lensd, c.tabled))
    for a, b in zip(*pools):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    c.fill().cuda()
    for a, b in zip(*(cg.attention_fwd_paged(q, c.kcd, c.vcd, cu, c.lensd, c.tabled, causal=True)
                      for cu in (c.cud, over))):
        assert torch.equal(a, b)
    assert cg.chain_check()[0] == 0


def test_largest_batch(cg):
    B = 8192
    lens = [(13 * i) % 45 + 1 for i in range(B)]
    c = Cache(lens, [1] * B, 1, 64, 16, 105).fill().cuda()
    q = cs.normal((B, 2, 64), 106)
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=True)
    assert cg.chain_check()[0] == 0
    some = list(range(0, B, 37)) + [B - 1]
    s = Cache([lens[i] for i in some], [1] * len(some), 1, 64, 16, 107)
    s.k, s.v = [c.k[i] for i in some], [c.v[i] for i in some]
    check(s, q[some], o[some], lse[:, some], True, 64 ** -0.5)


def test_shared_pages_and_pools_of_two_layouts(cg):
    # two sequences that share a prefix's pages, K token-major and V head-major, rows of the table further apart
    Hkv, d, page = 2, 128, 16
    c = Cache([48, 70], [1, 20], Hkv, d, page, 108)
    c.table[1, :3] = c.table[0, :3]
    c.k[1][:48], c.v[1][:48] = c.k[0], c.v[0]
    c.fill()
    wide = torch.full((2, c.table.shape[1] + 5), -3, dtype=torch.int32)
    wide[:, :c.table.shape[1]] = c.table
    vc = c.vc.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    c.cuda()
    q = cs.normal((c.total, 6, d), 109)
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, vc, c.cud, c.lensd, wide.cuda()[:, :c.table.shape[1]], causal=True)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, True, d ** -0.5)


# many units to a block, many key tiles to a unit: both forms of a unit, cut and whole
LONG = {
    "tokens, d 128": ([4000 - 61 * i for i in range(40)], [1] * 40, 16, 8, 128, 64),
    "tokens, d 64": ([4000 - 61 * i for i in range(40)], [1] * 40, 16, 8, 64, 16),
    "chunks, d 128": ([3100, 2500, 1700], [700, 129, 64], 16, 4, 128, 128),
    "chunks, d 64": ([3100, 2500, 1700], [700, 129, 64], 16, 4, 64, 32),
    "mixed, d 64": ([2900 - 83 * i for i in range(30)], [1 if i % 3 else 40 + 7 * i for i in range(30)], 8, 2, 64, 16),
    "mixed, d 128": ([2900 - 83 * i for i in range(30)], [1 if i % 3 else 40 + 7 * i for i in range(30)], 8, 2, 128, 16),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", LONG)
def test_long(cg, name, causal):
    lens, news, H, Hkv, d, page = LONG[name]
    c = Cache(lens, news, Hkv, d, page, 120 + len(name)).fill().cuda()
    q = cs.normal((c.total, H, d), 121)
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=causal)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, causal, d ** -0.5)


# calls with no more new tokens than sequences, or few rows in all: tiles of 16 rows
FEW = {
    "some tokens each": ([700, 0, 90, 5, 300], [3, 0, 2, 0, 0], 8, 2, 128, 16),
    "all in one sequence": ([10, 2000, 9, 9, 9, 9, 9], [0, 7, 0, 0, 0, 0, 0], 6, 2, 64, 32),
    "two tokens, cut": ([3000], [2], 8, 1, 128, 64),
    "four tokens of one sequence, cut": ([1500], [4], 12, 3, 64, 16),
    "sixteen rows, cut": ([2500], [1], 16, 1, 128, 64),
    "group of 11": ([400, 1, 129], [1, 1, 1], 22, 2, 64, 16),
    "group of 5, many units": ([33 * i + 1 for i in range(60)], [1] * 60, 15, 3, 128, 16),
    "one head, many units": ([77 * i + 1 for i in range(40)], [1] * 40, 6, 6, 64, 64),
    "more new than cached": ([1, 0, 300], [2, 1, 0], 4, 2, 128, 16),
    "seventeen rows a token": ([500, 3], [1, 1], 17, 1, 128, 16),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", FEW)
def test_few_rows(cg, name, causal):
    lens, news, H, Hkv, d, page = FEW[name]
    c = Cache(lens, news, Hkv, d, page, 140 + len(name), heads_first=len(name) % 2 == 0).fill().cuda()
    q = cs.normal((c.total, H, d), 141)
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=causal)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, causal, d ** -0.5)


def test_few_rows_strided_and_rows_behind_the_last_sequence(cg):
    c = Cache([200, 90, 400], [1, 1, 0], 2, 128, 16, 151, pad_rows=1).fill().cuda()
    H, d = 6, 128
    qkv = cs.normal((c.total, H + 4, d), 152)
    o = torch.full((c.total, 2 * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, c.total + 3), 9.0, device="cuda")
    ws = torch.full((cg.chain_fwd_paged_workspace_size(qkv[:, :H], c.kcd),), 255, dtype=torch.uint8, device="cuda")
    ov, lv = o[:, H:], lse[:, :c.total]
    cg.chain_fwd_paged(qkv.cuda()[:, :H], c.kcd, c.vcd, *c.args, cg.MASK_CAUSAL, 0.3, ov, lv, ws)
    assert cg.chain_check()[0] == 0
    check(c, qkv[:, :H], ov, lv, True, 0.3)
    n = int(c.cu[-1])
    assert bool((o[:, :H] == 7).all()) and bool((o[n:] == 7).all()) and bool((lse[:, n:] == 9).all())


def test_few_rows_large_scores(cg):
    c = Cache([900], [1], 1, 128, 64, 153)
    c.k[0] = (c.k[0].float() * torch.linspace(0.1, 20, 900)[:, None, None]).bfloat16()
    c.fill().cuda()
    q = cs.normal((1, 2, 128), 154) * 3
    o, lse = cg.attention_fwd_paged(q.cuda(), c.kcd, c.vcd, *c.args, causal=True, scale=0.5)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, True, 0.5)


@pytest.mark.parametrize("news", [[1, 1], [30, 20]])
def test_missing_pages_count_as_zeros(cg, news):
    # on both sides of the choice of kernel: reported, not accessed; the other sequence is as without
    c = Cache([300, 120], news, 2, 128, 16, 155).fill().cuda()
    q = cs.normal((sum(news), 8, 128), 156).cuda()
    ref, rl = cg.attention_fwd_paged(q, c.kcd, c.vcd, *c.args, causal=True)
    good = c.tabled.clone()
    for bad in (-1, c.kcd.shape[0], 2 ** 31 - 1):
        c.tabled.copy_(good)
        c.tabled[0, 3] = bad
        o, lse = cg.attention_fwd_paged(q, c.kcd, c.vcd, *c.args, causal=True)
        assert cg.chain_check()[0] == cg.ERR_ARG
        n = news[0]
        assert torch.equal(o[n:], ref[n:]) and torch.equal(lse[:, n:], rl[:, n:])
        z = Cache([300], news[:1], 2, 128, 16, 157)
        z.k, z.v = [c.k[0].clone()], [c.v[0].clone()]
        z.k[0][48:64], z.v[0][48:64] = 0, 0
        check(z, q[:n].cpu(), o[:n], lse[:, :n], True, 128 ** -0.5)
    assert cg.chain_check()[0] == 0


@pytest.mark.parametrize("H", [2, 20])
def test_fused_write_with_missing_pages(cg, H):
    # few heads and many: what cannot be written is reported and leaves the pools alone, its queries are still made
    Hkv, d, page = 1, 128, 16
    c = Cache([70, 33, 9], [40, 33, 2], Hkv, d, page, 161, pad_rows=2).cuda()
    q, k, v = (cs.normal((c.total, h, d), 162 + h).cuda() for h in (H, Hkv, Hkv))
    g, w = (1 + 0.1 * cs.normal((d,), 166, dtype=torch.float32)).cuda(), freqs(d).cuda()
    good = [c.kc.cuda(), c.vc.cuda()]
    qo = torch.full_like(q, 7.0)
    call = lambda table, lens, pools, out: cg.chain_qk_norm_rope_append(q, k, v, g, g, w, EPS, 0, c.cud, lens, table,
                                                                        *pools, out)
    call(c.tabled, c.lensd, good, qo)
    assert cg.chain_check()[0] == 0
    assert bool((qo[int(c.cu[-1]):] == 7).all())
    for bad in (-1, c.kc.shape[0], 2 ** 31 - 1):
        t = c.tabled.clone()
        lost = int(t[0, 3])  # positions 48 to 63 of the first sequence
        t[0, 3] = bad
        pools, out = [c.kc.cuda(), c.vc.cuda()], torch.full_like(q, 7.0)
        call(t, c.lensd, pools, out)
        assert cg.chain_check()[0] == cg.ERR_ARG
        assert torch.equal(out, qo)
        for a, b in zip(pools, good):
            assert bool(torch.isnan(a[lost]).all())
            a[lost] = b[lost]
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # a length below the new tokens: those before position 0 are reported, the others land where they belong
    pools = [c.kc.cuda(), c.vc.cuda()]
    call(c.tabled, torch.tensor([70, 33, 1], dtype=torch.int32, device="cuda"), pools, torch.empty_like(q))
    assert cg.chain_check()[0] == cg.ERR_ARG
    page0, other = int(c.tabled[2, 0]), int(c.tabled[0, 4])
    assert torch.isfinite(pools[0][page0, 0].float()).all() and torch.isnan(pools[0][page0, 1].float()).all()
    assert torch.equal(pools[1][other].view(torch.int16), good[1][other].view(torch.int16))
    assert cg.chain_check()[0] == 0
