"""GPU: attention over a paged cache for groups of sequences that share a prefix (chain_fwd_paged_prefix), against
the definition of each sequence by itself in 64 bits.

Tolerances: those of test_gpu_paged, which hold for a sum over two sets of keys as for one.  A row's two
sums are joined in fp32 with weights that are powers of two of differences of maxima: a rounding of 2^-24 each,
within the 2^-19 that is there for the exponentials."""
import pytest
import torch

import chain_synth as cs
from test_gpu_paged import Cache, cg, check, reference  # noqa: F401  (cg: the fixture)
from tol import assert_fwd_close, assert_lse_close

pytestmark = pytest.mark.gpu


class Shared(Cache):
    """Groups of (sequences, shared positions); sequences behind the groups share nothing.  The pages that hold a
    group's shared positions are one set for all its sequences with any cache; a sequence without cache has no pages."""

    def __init__(self, groups, lens, news, Hkv, d, page, seed, heads_first=False, pad_rows=0):
        super().__init__(lens, news, Hkv, d, page, seed, heads_first, pad_rows=pad_rows)
        self.prefix_cu, self.prefix_lens, b = [0], [], 0
        for count, P in groups:
            having = [i for i in range(b, b + count) if lens[i] > 0]
            for i in having[1:]:
                m = -(-P // page)
                self.table[i, :m] = self.table[having[0], :m]
                upto = min(m * page, lens[i])  # the last page's other positions are shared too
                first = min(upto, lens[having[0]])
                self.k[i][:first], self.v[i][:first] = self.k[having[0]][:first], self.v[having[0]][:first]
                if upto > first:  # this sequence reaches further into the last page: the first one has nothing there
                    assert upto - first < page
            b += count
            self.prefix_cu.append(b)
            self.prefix_lens.append(P)

    def cuda(self, wide=True):
        """wide: a table whose rows are so long that the call cannot tell its keys are few."""
        if wide:
            cols = -(-(2 ** 27 + 1) // (len(self.lens) * self.page * self.Hkv * self.d * 4))
            if cols > self.table.shape[1]:
                table = torch.full((len(self.lens), cols), -7, dtype=torch.int32)
                table[:, :self.table.shape[1]] = self.table
                self.table = table
        super().cuda()
        self.gcu = torch.tensor(self.prefix_cu, dtype=torch.int32).cuda()
        self.glens = torch.tensor(self.prefix_lens, dtype=torch.int32).cuda()
        return self

    @property
    def args(self):
        return (*super().args, self.gcu, self.glens)


def made(groups, lens, news, H, Hkv, d, page, seed, wide=True, **kw):
    c = Shared(groups, lens, news, Hkv, d, page, seed, **kw).fill().cuda(wide)
    return c, cs.normal((c.total, H, d), seed + 1)


def behind(P, own, page=16):
    """Lengths of sequences with `own` positions behind the pages of a prefix of P."""
    return [-(-P // page) * page + x for x in own]


# groups, lens, news, H, Hkv, d, page
CASES = {
    "one sequence": ([(1, 256)], [300], [1], 8, 2, 128, 16),
    "two tokens": ([(2, 128)], [129, 140], [1, 1], 8, 2, 128, 16),
    "less than a tile": ([(3, 127)], behind(127, [1, 50, 200]), [1, 1, 1], 8, 2, 64, 16),
    "no prefix at all": ([(3, 0)], [5, 200, 77], [1, 1, 1], 8, 2, 128, 16),
    "inside a page": ([(4, 301)], behind(301, [1, 2, 100, 33], 64), [1] * 4, 12, 4, 128, 64),
    "single tokens": ([(20, 1000)], behind(1000, [1 + 17 * i for i in range(20)]), [1] * 20, 8, 2, 128, 16),
    "single tokens, d 64": ([(20, 1000)], behind(1000, [1 + 17 * i for i in range(20)]), [1] * 20, 15, 5, 64, 16),
    "three rows of 16": ([(4, 700)], behind(700, [1, 9, 30, 300]), [1] * 4, 3, 1, 128, 16),
    "a long prefix": ([(40, 9000)], behind(9000, [1 + i for i in range(40)], 64), [1] * 40, 32, 8, 128, 64),
    "a long prefix, few rows": ([(2, 9000)], behind(9000, [1, 130], 64), [1] * 2, 8, 1, 128, 64),
    "two query tiles and more": ([(150, 640)], behind(640, [1 + i % 40 for i in range(150)], 32), [1] * 150, 8, 2, 64, 32),
    "groups": ([(5, 300), (1, 512), (9, 128), (2, 40)],
               behind(300, [1, 5, 9, 30, 200]) + [600] + behind(128, range(1, 10)) + [60, 90], [1] * 17, 8, 2, 128, 16),
    "many small groups": ([(2, 256 + 16 * i) for i in range(30)],
                          [256 + 16 * (i // 2) + 1 + i for i in range(60)], [1] * 60, 8, 2, 64, 16),
    "one large group among small ones": ([(1, 256), (60, 384), (1, 128), (1, 130)],
                                         [300] + behind(384, range(1, 61)) + [150, 190], [1] * 63, 8, 2, 128, 16),
    "sequences of no group": ([(3, 256)], [300, 257, 400, 30, 700], [1] * 5, 8, 2, 128, 16),
    "chunks": ([(6, 500)], behind(500, [40, 64, 1, 33, 7, 300], 32), [40, 64, 1, 20, 7, 150], 8, 2, 128, 32),
    "chunks, d 64": ([(6, 500)], behind(500, [40, 64, 1, 33, 7, 300], 32), [40, 64, 1, 20, 7, 150], 6, 6, 64, 32),
    "chunks over a long prefix": ([(12, 4000)], behind(4000, [9 * i + 9 for i in range(12)], 128),
                                  [9 * i + 9 for i in range(12)], 16, 4, 128, 128),
    "chunks of groups": ([(2, 300), (3, 1000)], behind(300, [40, 3]) + behind(1000, [70, 5, 1]), [30, 3, 70, 5, 1],
                         14, 2, 128, 16),
    "full query tiles": ([(3, 500)], behind(500, [200, 150, 150], 32), [200, 130, 100], 8, 2, 128, 32),
    "one head for all": ([(30, 700)], behind(700, range(1, 31), 64), [1] * 30, 64, 1, 64, 64),
    "a head for each": ([(30, 700)], behind(700, range(1, 31), 64), [1] * 30, 4, 4, 128, 64),
    "padded with empty sequences": ([(40, 400)], [0, 0] + behind(400, [5, 1, 90]) + [0] * 35, [0, 0, 1, 1, 1] + [0] * 35,
                                    8, 2, 128, 16),
    "a chunk in a padded batch": ([(60, 400)], [0, 0] + behind(400, [50, 1, 90]) + [0] * 55, [0, 0, 45, 1, 1] + [0] * 55,
                                  8, 2, 64, 16),
    "padded groups": ([(3, 256), (2, 0), (4, 128), (1, 0)], [0, 300, 270, 0, 0, 0, 0, 150, 129, 0],
                      [0, 1, 1, 0, 0, 0, 0, 1, 1, 0], 8, 2, 128, 16),
    "cached but idle": ([(5, 256)], [300, 280, 257, 260, 400], [0, 1, 0, 1, 0], 8, 2, 128, 16),
    "large pages": ([(3, 2048)], [2049, 2100, 3000], [1, 20, 1], 8, 4, 128, 1024),
    "group of 33 heads": ([(4, 300)], behind(300, [1, 2, 60, 30], 64), [1, 1, 20, 1], 66, 2, 128, 64),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_prefix(cg, name, wide, causal):
    groups, lens, news, H, Hkv, d, page = CASES[name]
    c, q = made(groups, lens, news, H, Hkv, d, page, 2000 + 7 * len(name), wide, heads_first=len(name) % 3 == 0)
    o, lse = cg.attention_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args, causal=causal)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, causal, d ** -0.5)


@pytest.mark.parametrize("name", ["single tokens", "a long prefix", "chunks over a long prefix", "groups", "chunks, d 64",
                                  "many small groups"])
def test_within_the_librarys_bounds(cg, name):
    groups, lens, news, H, Hkv, d, page = CASES[name]
    c, q = made(groups, lens, news, H, Hkv, d, page, 3000)
    o, lse = cg.attention_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args, causal=True)
    ref = [reference(c, q, b, True, d ** -0.5) for b in range(len(lens)) if news[b]]
    assert_fwd_close(o, torch.cat([r[0] for r in ref]))
    assert_lse_close(lse, torch.cat([r[2] for r in ref], 1))


@pytest.mark.parametrize("new", [0, 8])
def test_no_key_behind_the_prefix(cg, new):
    # without a mask a sequence may have nothing but its prefix
    c, q = made([(3, 256)], [256, 256, 300], [1 + new, 1, 1], 8, 2, 128, 16, 41)
    o, lse = cg.attention_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args, causal=False)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, False, 128 ** -0.5)


@pytest.mark.parametrize("news", [[1, 1, 1], [20, 1, 33]])
@pytest.mark.parametrize("rise", ["prefix", "own"])
def test_large_scores_on_either_side(cg, news, rise):
    # scores of hundreds before or behind the prefix's end: one part's weight vanishes beside the other's
    c = Shared([(3, 512)], [512 + 60, 512 + 90, 512 + 40], news, 1, 128, 64, 43)
    for i, x in enumerate(c.k):
        f = torch.ones(len(x), 1, 1)
        f[slice(0, 512) if rise == "prefix" else slice(512, None)] = 15
        c.k[i] = (x.float() * f).bfloat16()
    for x in c.k[1:]:
        x[:512] = c.k[0][:512]
    c.fill().cuda()
    q = cs.normal((c.total, 2, 128), 44) * 3
    o, lse = cg.attention_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args, causal=True, scale=0.5)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, True, 0.5)


# V's factor in each 32 positions in turn
FACTORS = {"large": [2.0 ** 12], "small": [2.0 ** -12], "tiny": [2.0 ** -100], "huge": [2.0 ** 100], "zeros": [0.0],
           "in turn": [1.0, 2.0 ** 10, 2.0 ** -30, 0.0, 300.0, 2.0 ** -9, 1.0]}


@pytest.mark.parametrize("d,H,Hkv,count", [(128, 16, 4, 40), (64, 16, 2, 20), (128, 8, 4, 3)])
@pytest.mark.parametrize("name", FACTORS)
def test_values_of_every_size(cg, name, d, H, Hkv, count):
    P, page = 1152, 32
    c = Shared([(count, P)], behind(P, [1 + 3 * i for i in range(count)], page), [1] * count, Hkv, d, page, 48)
    f = FACTORS[name]
    for i, x in enumerate(c.v):
        f_at = torch.tensor([f[(j // 32) % len(f)] for j in range(len(x))])[:, None, None]
        c.v[i] = (x.float() * f_at).bfloat16()
    c.fill().cuda()
    q = cs.normal((c.total, H, d), 49)
    o, lse = cg.attention_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args, causal=True)
    assert cg.chain_check()[0] == 0
    check(c, q, o, lse, True, d ** -0.5)
    if f != [0.0]:
        ref = [reference(c, q, b, True, d ** -0.5) for b in range(count)]
        assert_fwd_close(o.float() / max(f), torch.cat([r[0] for r in ref]) / max(f))


@pytest.mark.parametrize("news", [[1, 1, 1], [33, 1, 5]])
def test_strided_tensors_and_rows_behind_the_last_sequence(cg, news):
    H, d = 6, 128
    c = Shared([(3, 256)], [300, 290, 400], news, 2, d, 16, 45, pad_rows=4).fill().cuda()
    qkv = cs.normal((c.total, H + 4, d), 46)
    o = torch.full((c.total, 2 * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, c.total + 3), 9.0, device="cuda")
    ws = torch.full((cg.chain_fwd_paged_prefix_workspace_size(qkv[:, :H], c.kcd),), 255, dtype=torch.uint8, device="cuda")
    ov, lv = o[:, H:], lse[:, :c.total]
    cg.chain_fwd_paged_prefix(qkv.cuda()[:, :H], c.kcd, c.vcd, *c.args, cg.MASK_CAUSAL, 0.3, ov, lv, ws)
    assert cg.chain_check()[0] == 0
    check(c, qkv[:, :H], ov, lv, True, 0.3)
    n = int(c.cu[-1])
    assert bool((o[:, :H] == 7).all()) and bool((o[n:] == 7).all()) and bool((lse[:, n:] == 9).all())


@pytest.mark.parametrize("name", ["a long prefix", "chunks over a long prefix", "one large group among small ones",
                                  "a chunk in a padded batch"])
def test_the_same_bits_eager_and_replayed(cg, name):
    groups, lens, news, H, Hkv, d, page = CASES[name]
    c, q = made(groups, lens, news, H, Hkv, d, page, 47)
    qd = q.cuda()
    ref, rl = cg.attention_fwd_paged_prefix(qd, c.kcd, c.vcd, *c.args, causal=True)
    n = int(c.cu[-1])
    o, lse = torch.empty_like(ref), torch.empty_like(rl)
    ws = torch.empty(cg.chain_fwd_paged_prefix_workspace_size(qd, c.kcd), dtype=torch.uint8, device="cuda")
    call = lambda: cg.chain_fwd_paged_prefix(qd, c.kcd, c.vcd, *c.args, cg.MASK_CAUSAL, d ** -0.5, o, lse, ws)
    for _ in range(20):
        o.zero_()
        call()
        assert torch.equal(o[:n], ref[:n]) and torch.equal(lse[:, :n], rl[:, :n])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for _ in range(3):
        o.zero_()
        g.replay()
        assert torch.equal(o[:n], ref[:n]) and torch.equal(lse[:, :n], rl[:, :n])
    assert cg.chain_check()[0] == 0


def test_new_lengths_between_replays(cg):
    c, q = made([(8, 512)], behind(512, [200] * 8), [1] * 8, 8, 2, 128, 16, 49)
    qd = q.cuda()
    o, lse = torch.empty_like(qd), torch.empty(8, 8, device="cuda")
    ws = torch.empty(cg.chain_fwd_paged_prefix_workspace_size(qd, c.kcd), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cg.chain_fwd_paged_prefix(qd, c.kcd, c.vcd, *c.args, cg.MASK_CAUSAL, 128 ** -0.5, o, lse, ws)
    for P, own in ((512, 150), (300, 1), (0, 90), (500, 31)):
        c.lens = [512 + own + i for i in range(8)]
        c.lensd.copy_(torch.tensor(c.lens, dtype=torch.int32))
        c.glens.fill_(P)
        s = Cache(c.lens, [1] * 8, 2, 128, 16, 50)
        s.k, s.v = ([x[:L] for x, L in zip(t, c.lens)] for t in (c.k, c.v))
        g.replay()
        assert cg.chain_check()[0] == 0
        check(s, q, o, lse, True, 128 ** -0.5)


def test_two_calls_at_once(cg):
    pairs = [made(*CASES[n][:3], *CASES[n][3:], 51 + i) for i, n in enumerate(("a long prefix", "groups"))]
    ws = [torch.empty(cg.chain_fwd_paged_prefix_workspace_size(q, c.kcd), dtype=torch.uint8, device="cuda")
          for c, q in pairs]
    qs = [q.cuda() for _, q in pairs]
    call = lambda i, s: cg.attention_fwd_paged_prefix(qs[i], pairs[i][0].kcd, pairs[i][0].vcd, *pairs[i][0].args,
                                                      causal=True, workspace=ws[i], stream=s)
    ref = [[x.clone() for x in call(i, None)] for i in range(2)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(10):
        for i in range(2):
            outs[i].append(call(i, streams[i]))
    torch.cuda.synchronize()
    assert cg.chain_check()[0] == 0
    for i in range(2):
        for out in outs[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, ref[i]))


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("news", [[1, 1, 1], [20, 1, 30]])
def test_what_is_reported(cg, news, wide):
    c, q = made([(2, 256), (1, 128)], [300, 290, 400], news, 8, 2, 128, 16, 53, wide)
    q = q.cuda()
    run = lambda glens: cg.attention_fwd_paged_prefix(q, c.kcd, c.vcd, *c.args[:3], c.gcu,
                                                      torch.tensor(glens, dtype=torch.int32).cuda(), causal=True)
    ok = run([256, 128])
    assert cg.chain_check()[0] == 0
    n = news[0] + news[1]
    # a prefix that reaches into the new tokens, one past the table's end: the other group is right
    for bad in (290, 300, 512, 10 ** 9, 2 ** 31 - 1):
        o, lse = run([bad, 128])
        assert cg.chain_check()[0] == cg.ERR_ARG and cg.chain_check()[0] == 0
        assert torch.equal(o[n:], ok[0][n:])
    # a negative one counts as none
    o, lse = run([-5, 128])
    assert cg.chain_check()[0] == cg.ERR_ARG
    check(c, q.cpu(), o, lse, True, 128 ** -0.5)
    # a page that is missing counts as zeros
    c.tabled[:2, 3] = -1
    o, lse = run([256, 128])
    assert cg.chain_check()[0] == cg.ERR_ARG
    assert torch.equal(o[n:], ok[0][n:])
    for x in (c.k, c.v):
        x[0][48:64], x[1][48:64] = 0, 0
    check(c, q.cpu(), o, lse, True, 128 ** -0.5)


def test_groups_that_are_not_there(cg):
    # no groups; groups without sequences; sequences before and behind the groups; more groups than sequences
    c, q = made([(3, 256)], [300, 290, 400], [1, 1, 1], 8, 2, 128, 16, 55)
    qd = q.cuda()
    i = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    for gcu, glens in ((i(0), i()), (i(0, 0, 3, 3, 3), i(128, 256, 0, 512)), (i(1, 3), i(256)), (i(0, 2, 9), i(256, 128)),
                       (i(0, 1, 2, 3, 3, 3, 3), i(128, 256, 0, 1, 2, 3))):
        o, lse = cg.attention_fwd_paged_prefix(qd, c.kcd, c.vcd, *c.args[:3], gcu, glens, causal=True)
        assert cg.chain_check()[0] == 0
        check(c, q, o, lse, True, 128 ** -0.5)


def test_nothing_to_do(cg):
    c = Shared([(2, 128)], [150, 140], [0, 0], 2, 64, 16, 57).fill().cuda()
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = cg.attention_fwd_paged_prefix(e, c.kcd, c.vcd, *c.args, causal=True)
    assert o.numel() == 0 and cg.chain_check()[0] == 0
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")  # tokens, but none of them in a sequence
    cg.attention_fwd_paged_prefix(q, c.kcd, c.vcd, *c.args, causal=True)
    assert cg.chain_check()[0] == 0


def test_largest_batch(cg):
    B, P = 8192, 128
    lens = [P + 1 + (13 * i) % 45 for i in range(B)]
    c, q = made([(B // 2, P), (B // 2, P)], lens, [1] * B, 2, 1, 64, 16, 59)
    o, lse = cg.attention_fwd_paged_prefix(q.cuda(), c.kcd, c.vcd, *c.args, causal=True)
    assert cg.chain_check()[0] == 0
    some = list(range(0, B, 37)) + [B - 1]
    s = Cache([lens[i] for i in some], [1] * len(some), 1, 64, 16, 60)
    s.k, s.v = [c.k[i] for i in some], [c.v[i] for i in some]
    check(s, q[some], o[some], lse[:, some], True, 64 ** -0.5)


def test_refusals(cg):
    c, q = made([(2, 128)], [150, 140], [1, 1], 4, 2, 64, 16, 61)
    q = q.cuda()
    with pytest.raises(ValueError):
        cg.attention_fwd_paged_prefix(q, c.kcd, c.vcd, *c.args[:3], c.gcu[:1], c.glens, causal=True)
    with pytest.raises(ValueError):
        cg.attention_fwd_paged_prefix(q, c.kcd, c.vcd, *c.args[:3], c.gcu.cpu(), c.glens, causal=True)
    with pytest.raises(TypeError):
        cg.attention_fwd_paged_prefix(q.half(), c.kcd, c.vcd, *c.args, causal=True)
    with pytest.raises(cg.ChainError):  # the workspace of the call without prefixes
        ws = torch.empty(cg.chain_fwd_paged_workspace_size(q, c.kcd), dtype=torch.uint8, device="cuda")
        cg.attention_fwd_paged_prefix(q, c.kcd, c.vcd, *c.args, causal=True, workspace=ws)
    assert cg.chain_check()[0] == 0
