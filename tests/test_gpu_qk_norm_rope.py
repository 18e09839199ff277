"""GPU: per-head norm + rotation of queries and keys (chain_qk_norm_rope, its
backward) against the definition in 64 bits.

Tolerances.  Everything before the store is fp32 with fewer than 32 roundings
an element, each at most 2^-24 of the row's largest intermediate value: 2^-19
of it.  A bf16 result adds half a step, 2^-8 of its value.  A weight's gradient sums
N terms in fp32: at most N + 8 roundings of 2^-24 of the sum of their sizes."""
import math

import pytest
import torch

import chain_synth as cs

pytestmark = pytest.mark.gpu

EPS = 1e-6
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def cg():
    import chain_gb300
    chain_gb300.lib()
    return chain_gb300


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()


def rotate(x, pos, w, neighbour, sign=1):
    """x [T, heads, d] in 64 bits, turned by +-pos w."""
    if w is None:
        return x
    a = pos.double()[:, None, None] * w.double()
    c, s = a.cos(), sign * a.sin()
    half = w.numel()
    i = torch.arange(half)
    i, j = (2 * i, 2 * i + 1) if neighbour else (i, i + half)
    y = x.clone()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def forward(x, g, pos, w, neighbour, eps=EPS):
    x, g = x.double(), g.double()
    u = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * g
    return rotate(u, pos, w, neighbour), u.abs().amax(-1, keepdim=True)


def backward(dy, x, g, pos, w, neighbour, eps=EPS):
    """dx, its rows' largest intermediate, dg, the sum of its terms' sizes"""
    dy, x, g = dy.double(), x.double(), g.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    a = rotate(dy, pos, w, neighbour, -1)
    h = a * g
    mean = (h * x).mean(-1, keepdim=True)
    dx = r * (h - x * r * r * mean)
    biggest = r * (h.abs().amax(-1, keepdim=True) + x.abs().amax(-1, keepdim=True) * r * r *
                   (h * x).abs().mean(-1, keepdim=True))
    # a is formed from two products: its own error is 2^-24 of the larger of the pair
    reach = dy.abs().amax(-1, keepdim=True) * (x * r).abs()
    return dx, biggest, (a * x * r).sum((0, 1)), reach.sum((0, 1))


def close(got, ref, row, what):
    err = (got.cpu().double() - ref).abs()
    tol = STEP[got.dtype] * ref.abs() + 2.0 ** -19 * row
    assert bool((err <= tol).all()), f"{what}: {(err / tol.clamp_min(1e-300)).max():.2f} of the tolerance"


# (tokens, H, Hkv, d, rot, neighbour, type): one token, odd counts, one head, every kind of rotation
CASES = [(1, 32, 8, 128, 128, False, "bf16"), (1, 1, 1, 64, 64, True, "f32"), (7, 5, 1, 128, 64, False, "bf16"),
         (33, 3, 3, 64, 16, False, "f32"), (129, 7, 2, 128, 96, True, "bf16"), (300, 12, 4, 64, 32, True, "bf16"),
         (257, 9, 3, 128, 0, False, "f32"), (64, 40, 8, 128, 48, False, "bf16"), (3000, 4, 2, 64, 64, False, "bf16"),
         (5, 64, 64, 128, 112, False, "f32")]


def make(T, H, Hkv, d, rot, dt, seed, wt=None):
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    qkv = cs.normal((T, H + 2 * Hkv, d), seed, dtype=t)
    g = [(1 + 0.3 * cs.normal((d,), seed + k, dtype=torch.float32)).to(wt or t) for k in (1, 2)]
    gen = torch.Generator().manual_seed(seed)
    pos = torch.randint(-1000, 200000, (T,), generator=gen, dtype=torch.int32)
    return qkv, g, freqs(rot) if rot else None, pos


def cuda(x):
    return None if x is None else x.cuda()


@pytest.mark.parametrize("T,H,Hkv,d,rot,neighbour,dt", CASES)
def test_forward_and_backward(cg, T, H, Hkv, d, rot, neighbour, dt):
    qkv, (gq, gk), w, pos = make(T, H, Hkv, d, rot, dt, 100 + T + H)
    qkv_d = qkv.cuda()
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    qd, kd = qkv_d[:, :H], qkv_d[:, H:H + Hkv]  # views of the fused projection
    args = (gq.cuda(), gk.cuda(), cuda(w), pos.cuda())
    qo, ko = cg.qk_norm_rope(qd, kd, *args, eps=EPS, interleaved=neighbour)
    for got, x, g, what in ((qo, q, gq, "Q"), (ko, k, gk, "K")):
        ref, row = forward(x, g, pos, w, neighbour)
        close(got, ref, row, what)
    dqo, dko = (cs.normal(tuple(x.shape), 77 + T + i, dtype=x.dtype) for i, x in enumerate((q, k)))
    dq, dk, dgq, dgk = cg.qk_norm_rope_bwd(dqo.cuda(), dko.cuda(), qd, kd, *args, eps=EPS,
                                           interleaved=neighbour)
    assert torch.equal(qkv_d.cpu(), qkv)  # inputs are left alone
    for got, dg, dy, x, g, what in ((dq, dgq, dqo, q, gq, "dQ"), (dk, dgk, dko, k, gk, "dK")):
        ref, row, rg, size = backward(dy, x, g, pos, w, neighbour)
        close(got, ref, row, what)
        err = (dg.cpu().double() - rg).abs()
        assert dg.dtype == torch.float32
        assert bool((err <= (x.shape[0] * x.shape[1] + 16) * 2.0 ** -24 * size).all()), what + " weight"


def test_gradient_against_differences(cg):
    T, H, d, rot = 3, 2, 64, 32
    qkv, (gq, gk), w, pos = make(T, H, 1, d, rot, "f32", 5)
    q, k = qkv[:, :H].contiguous(), qkv[:, H:H + 1].contiguous()
    dy = cs.normal((T, H, d), 6, dtype=torch.float32)
    dko = torch.zeros_like(k)
    dq, dk, dgq, _ = cg.qk_norm_rope_bwd(dy.cuda(), dko.cuda(), q.cuda(), k.cuda(), gq.cuda(), gk.cuda(),
                                         w.cuda(), pos.cuda(), eps=EPS)
    assert not dk.any()
    loss = lambda x, g: (forward(x, g, pos, w, False)[0] * dy.double()).sum()
    h = 1e-5  # the central difference of a smooth loss: h^2 third derivatives ~ 1e-8, rounding 1e-16 / h ~ 1e-10
    for e in range(0, d, 7):
        for t, hd in ((0, 1), (2, 0)):
            x1, x2 = q.double().clone(), q.double().clone()
            x1[t, hd, e] += h
            x2[t, hd, e] -= h
            num = (loss(x1, gq) - loss(x2, gq)) / (2 * h)
            assert abs(num - dq[t, hd, e].cpu().double()) <= 2e-5 * dq[t, hd].abs().max().cpu()
        g1, g2 = gq.double().clone(), gq.double().clone()
        g1[e] += h
        g2[e] -= h
        num = (loss(q, g1) - loss(q, g2)) / (2 * h)
        assert abs(num - dgq[e].cpu().double()) <= 2e-5 * dgq.abs().max().cpu()


def test_far_positions(cg):
    # all of int32, frequencies up to many turns a position: angles are exact modulo a turn
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 10 ** 9 + 7], dtype=torch.int32)
    w = torch.tensor([1.0, 0.5, 1e-3, 3.0, 1e-9, 100.25, 6.2831855, -0.75] * 4, dtype=torch.float32)
    x = cs.normal((len(pos), 2, 64), 9, dtype=torch.float32)
    g = torch.ones(64)
    qo, ko = cg.qk_norm_rope(x.cuda(), x.cuda(), g.cuda(), g.cuda(), w.cuda(), pos.cuda(), eps=EPS)
    # the reference angle: p w is a product of 31 and 24 bits, not always exact in 64-bit
    # floats; its remainder modulo a turn by integers
    from fractions import Fraction
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    turns = torch.tensor([[float((Fraction(int(p)) * Fraction(float(f)) / (2 * pi)) % 1) for f in w] for p in pos],
                         dtype=torch.float64)
    a = (turns * 2 * math.pi)[:, None, :]
    u = x.double() / (x.double().square().mean(-1, keepdim=True) + EPS).sqrt()
    y = torch.cat((u[..., :32] * a.cos() - u[..., 32:] * a.sin(), u[..., :32] * a.sin() + u[..., 32:] * a.cos()), -1)
    for got in (qo, ko):
        close(got, y, u.abs().amax(-1, keepdim=True), "far positions")


def test_layouts(cg):
    # 4-D [B][n][H][d]; head-major through a transposed view, written head-major; default positions
    B, n, H, Hkv, d = 3, 37, 6, 2, 128
    q, k = cs.normal((B, H, n, d), 20), cs.normal((B, Hkv, n, d), 21)
    g = (1 + 0.1 * cs.normal((d,), 22, dtype=torch.float32)).cuda()  # f32 weights with bf16 heads
    w = freqs(d).cuda()
    qd, kd = q.cuda(), k.cuda()
    qo, ko = torch.empty_like(qd), torch.empty_like(kd)
    tr = lambda x: x.transpose(1, 2)
    cg.chain_qk_norm_rope(tr(qd), tr(kd), g, g, w, None, EPS, cg.PAIRS_HALF, tr(qo), tr(ko))
    pos = torch.arange(n, dtype=torch.int32).repeat(B)
    for got, x in ((qo, q), (ko, k)):
        flat = tr(x).reshape(B * n, -1, d)
        ref, row = forward(flat, g.cpu(), pos, w.cpu(), False)
        close(tr(got).reshape(B * n, -1, d), ref, row, "head-major")
    # packed and 4-D calls agree, and so does a call in place
    q3, k3 = tr(qd).reshape(B * n, H, d).clone(), tr(kd).reshape(B * n, Hkv, d).clone()
    cg.chain_qk_norm_rope(q3, k3, g, g, w, pos.cuda(), EPS, cg.PAIRS_HALF, q3, k3)
    assert torch.equal(q3, tr(qo).reshape(B * n, H, d)) and torch.equal(k3, tr(ko).reshape(B * n, Hkv, d))
    # the backward in place: over the incoming gradient
    dy, dk = cs.normal((B * n, H, d), 23).cuda(), cs.normal((B * n, Hkv, d), 24).cuda()
    x3, y3 = tr(qd).reshape(B * n, H, d).contiguous(), tr(kd).reshape(B * n, Hkv, d).contiguous()
    ref = cg.qk_norm_rope_bwd(dy, dk, x3, y3, g, g, w, pos.cuda(), eps=EPS)
    ws = torch.empty(cg.chain_qk_norm_rope_bwd_workspace_size(x3), dtype=torch.uint8, device="cuda")
    dg = torch.empty(2, d, device="cuda")
    cg.chain_qk_norm_rope_bwd(dy, dk, x3, y3, g, g, w, pos.cuda(), EPS, 0, dy, dk, dg[0], dg[1], ws)
    for a, b in zip((dy, dk, dg[0], dg[1]), ref):
        assert torch.equal(a, b)  # the same bits twice, too


def test_values_that_are_not_finite_stay_in_their_rows(cg):
    x = cs.normal((4, 2, 64), 30)
    x[1, 0, 3], x[2, 1, 5] = float("nan"), float("inf")
    x[3, 0] = 0
    g = torch.ones(64).cuda()
    qo, _ = cg.qk_norm_rope(x.cuda(), x.cuda(), g, g, freqs(64).cuda(), None, eps=EPS)
    bad = ~torch.isfinite(qo.float()).all(-1).cpu()
    want = torch.zeros(4, 2, dtype=torch.bool)
    want[1, 0] = want[2, 1] = True
    assert torch.equal(bad, want)
    assert not qo[3, 0].any()


def test_no_tokens(cg):
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    g, w = torch.ones(64, device="cuda"), freqs(64).cuda()
    qo, ko = cg.qk_norm_rope(e, e, g, g, w)
    assert qo.shape == e.shape
    out = cg.qk_norm_rope_bwd(e, e, e, e, g, g, w)
    assert not out[2].any() and not out[3].any()


def test_refusals(cg):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    g, w = torch.ones(64, device="cuda"), freqs(64).cuda()
    with pytest.raises(TypeError):
        cg.qk_norm_rope(q.half(), q.half(), g, g, w)
    with pytest.raises(ValueError):
        cg.qk_norm_rope(q.cpu(), q, g, g, w)
    with pytest.raises(ValueError):
        cg.qk_norm_rope(q, q, g, g, w, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        cg.qk_norm_rope(q, q, g, g, w, torch.zeros(4, dtype=torch.int64, device="cuda"))
    for bad in (dict(eps=0.0), dict(eps=float("nan"))):
        with pytest.raises(cg.ChainError):
            cg.qk_norm_rope(q, q, g, g, w, None, **bad)
    with pytest.raises(cg.ChainError):
        cg.qk_norm_rope(q, q, g, g, freqs(72)[:36].cuda())   # more than d
    with pytest.raises(cg.ChainError):
        cg.qk_norm_rope(q, q.float(), g, g, w)               # two types
    with pytest.raises(cg.ChainError):
        cg.qk_norm_rope(q[..., :48], q[..., :48], g, g, w)   # head dimension


def test_other_stream(cg):
    q, k = cs.normal((50, 8, 128), 40).cuda(), cs.normal((50, 2, 128), 41).cuda()
    g, w = torch.ones(128, device="cuda"), freqs(128).cuda()
    ref = cg.qk_norm_rope(q, k, g, g, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = [torch.zeros_like(q), torch.zeros_like(k)]
    s.wait_stream(torch.cuda.current_stream())
    cg.chain_qk_norm_rope(q, k, g, g, w, None, EPS, 0, *out, stream=s)
    s.synchronize()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
