"""The serving-side operators beside the attention: per-head query/key norm with rotary
embedding (forward, backward), the write of new keys and values into a paged cache, and the
attention of a chunk of new tokens over that cache.

Each case is one call of one operator.  ``run`` computes it in its plain form, or, with
``own`` set, through ``chain_gb300``.
"""
import math
import random

import torch

own = False

EPS = 1e-6
#: limits of a drawn case: padded scores and gathered keys of the plain form (elements), (head, query,
#: key) triples, elements of Q and K
MOST_SCORES, MOST_KEYS, MOST_PAIRS, MOST_ELEMENTS = 2 ** 31, 2 ** 30, 2 ** 31, 2 ** 27 + 2 ** 25


def listed():
    return [
        # one token of one sequence between its projection and its attention: launch latency
        dict(name="rope_1tok", op="rope", tokens=1, H=32, Hkv=8, d=128, rot=128, pairs="half", dtype="bf16", far=131072),
        # the grouped-query training sequence: 32 query heads over 8 key heads, 32768 positions
        dict(name="rope_32k_gqa", op="rope", tokens=32768, H=32, Hkv=8, d=128, rot=128, pairs="half", dtype="bf16", far=32768),
        # a small fp32 model: partial rotation, neighbouring pairs, an odd number of tokens far into a document
        dict(name="rope_f32_odd", op="rope", tokens=3001, H=6, Hkv=3, d=64, rot=32, pairs="neighbour", dtype="f32", far=1 << 20),
        # gradients of the training sequence
        dict(name="rope_bwd_32k_gqa", op="rope_bwd", tokens=32768, H=32, Hkv=8, d=128, rot=128, pairs="half", dtype="bf16", far=32768),
        # gradients of a short odd batch, one key head for all queries
        dict(name="rope_bwd_1111_mqa", op="rope_bwd", tokens=1111, H=16, Hkv=1, d=64, rot=64, pairs="half", dtype="bf16", far=4096),
        # a decoding step's new keys and values: one token for each of 128 sequences
        dict(name="append_128x1", op="append", batch=128, new=1, kv=2048, ragged=True, H=32, Hkv=8, d=128, page=64),
        # prompts: 16 of up to 2048 tokens written at once, small pages
        dict(name="append_prompts", op="append", batch=16, new=2048, kv=4096, ragged=True, H=32, Hkv=8, d=128, page=16),
        # one token over a short cache: latency
        dict(name="paged_1x1_kv100", op="paged", batch=1, new=1, kv=100, ragged=False, H=32, Hkv=8, d=128, page=64, causal=True),
        # one token over the longest cache (131072 positions): one sequence has to fill the card
        dict(name="paged_1x1_kv128k", op="paged", batch=1, new=1, kv=131072, ragged=False, H=32, Hkv=8, d=128, page=64, causal=True),
        # a decoding step: one token of 64 sequences of mixed lengths up to 16384
        dict(name="paged_64x1_kv16k", op="paged", batch=64, new=1, kv=16384, ragged=True, H=32, Hkv=8, d=128, page=64, causal=True),
        # a mixed step: chunks and single tokens of 24 sequences, d = 64, small pages, odd group
        dict(name="paged_mixed_24", op="paged", batch=24, new=300, kv=5000, ragged=True, H=15, Hkv=5, d=64, page=16, causal=True),
        # a prompt's chunk of 2048 tokens at the end of 32768 cached positions
        dict(name="paged_chunk_2k_kv32k", op="paged", batch=1, new=2048, kv=32768, ragged=False, H=32, Hkv=8, d=128, page=128, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rope", "rope_bwd", "append", "paged", "paged"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 5, 8, 16))
    H = Hkv * rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 16))
    if op in ("rope", "rope_bwd"):
        tokens = _log(rng, 1, min(32768, MOST_ELEMENTS // ((H + Hkv) * d)))
        rot = rng.choice((d, d, d // 2, d // 4))
        return dict(op=op, tokens=tokens, H=H, Hkv=Hkv, d=d, rot=rot, pairs=rng.choice(("half", "neighbour")),
                    dtype=rng.choice(("bf16", "bf16", "f32")), far=_log(rng, tokens, 1 << 20))
    batch = _log(rng, 1, 128)
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "append":
        new = rng.choice((1, _log(rng, 1, 2048)))
        most = max(1, MOST_ELEMENTS // (batch * (H + 2 * Hkv) * d))
        new = min(new, most)
        kv = _log(rng, new, max(new, min(16384, MOST_KEYS // (batch * Hkv * d))))
        return dict(op=op, batch=batch, new=new, kv=kv, ragged=rng.random() < 0.7, H=H, Hkv=Hkv, d=d, page=page)
    new = rng.choice((1, 1, _log(rng, 2, 64), _log(rng, 64, 2048)))
    new = max(1, min(new, MOST_SCORES // (batch * H * 64)))
    most = min(131072, MOST_KEYS // (batch * Hkv * d), MOST_SCORES // (batch * H * new))
    kv = _log(rng, min(16, most), most)
    return dict(op=op, batch=batch, new=new, kv=kv, ragged=rng.random() < 0.7, H=H, Hkv=Hkv, d=d, page=page,
                causal=rng.random() < 0.8)


def _lengths(case):
    """(new tokens, cached positions with them) of each sequence.  They belong to the case, so that its work is known."""
    B, new, kv = case["batch"], case["new"], case["kv"]
    if not case["ragged"]:
        return [(new, max(new, kv))] * B if case["op"] == "append" else [(new, kv)] * B
    rng = random.Random("%d %d %d" % (B, new, kv))
    got = []
    for b in range(B):
        n = new if new == 1 or b == 0 else rng.randint(1, new)
        L = kv if b == 0 else rng.randint(max(1, kv // 16), kv)
        got.append((n, max(n, L) if case["op"] == "append" else L))
    return got


def work(case):
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] in ("rope", "rope_bwd"):
        rows, size = case["tokens"] * (H + Hkv), 2 if case["dtype"] == "bf16" else 4
        arrays, flops = (2, 10) if case["op"] == "rope" else (3, 20)
        more = 4 * case["tokens"] + 2 * size * d + 2 * case["rot"] + (0 if case["op"] == "rope" else 8 * d)
        return {"bytes": arrays * rows * d * size + more, "flops": flops * rows * d}
    lens, page = _lengths(case), case["page"]
    total = sum(n for n, _ in lens)
    if case["op"] == "append":
        tables = sum((L - 1) // page - (L - n) // page + 1 for n, L in lens) * 4 + 8 * len(lens) + 4
        return {"bytes": 4 * total * (H + 2 * Hkv) * d + tables + 4 * d + 2 * case["d"], "flops": 10 * total * (H + Hkv) * d}
    seen = 0
    for n, L in lens:  # keys that the chunk's tokens see
        if not case["causal"]:
            seen += n * L
        else:
            first = max(0, n - L)  # tokens that see nothing
            seen += (n - first) * (L - n + first + 1 + L) // 2
    keys = sum(L for _, L in lens)
    tables = sum(-(-L // page) for _, L in lens) * 4 + 8 * len(lens) + 4
    return {"bytes": 4 * total * H * d + 4 * total * H + 4 * keys * Hkv * d + tables, "flops": 4 * seen * H * d}


def _rand(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _norm_inputs(s, gen, case, dtype):
    d = case["d"]
    s["gq"] = (1 + 0.2 * _rand(gen, d, dtype=torch.float32)).to(dtype)
    s["gk"] = (1 + 0.2 * _rand(gen, d, dtype=torch.float32)).to(dtype)
    rot = case.get("rot", d)
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    s["neighbour"] = case.get("pairs", "half") == "neighbour"


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    s = dict(case=dict(case))
    if case["op"] in ("rope", "rope_bwd"):
        T, dtype = case["tokens"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # queries, keys and values come out of one projection
        qkv = _rand(gen, T, H + 2 * Hkv, d, dtype=dtype)
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        start = int(torch.randint(0, max(1, case["far"] - T + 1), (1,), generator=gen, device="cuda"))
        s["positions"] = torch.arange(start, start + T, dtype=torch.int32, device="cuda")
        _norm_inputs(s, gen, case, dtype)
        if case["op"] == "rope_bwd":
            s["dqo"], s["dko"] = _rand(gen, T, H, d, dtype=dtype), _rand(gen, T, Hkv, d, dtype=dtype)
        return s
    lens, page = _lengths(case), case["page"]
    total = sum(n for n, _ in lens)
    need = [-(-L // page) for _, L in lens]
    pool = sum(need) + 7
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32)
    at = torch.cumsum(torch.tensor([0] + need), 0)
    cols = torch.arange(max(need))
    has = cols[None, :] < torch.tensor(need)[:, None]
    table = torch.where(has, at[:-1, None] + cols[None, :], torch.zeros((), dtype=torch.int64)).cuda()
    s["table"] = order[table].contiguous()
    s["cu"] = torch.tensor([0] + [n for n, _ in lens], dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    s["lens"] = torch.tensor([L for _, L in lens], dtype=torch.int32).cuda()
    s["max_new"], s["max_len"] = max(n for n, _ in lens), max(L for _, L in lens)
    s["kc"], s["vc"] = _rand(gen, pool, page, Hkv, d), _rand(gen, pool, page, Hkv, d)
    if case["op"] == "append":
        qkv = _rand(gen, total, H + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        _norm_inputs(s, gen, case, torch.bfloat16)
    else:
        s["q"] = _rand(gen, total, H, d)
        if own:
            import chain_gb300
            # the scratch of the attention, kept by a program that decodes
            s["workspace"] = torch.empty(chain_gb300.chain_fwd_paged_workspace_size(s["q"], s["kc"]),
                                         dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain form
def _rotate(x, cos, sin, neighbour):
    """x [T, heads, d]; cos, sin [T, 1, rot / 2]."""
    r = 2 * cos.shape[-1]
    if neighbour:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
    u, w = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((u, w), -1).flatten(-2) if neighbour else torch.cat((u, w), -1)
    return torch.cat((y, x[..., r:]), -1)


def _angles(positions, inv_freq):
    a = positions.double()[:, None] * inv_freq.double()[None, :]  # far positions lose their angle in 32 bits
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _norm_rope(x, g, cos, sin, neighbour):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _rotate(x * r * g.float(), cos, sin, neighbour)


def _norm_rope_bwd(dy, x, g, cos, sin, neighbour):
    x, g = x.float(), g.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    a = _rotate(dy.float(), cos, -sin, neighbour)
    h = a * g
    dx = r * (h - x * (r * r) * (h * x).mean(-1, keepdim=True))
    return dx, (a * x * r).sum((0, 1))


def _places(s, total):
    """Sequence and cache position of each packed token."""
    at = torch.arange(total, device="cuda")
    b = (at[:, None] >= s["cu"][None, 1:]).sum(1)
    i = at - s["cu"][b]
    return b, i, s["lens"][b] - (s["cu"][b + 1] - s["cu"][b]) + i


def _plain_append(s):
    b, _, pos = _places(s, s["q"].shape[0])
    cos, sin = _angles(pos, s["inv_freq"])
    q = _norm_rope(s["q"], s["gq"], cos, sin, False).to(s["q"].dtype)
    k = _norm_rope(s["k"], s["gk"], cos, sin, False).to(s["k"].dtype)
    page = s["kc"].shape[1]
    p = s["table"][b, pos // page].long()
    s["kc"][p, pos % page] = k
    s["vc"][p, pos % page] = s["v"]
    return q, s["kc"], s["vc"]


def _plain_paged(s):
    q, page = s["q"].float(), s["kc"].shape[1]
    total, H, d = q.shape
    B, Hkv, G = s["lens"].numel(), s["kc"].shape[2], H // s["kc"].shape[2]
    n, L = s["max_new"], s["max_len"]
    b, i, _ = _places(s, total)
    padded = torch.zeros(B, n, H, d, device="cuda")
    padded[b, i] = q
    x = padded.view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    table = s["table"].long()
    there = torch.arange(L, device="cuda")[None, :] < s["lens"][:, None]  # [B, L]
    k = s["kc"][table].view(B, -1, Hkv, d)[:, :L].float()
    v = s["vc"][table].view(B, -1, Hkv, d)[:, :L].float()
    k, v = (t.masked_fill(~there[:, :, None, None], 0).permute(0, 2, 1, 3) for t in (k, v))
    score = torch.matmul(x, k.transpose(2, 3)).mul_(d ** -0.5).view(B, Hkv, G, n, L)
    new = (s["cu"][1:] - s["cu"][:-1])[:, None]
    rows = torch.arange(n, device="cuda")[None, :]
    last = s["lens"][:, None] - new + rows if s["case"]["causal"] else s["lens"][:, None].expand(B, n) - 1
    hidden = torch.arange(L, device="cuda")[None, None, :] > last[:, :, None]
    hidden |= ~there[:, None, :]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top.masked_fill_(top == -math.inf, 0)
    weight = score.sub_(top).exp_()
    mass = weight.sum(-1, keepdim=True)
    o = torch.matmul(weight.view(B, Hkv, G * n, L), v).view(B, Hkv, G, n, d)
    o = torch.where(mass > 0, o / mass, torch.zeros((), device="cuda"))
    lse = (top + mass.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, H, d)[b, i]
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, H)[b, i]
    return o.to(s["q"].dtype), lse.t().contiguous()


def run(s):
    op = s["case"]["op"]
    if own:
        import chain_gb300 as cg
        if op == "rope":
            return cg.qk_norm_rope(s["q"], s["k"], s["gq"], s["gk"], s["inv_freq"], s["positions"], eps=EPS,
                                   interleaved=s["neighbour"])
        if op == "rope_bwd":
            return cg.qk_norm_rope_bwd(s["dqo"], s["dko"], s["q"], s["k"], s["gq"], s["gk"], s["inv_freq"],
                                       s["positions"], eps=EPS, interleaved=s["neighbour"])
        if op == "append":
            q = cg.qk_norm_rope_append(s["q"], s["k"], s["v"], s["gq"], s["gk"], s["inv_freq"], s["kc"], s["vc"],
                                       s["cu"], s["lens"], s["table"], eps=EPS)
            return q, s["kc"], s["vc"]
        return cg.attention_fwd_paged(s["q"], s["kc"], s["vc"], s["cu"], s["lens"], s["table"],
                                      causal=s["case"]["causal"], workspace=s["workspace"])
    if op == "append":
        return _plain_append(s)
    if op == "paged":
        return _plain_paged(s)
    cos, sin = _angles(s["positions"], s["inv_freq"])
    if op == "rope":
        return tuple(_norm_rope(x, g, cos, sin, s["neighbour"]).to(x.dtype)
                     for x, g in ((s["q"], s["gq"]), (s["k"], s["gk"])))
    dq, dgq = _norm_rope_bwd(s["dqo"], s["q"], s["gq"], cos, sin, s["neighbour"])
    dk, dgk = _norm_rope_bwd(s["dko"], s["k"], s["gk"], cos, sin, s["neighbour"])
    return dq.to(s["q"].dtype), dk.to(s["k"].dtype), dgq, dgk


# ------------------------------------------------------- the definition, 64 bits
def _matrix(positions, inv_freq, d, neighbour):
    """Rotation of each token as a [T, d, d] matrix."""
    T, half = positions.numel(), inv_freq.numel()
    angle = positions.double().view(T, 1) * inv_freq.double().view(1, half)
    m = torch.eye(d, dtype=torch.float64, device="cuda").repeat(T, 1, 1)
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if neighbour else (i, i + half)
    m[:, first, first] = torch.cos(angle)
    m[:, second, second] = torch.cos(angle)
    m[:, first, second] = -torch.sin(angle)
    m[:, second, first] = torch.sin(angle)
    return m


def _exact_rope(x, g, positions, inv_freq, neighbour):
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for a in range(0, x.shape[0], 4096):
        part = x[a:a + 4096].double()
        unit = part / torch.sqrt(torch.mean(part ** 2, dim=-1, keepdim=True) + EPS)
        m = _matrix(positions[a:a + 4096], inv_freq, x.shape[2], neighbour)
        out[a:a + 4096] = torch.einsum("tij,thj->thi", m, unit * g.double())
    return out


def _exact_rope_bwd(dy, x, g, positions, inv_freq, neighbour):
    dx = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    dg = torch.zeros(x.shape[2], dtype=torch.float64, device="cuda")
    for a in range(0, x.shape[0], 4096):
        part = x[a:a + 4096].double()
        m = _matrix(positions[a:a + 4096], inv_freq, x.shape[2], neighbour)
        back = torch.einsum("tji,thj->thi", m, dy[a:a + 4096].double())
        size = torch.sqrt(torch.mean(part ** 2, dim=-1, keepdim=True) + EPS)
        dg += torch.einsum("thi,thi->i", back, part / size)
        up = back * g.double()
        along = torch.sum(up * part, dim=-1, keepdim=True) / x.shape[2]
        dx[a:a + 4096] = up / size - part * along / size ** 3
    return dx, dg


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return tuple(_exact_rope(x, g, s["positions"], s["inv_freq"], s["neighbour"])
                     for x, g in ((s["q"], s["gq"]), (s["k"], s["gk"])))
    if case["op"] == "rope_bwd":
        dq, dgq = _exact_rope_bwd(s["dqo"], s["q"], s["gq"], s["positions"], s["inv_freq"], s["neighbour"])
        dk, dgk = _exact_rope_bwd(s["dko"], s["k"], s["gk"], s["positions"], s["inv_freq"], s["neighbour"])
        return dq, dk, dgq, dgk
    lens, page, d = _lengths(case), case["page"], case["d"]
    starts = [sum(n for n, _ in lens[:b]) for b in range(len(lens))]
    if case["op"] == "append":
        kc, vc, q = s["kc"].double(), s["vc"].double(), torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, (n, L) in enumerate(lens):
            rows, pos = slice(starts[b], starts[b] + n), torch.arange(L - n, L, device="cuda")
            q[rows] = _exact_rope(s["q"][rows], s["gq"], pos, s["inv_freq"], False)
            pages, slots = s["table"][b][pos // page].long(), pos % page
            kc[pages, slots] = _exact_rope(s["k"][rows], s["gk"], pos, s["inv_freq"], False)
            vc[pages, slots] = s["v"][rows].double()
        return q, kc, vc
    H, G = case["H"], case["H"] // case["Hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((H, s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, L) in enumerate(lens):
        pages = s["table"][b][:-(-L // page)].long()
        limit = torch.arange(L - n + 1, L + 1, device="cuda") if case["causal"] else torch.full((n,), L, device="cuda")
        blocked = torch.arange(L, device="cuda")[None, :] >= limit[:, None]
        some = (limit > 0).nonzero().view(-1)
        rows = starts[b] + some
        for h in range(H):
            k = s["kc"][pages, :, h // G].reshape(-1, d)[:L].double()
            v = s["vc"][pages, :, h // G].reshape(-1, d)[:L].double()
            z = (s["q"][rows, h].double() @ k.T / math.sqrt(d)).masked_fill(blocked[some], -math.inf)
            lse[h, rows] = torch.logsumexp(z, dim=-1)
            o[rows, h] = torch.softmax(z, dim=-1) @ v
    return o, lse
