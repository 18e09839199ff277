"""The bookkeeping of a paged K/V cache on the GPU -- pages given to new tokens, with the tables and
slot maps that the cache's writes and its attention take, and pages given back -- and the attention
of a batch whose sequences share a long prefix, which is read and multiplied once for all of them.

Each case is one call of one operator.  ``run`` computes it in its plain form, or, with
``own`` set, through ``chain_gb300``.
"""
import math
import random

import torch

own = False

#: limits of a drawn case: (head, query, key) triples of the shared part, elements of the sequences'
#: own keys (padded), scores of the own part (padded), packed tokens of a plan, entries of a table
MOST_PAIRS, MOST_KEYS, MOST_SCORES, MOST_TOKENS, MOST_ENTRIES = 2 ** 29, 2 ** 26, 2 ** 27, 2 ** 20, 2 ** 20


def listed():
    return [
        # one request's next token: launch latency
        dict(name="plan_1x1", op="plan", batch=1, new=1, kv=100, ragged=False, page=64, pad=0),
        # a decoding step of 512 requests, rows padded to the captured graph's 640
        dict(name="plan_step_512", op="plan", batch=512, new=1, kv=16384, ragged=True, page=64, pad=128),
        # 64 prompts of up to 32768 tokens begun at once, small pages: a million rows
        dict(name="plan_prompts_64", op="plan", batch=64, new=32768, kv=0, ragged=True, page=16, pad=0),
        # rejected tokens of 300 sequences given back after a speculated step
        dict(name="trim_step_300", op="trim", batch=300, kv=5000, ragged=True, page=16, drop="tail"),
        # a batch of 512 that ends: two thirds of the sequences are done, their pages go back
        dict(name="trim_done_512", op="trim", batch=512, kv=32768, ragged=True, page=16, drop="whole"),
        # five answers to a short prompt: latency
        dict(name="prefix_5x1_kv600", op="prefix", groups=1, batch=5, idle=0, new=1, prefix=600, kv=50, ragged=True,
             H=32, Hkv=8, d=128, page=64, causal=True),
        # 64 requests behind one system prompt of 8192 tokens, up to 512 tokens into their own text
        dict(name="prefix_64x1_kv8k", op="prefix", groups=1, batch=64, idle=0, new=1, prefix=8192, kv=512, ragged=True,
             H=32, Hkv=8, d=128, page=64, causal=True),
        # 128 answers about one document of 32768 tokens
        dict(name="prefix_128x1_kv32k", op="prefix", groups=1, batch=128, idle=0, new=1, prefix=32768, kv=1024,
             ragged=True, H=32, Hkv=8, d=128, page=64, causal=True),
        # 16 prompts sampled eight times each, d = 64, an odd group of heads, small pages
        dict(name="prefix_16g_8x1", op="prefix", groups=16, batch=128, idle=0, new=1, prefix=4000, kv=700, ragged=True,
             H=15, Hkv=5, d=64, page=16, causal=True),
        # few sequences behind the longest prefix: the shared keys alone have to fill the card
        dict(name="prefix_6x1_kv128k", op="prefix", groups=1, batch=6, idle=0, new=1, prefix=131072, kv=300, ragged=True,
             H=16, Hkv=2, d=128, page=128, causal=True),
        # 32 questions of up to 64 tokens about one document of 16384 tokens, read in one step
        dict(name="prefix_32x64_kv16k", op="prefix", groups=1, batch=32, idle=0, new=64, prefix=16384, kv=64,
             ragged=True, H=32, Hkv=8, d=128, page=64, causal=True),
    ]


def _log(rng, lo, hi):
    lo, hi = min(lo, hi), max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("plan", "trim", "prefix", "prefix", "prefix"))
    page = rng.choice((16, 32, 64, 128, 256))
    if op != "prefix":
        batch = _log(rng, 1, 2048)
        kv = _log(rng, 1, max(1, min(32768, MOST_ENTRIES * page // batch)))
        if op == "trim":
            return dict(op=op, batch=batch, kv=kv, ragged=rng.random() < 0.8, page=page,
                        drop=rng.choice(("tail", "whole")))
        new = rng.choice((1, _log(rng, 1, max(1, min(32768, MOST_TOKENS // batch)))))
        return dict(op=op, batch=batch, new=new, kv=min(kv, max(1, MOST_ENTRIES * page // batch - new)),
                    ragged=rng.random() < 0.8, page=page, pad=rng.choice((0, _log(rng, 1, 512))))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 5, 8))
    H = Hkv * rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    batch = _log(rng, 1, 256)
    groups = rng.choice((1, 1, _log(rng, 1, min(batch, 32))))
    new = rng.choice((1, 1, _log(rng, 2, 64)))
    new = max(1, min(new, 4096 // batch))
    prefix = _log(rng, 128, min(131072, MOST_PAIRS // (batch * new * H), MOST_KEYS // (groups * Hkv * d)))
    kv = _log(rng, new, min(2048, max(new, min(MOST_KEYS // (batch * Hkv * d), MOST_SCORES // (batch * new * H)))))
    return dict(op=op, groups=groups, batch=batch, idle=rng.choice((0, 0, 3)), new=new, prefix=prefix, kv=kv,
                ragged=rng.random() < 0.8, H=H, Hkv=Hkv, d=d, page=page, causal=rng.random() < 0.8)


# ---------------------------------------------------------------- what a case's sequences are
# Lengths belong to the case, so that its work is known.
def _numbers(case):
    return random.Random("%d %d %d" % (case["batch"], case.get("new", 0), case["kv"]))


def _planned(case):
    """(new tokens, cached positions before them) of each sequence."""
    if not case["ragged"]:
        return [(case["new"], case["kv"])] * case["batch"]
    rng = _numbers(case)
    return [(case["new"] if case["new"] == 1 or b == 0 else rng.randint(0, case["new"]),
             case["kv"] if b == 0 else rng.randint(0, case["kv"])) for b in range(case["batch"])]


def _trimmed(case):
    """(cached positions, positions kept) of each sequence."""
    rng = _numbers(case)
    got = []
    for b in range(case["batch"]):
        L = rng.randint(1, case["kv"]) if case["ragged"] and b else case["kv"]
        if case["drop"] == "whole":
            got.append((L, 0 if rng.random() < 0.67 else L))
        else:
            got.append((L, max(0, L - rng.randint(0, 8))))
    return got


def _groups(case):
    """Of each group its shared positions (whole pages) and the (new tokens, cached positions) of its sequences."""
    rng, page = _numbers(case), case["page"]
    at = [case["batch"] * g // case["groups"] for g in range(case["groups"] + 1)]
    got = []
    for g in range(case["groups"]):
        P = rng.randint(max(1, case["prefix"] // 4), case["prefix"]) if case["ragged"] and g else case["prefix"]
        own_ = []
        for b in range(at[g], at[g + 1]):
            n = case["new"] if case["new"] == 1 or b == 0 or not case["ragged"] else rng.randint(1, case["new"])
            k = rng.randint(1, case["kv"]) if case["ragged"] and b else case["kv"]
            own_.append((n, P + max(n, k)))
        got.append((P // page * page, own_))
    return got


def _pages(n, page):
    return -(-n // page)


def work(case):
    page, B = case["page"], case["batch"]
    if case["op"] == "plan":
        lens = _planned(case)
        rows = sum(n for n, _ in lens)
        given = sum(_pages(L + n, page) - _pages(L, page) for n, L in lens)
        partly = sum(1 for n, L in lens if n and L % page)
        return {"bytes": 16 * B + 12 + 8 * given + 4 * partly + 12 * (rows + case["pad"]), "flops": 2 * rows + 4 * B}
    if case["op"] == "trim":
        back = sum(_pages(L, page) - _pages(k, page) for L, k in _trimmed(case))
        return {"bytes": 12 * B + 8 + 8 * back, "flops": back + 4 * B}
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    total = seen = keys = tables = 0
    for P, seqs in _groups(case):
        keys += P
        tables += 4 * _pages(P, page) + 8
        for n, L in seqs:
            total += n
            keys += L - P
            tables += 4 * (_pages(L, page) - P // page) + 8
            seen += n * L - (n * (n - 1) // 2 if case["causal"] else 0)
    return {"bytes": 4 * total * H * (d + 1) + 4 * keys * Hkv * d + tables, "flops": 4 * seen * H * d}


# ------------------------------------------------------------------------------ inputs
def _ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def _stack(gen, pool):
    return torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)


def _table(order, need, wide):
    """Rows of `wide` entries, row b with need[b] pages from `order` on, the rest never read."""
    need = torch.tensor(need, device="cuda")
    cols = torch.arange(wide, device="cuda")[None, :]
    at = need.cumsum(0) - need
    has = cols < need[:, None]
    index = torch.where(has, at[:, None] + cols, torch.zeros((), dtype=torch.int64, device="cuda"))
    return torch.where(has, order[index], torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    page, s = case["page"], dict(case=dict(case))
    if case["op"] == "plan":
        lens = _planned(case)
        need, most = [_pages(L, page) for _, L in lens], max(_pages(L + n, page) for n, L in lens)
        given = sum(_pages(L + n, page) for n, L in lens) - sum(need)
        order = _stack(gen, sum(need) + given + 5)
        s["table"] = _table(order, need, most + 2)
        # the free pages lie at the bottom of a stack that holds as many as the pool has
        free = order[sum(need):]
        s["free"] = torch.cat((free, torch.full((sum(need),), -1, dtype=torch.int32, device="cuda")))
        s["count"] = _ints([free.numel()])
        s["new"], s["kv"] = _ints([n for n, _ in lens]), _ints([L for _, L in lens])
        s["rows"] = sum(n for n, _ in lens) + case["pad"]
        if own:
            import chain_gb300
            # a program that steps keeps the arrays of its step, and the scratch
            i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
            s["out"] = (i32(case["batch"] + 1), i32(case["batch"]), i32(1), i32(s["rows"]),
                        torch.empty(s["rows"], dtype=torch.int64, device="cuda"))
            s["workspace"] = torch.empty(chain_gb300.chain_page_plan_workspace_size(case["batch"]),
                                         dtype=torch.uint8, device="cuda")
        return s
    if case["op"] == "trim":
        lens = _trimmed(case)
        need = [_pages(L, page) for L, _ in lens]
        order = _stack(gen, sum(need) + 5)
        s["table"] = _table(order, need, max(need) + 2)
        s["free"] = torch.cat((order[sum(need):], torch.full((sum(need),), -1, dtype=torch.int32, device="cuda")))
        s["count"] = _ints([5])
        s["kv"], s["keep"] = _ints([L for L, _ in lens]), _ints([k for _, k in lens])
        s["pool"] = sum(need) + 5
        if own:
            import chain_gb300
            s["out"] = (torch.empty_like(s["kv"]), torch.empty_like(s["count"]))
            s["workspace"] = torch.empty(chain_gb300.chain_page_trim_workspace_size(case["batch"]),
                                         dtype=torch.uint8, device="cuda")
        return s
    groups, idle = _groups(case), case["idle"]
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    seqs = [x for _, own_ in groups for x in own_] + [(0, 0)] * idle
    shared = [P // page for P, _ in groups]
    start = [P for P, own_ in groups for _ in own_] + [0] * idle
    need = [_pages(L, page) - P // page for (_, L), P in zip(seqs, start)]
    pool = sum(shared) + sum(need) + 7
    order = _stack(gen, pool)
    wide = max(_pages(L, page) for _, L in seqs)
    table = torch.full((len(seqs), wide), -1, dtype=torch.int64)
    at, b = 0, 0
    for (_, own_), m in zip(groups, shared):
        for _ in own_:
            table[b, :m] = torch.arange(at, at + m)
            b += 1
        at += m
    for b, (P, m) in enumerate(zip(start, need)):
        table[b, P // page:P // page + m] = torch.arange(at, at + m)
        at += m
    table = table.cuda()
    s["table"] = torch.where(table >= 0, order[table.clamp_min(0)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    s["cu"] = _ints([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32)
    s["lens"] = _ints([L for _, L in seqs])
    s["prefix_cu"] = _ints([0] + [len(own_) for _, own_ in groups]).cumsum(0).to(torch.int32)
    s["prefix_lens"] = _ints([P for P, _ in groups])
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)
    s["kc"], s["vc"] = rand(pool, page, Hkv, d), rand(pool, page, Hkv, d)
    s["q"] = rand(sum(n for n, _ in seqs), H, d)
    s["max_new"], s["max_own"] = max(n for n, _ in seqs), max(L - P for (_, L), P in zip(seqs, start))
    s["start"] = _ints(start)
    if own:
        import chain_gb300
        # the outputs and the scratch of the attention, kept by a program that decodes
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(H, s["q"].shape[0], device="cuda")
        s["workspace"] = torch.empty(chain_gb300.chain_fwd_paged_prefix_workspace_size(s["q"], s["kc"]),
                                     dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------------------------------- plain form
def _plain_plan(s):
    page, new, kv, table = s["case"]["page"], s["new"].long(), s["kv"].long(), s["table"]
    have, want = (kv + page - 1) // page, (kv + new + page - 1) // page
    need = want - have
    before = need.cumsum(0) - need
    cu = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)))
    # pages from the top of the stack, in the order of the sequences
    cols = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (cols >= have[:, None]) & (cols < want[:, None])
    top = s["count"].long() - 1
    index = (top - before[:, None] - cols + have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][index], table))
    at = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(cu[1:], at, right=True)
    inside = b < new.numel()
    b = b.clamp_max(new.numel() - 1)
    pos = kv[b] + at - cu[b]
    pos = torch.where(inside, pos, torch.zeros_like(pos))
    slot = table[b, pos // page].long() * page + pos % page
    none = torch.full_like(pos, -1)
    return (cu.int(), (kv + new).int(), (s["count"] - need.sum()).int(), torch.where(inside, pos, none).int(),
            torch.where(inside, slot, none), table)


def _plain_trim(s):
    page, kv, table, free = s["case"]["page"], s["kv"].long(), s["table"], s["free"]
    left = torch.minimum(kv, s["keep"].long())
    first, last = (left + page - 1) // page, (kv + page - 1) // page
    back = last - first
    before = back.cumsum(0) - back
    cols = torch.arange(table.shape[1], device="cuda")[None, :]
    goes = (cols >= first[:, None]) & (cols < last[:, None])
    place = s["count"].long() + before[:, None] + cols - first[:, None]
    # what stays goes to a place behind the stack
    place = torch.where(goes, place, torch.full_like(place, free.numel()))
    longer = torch.cat((free, free.new_zeros(1)))
    longer[place.flatten()] = table.flatten()
    free.copy_(longer[:-1])
    return left.int(), (s["count"] + back.sum()).int(), free


def _rows(s):
    """Sequence and number in it of each packed token."""
    at = torch.arange(s["q"].shape[0], device="cuda")
    b = (at[:, None] >= s["cu"][None, 1:]).sum(1)
    return b, at - s["cu"][b]


def _scores(x, k, scale):
    return torch.matmul(x, k.transpose(-1, -2)).mul_(scale)


def _weights(score):
    """exp(score - top) in place, top (0 for a row that sees nothing) and the weights' sum."""
    top = score.amax(-1, keepdim=True)
    top.masked_fill_(top == -math.inf, 0)
    weight = score.sub_(top).exp_()
    return weight, top, weight.sum(-1, keepdim=True)


def _plain_prefix(s):
    case, page = s["case"], s["kc"].shape[1]
    q = s["q"].float()
    total, H, d = q.shape
    Hkv, G, scale = case["Hkv"], H // case["Hkv"], d ** -0.5
    B = s["lens"].numel()
    x = q.view(total, Hkv, G, d)
    # the prefix of a group against all rows of its sequences
    po = torch.zeros(total, Hkv, G, d, device="cuda")
    ptop, pmass = (torch.zeros(total, Hkv, G, 1, device="cuda") for _ in range(2))
    at = b = 0
    for P, seqs in _groups(case):
        rows = sum(n for n, _ in seqs)
        if P and rows:
            pages = s["table"][b, :_pages(P, page)].long()
            k, v = (c[pages].view(-1, Hkv, d)[:P].float().transpose(0, 1) for c in (s["kc"], s["vc"]))
            mine = x[at:at + rows].permute(1, 2, 0, 3).reshape(Hkv, G * rows, d)
            weight, top, mass = _weights(_scores(mine, k, scale))
            o = torch.matmul(weight, v)
            back = lambda t: t.view(Hkv, G, rows, -1).permute(2, 0, 1, 3)
            po[at:at + rows], ptop[at:at + rows], pmass[at:at + rows] = back(o), back(top), back(mass)
            del weight
        at += rows
        b += len(seqs)
    # each sequence's own keys, padded
    b, i = _rows(s)
    n, W = s["max_new"], s["max_own"]
    y = torch.zeros(B, n, Hkv, G, d, device="cuda")
    y[b, i] = x
    y = y.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    pos = s["start"].long()[:, None] + torch.arange(W, device="cuda")[None, :]
    there = pos < s["lens"][:, None]
    inside = torch.where(there, pos, torch.zeros_like(pos))
    pages = s["table"].gather(1, inside // page).long().clamp_min(0)
    k, v = (c[pages, inside % page].float().masked_fill(~there[:, :, None, None], 0).transpose(1, 2)
            for c in (s["kc"], s["vc"]))
    score = _scores(y, k, scale).view(B, Hkv, G, n, W)
    new = (s["cu"][1:] - s["cu"][:-1])[:, None]
    last = s["lens"][:, None] - (new - torch.arange(n, device="cuda")[None, :] if case["causal"] else 1)
    hidden = ~there[:, None, :] | (pos[:, None, :] > last.expand(B, n)[:, :, None])
    weight, top, mass = _weights(score.masked_fill_(hidden[:, None, None], -math.inf))
    o = torch.matmul(weight.view(B, Hkv, G * n, W), v).view(B, Hkv, G, n, d)
    so, stop, smass = (t.permute(0, 3, 1, 2, 4)[b, i] for t in (o, top, mass))
    # both parts of a row
    high = torch.maximum(torch.where(pmass > 0, ptop, stop), torch.where(smass > 0, stop, ptop))
    wp, ws = (torch.where(m > 0, (t - high).exp(), torch.zeros_like(m)) for t, m in ((ptop, pmass), (stop, smass)))
    mass = wp * pmass + ws * smass
    o = (wp * po + ws * so) / mass
    return o.reshape(total, H, d).to(s["q"].dtype), (high + mass.log()).reshape(total, H).t().contiguous()


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "trim": _plain_trim, "prefix": _plain_prefix}[op](s)
    import chain_gb300 as cg
    if op == "plan":
        return (*cg.page_plan(s["new"], s["kv"], s["table"], s["free"], s["count"], s["case"]["page"], s["rows"],
                              out=s["out"], workspace=s["workspace"]), s["table"])
    if op == "trim":
        return (*cg.page_trim(s["keep"], s["kv"], s["table"], s["free"], s["count"], s["case"]["page"], s["pool"],
                              out=s["out"], workspace=s["workspace"]), s["free"])
    cg.chain_fwd_paged_prefix(s["q"], s["kc"], s["vc"], s["cu"], s["lens"], s["table"], s["prefix_cu"],
                              s["prefix_lens"], cg.MASK_CAUSAL if s["case"]["causal"] else cg.MASK_NONE,
                              s["q"].shape[2] ** -0.5, s["o"], s["lse"], s["workspace"])
    return s["o"], s["lse"]


# ------------------------------------------------------------- the definition, 64 bits
def _exact_plan(case, s):
    page, table, free = case["page"], s["table"].cpu().long(), s["free"].cpu().tolist()
    cu, kv, count, positions, slots = [0], [], int(s["count"]), [], []
    for b, (n, L) in enumerate(_planned(case)):
        for k in range(_pages(L, page), _pages(L + n, page)):
            count -= 1
            table[b, k] = free[count]
        p = torch.arange(L, L + n)
        positions.append(p)
        slots.append(table[b][p // page] * page + p % page)
        cu.append(cu[-1] + n)
        kv.append(L + n)
    rest = torch.full((case["pad"],), -1, dtype=torch.int64)
    positions, slots = torch.cat(positions + [rest]), torch.cat(slots + [rest])
    return _ints(cu), _ints(kv), _ints([count]), positions.int().cuda(), slots.cuda(), table.int().cuda()


def _exact_trim(case, s):
    page, table, free = case["page"], s["table"].cpu().tolist(), s["free"].cpu().tolist()
    kv, count = [], int(s["count"])
    for b, (L, keep) in enumerate(_trimmed(case)):
        for k in range(_pages(keep, page), _pages(L, page)):
            free[count] = table[b][k]
            count += 1
        kv.append(keep)
    return _ints(kv), _ints([count]), _ints(free)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "prefix":
        return (_exact_plan if case["op"] == "plan" else _exact_trim)(case, s)
    H, Hkv, d, page = case["H"], case["Hkv"], case["d"], case["page"]
    G = H // Hkv
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(H, s["q"].shape[0], dtype=torch.float64, device="cuda")
    at = b = 0
    for _, seqs in _groups(case):
        for n, L in seqs:
            pages = s["table"][b, :_pages(L, page)].long()
            sees = torch.arange(L - n + 1, L + 1, device="cuda") if case["causal"] else torch.full((n,), L, device="cuda")
            blocked = torch.arange(L, device="cuda")[None, :] >= sees[:, None]
            for h in range(Hkv):
                k, v = (c[pages, :, h].reshape(-1, d)[:L].double() for c in (s["kc"], s["vc"]))
                heads = slice(h * G, (h + 1) * G)
                z = torch.einsum("nhd,kd->hnk", s["q"][at:at + n, heads].double(), k) / math.sqrt(d)
                z = z.masked_fill(blocked[None], -math.inf)
                lse[heads, at:at + n] = torch.logsumexp(z, dim=-1)
                o[at:at + n, heads] = torch.einsum("hnk,kd->nhd", torch.softmax(z, dim=-1), v)
            at += n
            b += 1
    return o, lse
