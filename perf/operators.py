"""What the verification side of a draft step costs: attention of drafted blocks over a paged cache
with a shared prefix, the cache's page operations, and the verification of the drafts.

``run`` computes each case in its plain form (elementary torch operations); with ``own`` it makes
the calls that a user makes of ``jacobi_block_refiner_amd.xpress``. Sizes follow the synthetic
workloads of this repository: blocks of 16 slots, 1, 32 and 256 requests, 151936 ids, hidden sizes
4096 and 5120 (32 and 40 heads of 128).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # attend: B query tokens for each of N requests over `shared` common positions and up to
        # `own_max` of their own (ragged; the block's own tokens among them).
        # One request, one block, a short conversation: the smallest call, latency alone.
        dict(name="attend_single", op="attend", N=1, B=16, Hkv=8, G=4, D=128, page=64, shared=0,
             own_max=1000, dtype="bf16", empty=0),
        # Plain decoding (one token a request) behind a system prompt.
        dict(name="attend_decode32", op="attend", N=32, B=1, Hkv=8, G=4, D=128, page=64,
             shared=4096, own_max=1024, dtype="bf16", empty=0),
        # Odd everything: 5 requests, 7 slots, groups of 3 heads of 64, a prefix that ends inside
        # a page of 16, one request of no tokens (a padded batch).
        dict(name="attend_odd", op="attend", N=5, B=7, Hkv=4, G=3, D=64, page=16, shared=777,
             own_max=333, dtype="f16", empty=1),
        # The 32-block workload scored behind a long prompt; 40 heads in groups of 5.
        dict(name="attend_block32", op="attend", N=32, B=16, Hkv=8, G=5, D=128, page=64,
             shared=8192, own_max=700, dtype="bf16", empty=0),
        # The 256-block workload behind a very long prompt: the largest, bound by the matrix core.
        dict(name="attend_block256", op="attend", N=256, B=16, Hkv=8, G=5, D=128, page=64,
             shared=16384, own_max=512, dtype="bf16", empty=0),
        # verify: the target's logits of N blocks of B rows against the drafts.
        # A single request, sampling, a draft that is a greedy choice (no draft probabilities).
        dict(name="verify_single", op="verify", N=1, B=16, V=151936, dtype="bf16", q="none",
             temps="sample", ragged=0),
        # 32 requests whose drafts were sampled from probabilities that are given.
        dict(name="verify_batch32_q", op="verify", N=32, B=16, V=151936, dtype="bf16", q="bf16",
             temps="sample", ragged=0),
        # The 256-block workload, some requests greedy and some sampling, ragged draft lengths.
        dict(name="verify_batch256", op="verify", N=256, B=16, V=151936, dtype="bf16", q="none",
             temps="mixed", ragged=1),
        # turn: the page work of one turn: rows are forked, all are extended by a block (copies
        # of shared last pages), the block's K/V is written, what was refused is given back.
        # Four samples of one prompt, small pages.
        dict(name="turn_best_of_4", op="turn", rows=4, forks=3, B=16, layers=4, Hkv=8, D=128,
             page=16, n_pages=256, shared=512, own_max=200, dtype="bf16"),
        # 32 rows behind one prompt, a few of them forked this turn.
        dict(name="turn_batch32", op="turn", rows=32, forks=6, B=16, layers=4, Hkv=8, D=128,
             page=64, n_pages=768, shared=8192, own_max=700, dtype="bf16"),
        # compact: a pool in use at random places moves its live pages to the front.
        # A small pool of small pages: a tiny head.
        dict(name="compact_small", op="compact", rows=16, layers=2, Hkv=2, D=64, page=16,
             n_pages=300, live=0.4, dtype="f16"),
        # A pool of 2048 pages of 1 MiB, half of them live.
        dict(name="compact_large", op="compact", rows=256, layers=4, Hkv=8, D=128, page=64,
             n_pages=2048, live=0.5, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "verify", "verify", "turn", "compact"])
    most = {c["name"]: work(c) for c in listed()}
    if op == "attend":
        while True:
            c = dict(op=op, N=_log(rng, 1, 256), B=rng.choice([1, 1, 2, 4, 5, 8, 13, 16, 16]),
                     Hkv=rng.choice([1, 2, 4, 8, 8]), G=rng.choice([1, 2, 3, 4, 5, 6, 7, 8]),
                     D=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]),
                     shared=rng.choice([0, _log(rng, 1, 16384), _log(rng, 256, 16384)]),
                     own_max=_log(rng, 16, 1500), dtype=rng.choice(["bf16", "bf16", "f16"]),
                     empty=rng.choice([0, 0, 1]))
            # as many scores and products as the largest listed case at most
            if work(c)["flops"] <= most["attend_block256"]["flops"] * min(1, c["D"] / 128):
                return c
    if op == "verify":
        while True:
            c = dict(op=op, N=_log(rng, 1, 256), B=rng.randint(2, 16),
                     V=rng.choice([151936, _log(rng, 1000, 151936)]),
                     dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                     q=rng.choice(["none", "none", "bf16", "f16", "f32"]),
                     temps=rng.choice(["sample", "sample", "greedy", "mixed"]),
                     ragged=rng.choice([0, 1]))
            if work(c)["bytes"] <= most["verify_batch256"]["bytes"]:
                return c
    if op == "turn":
        rows = _log(rng, 2, 64)
        page = rng.choice([16, 32, 64])
        own_max, shared = _log(rng, 16, 700), rng.choice([0, _log(rng, 16, 8192)])
        c = dict(op=op, rows=rows, forks=rng.randint(0, rows // 2), B=rng.randint(1, 16),
                 layers=rng.choice([1, 2, 4]), Hkv=rng.choice([1, 2, 4]), D=rng.choice([64, 128]),
                 page=page, n_pages=0, shared=shared, own_max=own_max,
                 dtype=rng.choice(["bf16", "f16"]))
        c["n_pages"] = shared // page + rows * (-(-(own_max + 16) // page) + 3) + rng.randint(0, 99)
        return c
    return dict(op=op, rows=_log(rng, 4, 256), layers=rng.choice([1, 2, 4]),
                Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=rng.choice([16, 32, 64]),
                n_pages=_log(rng, 64, 2048), live=rng.choice([0.1, 0.3, 0.5, 0.8, 0.95]),
                dtype=rng.choice(["bf16", "f16"]))


# --------------------------------------------------------------------------------------- inputs
def _cpu(seed):
    return torch.Generator().manual_seed(seed)


def _gpu(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pool(case, n_pages, layers, seed):
    shape = (layers, n_pages, case["Hkv"], case["page"], case["D"])
    g, dt = _gpu(seed), DTYPES[case["dtype"]]
    return (torch.randn(shape, generator=g, device="cuda", dtype=dt),
            torch.randn(shape, generator=g, device="cuda", dtype=dt))


def _tables(lengths, shared, page, n_pages, rows, width, g):
    """Page tables of rows whose first shared//page pages are the same, on pages drawn at random.
    Row n holds lengths[n] tokens (0: no pages). Returns table, ref (CPU, int32)."""
    perm = torch.randperm(n_pages, generator=g, dtype=torch.int64)
    first = shared // page
    table = torch.full((rows, width), -1, dtype=torch.int64)
    used = first
    for n in range(rows):
        need = -(-int(lengths[n]) // page)
        common = min(first, need)
        table[n, :common] = perm[:common]
        table[n, common:need] = perm[used:used + need - common]
        used += need - common
    assert used <= n_pages
    ref = torch.bincount(table[table >= 0], minlength=n_pages)
    return table.to(torch.int32), ref.to(torch.int32)


def _meta(ref, length, table):
    """ref, length and table as views of one int32 buffer on the GPU, and the buffer."""
    parts = [ref, length, table.reshape(-1)]
    sizes = [-(-p.numel() // 4) * 4 for p in parts]
    flat = torch.zeros(sum(sizes), dtype=torch.int32)
    views, at = [], 0
    for p, s in zip(parts, sizes):
        flat[at:at + p.numel()] = p
        views.append((at, p.numel()))
        at += s
    flat = flat.cuda()
    (a, n), (b, m), (c, k) = views
    return flat, flat[a:a + n], flat[b:b + m], flat[c:c + k].view(table.shape)


def prepare(case, seed):
    g, op = _cpu(seed), case["op"]
    if op == "attend":
        N, B, Hkv, G, D, page = (case[k] for k in ("N", "B", "Hkv", "G", "D", "page"))
        shared, own_max = case["shared"], case["own_max"]
        # every request holds the prefix and its own tokens, the block of B among them
        lengths = shared + B + (torch.rand(N, generator=g) * max(own_max - B, 1)).long()
        lengths[0] = shared + max(own_max, B)
        if case["empty"] and N > 1:
            lengths[1 + int(torch.randint(N - 1, (1,), generator=g))] = 0
        width = -(-int(lengths.max()) // page) + 1
        n_pages = shared // page + N * (-(-max(own_max, B) // page) + 1)
        table, ref = _tables(lengths, shared, page, n_pages, N, width, g)
        k, v = _pool(case, n_pages, 1, seed)
        # the rows' common tokens past the last whole shared page are the same values too
        first, rest = shared // page, shared % page
        if rest:
            rows = [n for n in range(N) if int(lengths[n]) > first * page]
            to = table[rows, first].long().cuda()
            for pool in (k, v):
                pool[0, to, :, :rest] = pool[0, to[0], :, :rest].clone()
        # q is the first part of a fused projection's output
        qkv = torch.randn(N * B, (G + 2) * Hkv * D, generator=_gpu(seed + 1), device="cuda",
                          dtype=DTYPES[case["dtype"]])
        return dict(case=case, k=k, v=v, table=table.cuda(), length=lengths.to(torch.int32).cuda(),
                    ref=ref.cuda(), q=qkv[:, :G * Hkv * D], lengths=lengths.tolist())
    if op == "verify":
        N, B, V = case["N"], case["B"], case["V"]
        gg = _gpu(seed)
        logits = torch.randn(N * B, V, generator=gg, device="cuda", dtype=torch.float32).mul_(2)
        blk = torch.randint(V, (N, B), generator=g).cuda()
        # the target mostly agrees with the draft: its logit is near the rest's log-sum-exp
        row = torch.arange(N * B, device="cuda").view(N, B)[:, :-1].reshape(-1)
        mark = math.log(V) + 3.0 + 1.5 * torch.randn(len(row), generator=g)
        logits[row, blk[:, 1:].reshape(-1)] = mark.cuda()
        q = None
        if case["q"] != "none":
            noisy = logits.view(N, B, V)[:, :-1].reshape(-1, V)
            noisy = noisy + 0.5 * torch.randn(noisy.shape, generator=gg, device="cuda")
            q = torch.softmax(noisy, -1).to(DTYPES[case["q"]])
        logits = logits.to(DTYPES[case["dtype"]])
        kind = torch.randint(3, (N,), generator=g)
        temps = {"greedy": torch.zeros(N), "sample": 0.6 + 0.2 * kind,
                 "mixed": torch.where(kind == 0, torch.zeros(N), 0.5 + 0.25 * kind)}
        draft = torch.randint(0, B, (N,), generator=g) if case["ragged"] else torch.full((N,), B - 1)
        return dict(case=case, logits=logits, blk=blk, q=q, u=torch.rand(N, B, generator=g).cuda(),
                    temperature=temps[case["temps"]].float().cuda(),
                    draft_len=draft.to(torch.int32).cuda())
    if op == "turn":
        rows, forks, B, page = (case[k] for k in ("rows", "forks", "B", "page"))
        lengths = case["shared"] + 1 + (torch.rand(rows, generator=g) * case["own_max"]).long()
        lengths[rows - forks:] = case["shared"] // 2  # finished rows, forked over this turn
        width = -(-(case["shared"] + case["own_max"] + 1 + B) // page) + 1
        table, ref = _tables(lengths, case["shared"], page, case["n_pages"], rows, width, g)
        flat, ref, length, table = _meta(ref, lengths.to(torch.int32), table)
        k, v = _pool(case, case["n_pages"], case["layers"], seed)
        src = torch.randint(max(rows - forks, 1), (forks,), generator=g, dtype=torch.int32)
        dst = torch.arange(rows - forks, rows, dtype=torch.int32)
        new = torch.randn(case["layers"], rows * B, 2 * case["Hkv"] * case["D"], device="cuda",
                          generator=_gpu(seed + 1), dtype=DTYPES[case["dtype"]])
        return dict(case=case, k=k, v=v, now=flat.clone(), flat=flat, ref=ref, length=length,
                    table=table, src=src.cuda(), dst=dst.cuda(), new=new,
                    drop=torch.randint(B, (rows,), generator=g).to(torch.int32).cuda())
    rows, page, n_pages = case["rows"], case["page"], case["n_pages"]
    live = max(1, int(n_pages * case["live"]))
    width = 4 * -(-live // rows) + 8
    each = torch.bincount(torch.randint(rows, (live,), generator=g), minlength=rows)
    each = each.clamp(max=width)
    lengths = (each * page - (torch.rand(rows, generator=g) * page).long()).clamp(min=0)
    lengths = torch.where(each > 0, lengths, 0)
    table, ref = _tables(lengths, 0, page, n_pages, rows, width, g)
    flat, ref, length, table = _meta(ref, lengths.to(torch.int32), table)
    k, v = _pool(case, n_pages, case["layers"], seed)
    return dict(case=case, k=k, v=v, now=flat.clone(), flat=flat, ref=ref, length=length,
                table=table, live=torch.zeros(1, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------------------- plain forms
def _gather(pool, table, lo, hi):
    """Tokens lo..hi-1 of every row of `table` from one layer's pages: [rows, Hkv, hi-lo, D], fp32."""
    page = pool.shape[2]
    pos = torch.arange(lo, hi, device=pool.device)
    ids = table[:, pos // page].long().clamp(min=0)
    return pool[ids, :, pos % page].float().transpose(1, 2)


def _attend(s):
    case = s["case"]
    N, B, Hkv, G, D, shared = (case[k] for k in ("N", "B", "Hkv", "G", "D", "shared"))
    own_len = max(s["lengths"]) - shared
    q = s["q"].float().view(N, B, Hkv, G, D).permute(0, 2, 1, 3, 4) * D ** -0.5
    last = s["length"].long()[:, None] - B + torch.arange(B, device="cuda")  # [N, B]
    last = last[:, None, :, None, None]
    parts = []
    own_k = _gather(s["k"][0], s["table"], shared, shared + own_len)
    own_v = _gather(s["v"][0], s["table"], shared, shared + own_len)
    if shared:
        pre_k = _gather(s["k"][0], s["table"][:1], 0, shared)[0]  # [Hkv, shared, D]
        pre_v = _gather(s["v"][0], s["table"][:1], 0, shared)[0]
        rows = q.permute(1, 0, 2, 3, 4).reshape(Hkv, N * B * G, D)
        score = (rows @ pre_k.transpose(1, 2).contiguous()).view(Hkv, N, B, G, shared)
        parts.append(score.transpose(0, 1))
    own_score = q.reshape(N, Hkv, B * G, D) @ own_k.transpose(2, 3).contiguous()
    parts.append(own_score.view(N, Hkv, B, G, own_len))
    score = torch.cat(parts, -1)
    pos = torch.arange(shared + own_len, device="cuda")
    score.masked_fill_(pos > last, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    weight = (score - top).exp_()
    total = weight.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    lse = torch.where(total.squeeze(-1) > 0, lse, -math.inf)
    out = (weight[..., shared:].reshape(N, Hkv, B * G, own_len) @ own_v).view(N, Hkv, B, G, D)
    if shared:
        rows = weight[..., :shared].transpose(0, 1).reshape(Hkv, N * B * G, shared)
        out = out + (rows @ pre_v).view(Hkv, N, B, G, D).transpose(0, 1)
    out = torch.where(total > 0, out / total, 0.0)
    out = out.permute(0, 2, 1, 3, 4).reshape(N * B, Hkv * G * D)
    return dict(out=out.to(s["q"].dtype), lse=lse.permute(0, 2, 1, 3).reshape(N * B, Hkv * G))


def _verify(s):
    """Draft slot i+1 stands while u[i] q(d) < p(d); then a token is drawn from what is left."""
    case = s["case"]
    N, B, V = case["N"], case["B"], case["V"]
    x = s["logits"]
    temp = s["temperature"].double()
    greedy = temp == 0
    inv = torch.where(greedy, 1.0, 1.0 / torch.where(greedy, 1.0, temp))
    top, best = x.max(-1)  # the lowest id among equal ones
    total = ((x.float() - top.float()[:, None]) * inv.float().repeat_interleave(B)[:, None]).exp()
    total = total.sum(-1, dtype=torch.float64).view(N, B)
    top, best = top.double().view(N, B), best.view(N, B)
    draft = s["blk"][:, 1:]
    at = x.view(N, B, V)[:, :-1].gather(2, draft[..., None]).squeeze(-1).double()
    weight = ((at - top[:, :-1]) * inv[:, None]).exp()
    given = 1.0
    if s["q"] is not None:
        given = s["q"].view(N, B - 1, V).gather(2, draft[..., None]).squeeze(-1).double()
    ok = s["u"][:, :-1].double() * given * total[:, :-1] < weight
    ok = torch.where(greedy[:, None], draft == best[:, :-1], ok)
    slot = torch.arange(B - 1, device="cuda")
    limit = s["draft_len"].long()
    ok &= slot < limit[:, None]
    accepted = ok.long().cumprod(1).sum(1)
    n = torch.arange(N, device="cuda")
    # the row where the next token is drawn, in 64 bits: a draw's border lies between two ids
    row = x.view(N, B, V)[n, accepted].double()
    mass = ((row - top[n, accepted][:, None]) * inv[:, None]).exp()
    refused = accepted < limit
    if s["q"] is None:
        tried = draft[n, accepted.clamp(max=B - 2)]
        left = mass.clone()
        left[n, tried] = 0
    else:
        gone = s["q"].view(N, B - 1, V)[n, accepted.clamp(max=B - 2)].double()
        left = (mass / mass.sum(1, keepdim=True) - gone).clamp(min=0)
    left = torch.where((refused & (left.sum(1) > 0))[:, None], left, mass)
    run = left.cumsum(1)
    goal = s["u"][:, -1].double() * run[:, -1]
    token = (run <= goal[:, None]).sum(1).clamp(max=V - 1)
    token = torch.where(greedy, best[n, accepted], token)
    pos = torch.arange(B, device="cuda")
    out = torch.where(pos < accepted[:, None], torch.cat([draft, draft[:, :1]], 1), -1)
    out[n, accepted] = token
    return dict(out=out, accepted=accepted.int(), drop=(B - 1 - accepted).int())


def _held(table, length, page):
    """Which entries of a table belong to its rows' tokens."""
    pages = (length.long() + page - 1) // page
    return torch.arange(table.shape[1], device=table.device) < pages[:, None]


def _turn(s):
    case = s["case"]
    rows, B, page = case["rows"], case["B"], case["page"]
    ref, length, table, k, v = s["ref"], s["length"], s["table"], s["k"], s["v"]
    s["flat"].copy_(s["now"])  # the same tables before every pass
    one = torch.ones((), dtype=torch.int32, device="cuda")
    # fork
    src, dst = s["src"].long(), s["dst"].long()
    old = table[dst][_held(table[dst], length[dst], page)].long()
    ref.index_add_(0, old, -one.expand(old.numel()))
    table[dst], length[dst] = table[src], length[src]
    fresh = table[dst][_held(table[dst], length[dst], page)].long()
    ref.index_add_(0, fresh, one.expand(fresh.numel()))
    # extend: a copy of a shared last page first, then new pages, lowest free ids in order
    before = length.long()
    part = before % page != 0
    at = before // page
    n = torch.arange(rows, device="cuda")
    held = table[n, at].long()
    cow = part & (ref[held.clamp(min=0)] > 1)
    first = torch.where(cow, at, (before + page - 1) // page)
    end = (before + B + page - 1) // page
    col = torch.arange(table.shape[1], device="cuda")
    wanted = (col >= first[:, None]) & (col < end[:, None])
    free = (ref == 0).nonzero().squeeze(1)
    count = int(wanted.sum())
    free = free[:count]
    table[wanted] = free.to(torch.int32)
    ref[free] = 1
    left = held[cow]
    ref.index_add_(0, left, -one.expand(left.numel()))
    to = table[n, at].long()[cow]
    k[:, to] = k[:, left]
    v[:, to] = v[:, left]
    length += B
    # append
    pos = (length.long() - B)[:, None] + torch.arange(B, device="cuda")
    page_of = table.long().gather(1, pos // page).reshape(-1)
    line = (pos % page).reshape(-1)
    width = case["Hkv"] * case["D"]
    shape = (case["layers"], rows * B, case["Hkv"], case["D"])
    for pool, part_ in ((k, s["new"][..., :width]), (v, s["new"][..., width:])):
        pool.transpose(2, 3)[:, page_of, line] = part_.reshape(shape)
    # trim
    after = length - s["drop"]
    gone = _held(table, length, page) & ~_held(table, after, page)
    lost = table[gone].long()
    ref.index_add_(0, lost, -one.expand(lost.numel()))
    table[gone] = -1
    length.copy_(after)
    return dict(ref=ref, length=length, table=table, k=k, v=v)


def _compact(s):
    ref, table, k, v = s["ref"], s["table"], s["k"], s["v"]
    s["flat"].copy_(s["now"])
    alive = ref > 0
    live = alive.sum()
    ids = torch.arange(len(ref), device="cuda")
    frm = (alive & (ids >= live)).nonzero().squeeze(1)
    to = (~alive & (ids < live)).nonzero().squeeze(1)
    k[:, to] = k[:, frm]
    v[:, to] = v[:, frm]
    ref[to] = ref[frm]
    ref[frm] = 0
    place = ids.to(torch.int32)
    place[frm] = to.to(torch.int32)
    held = _held(table, s["length"], s["case"]["page"])
    table.copy_(torch.where(held, place[table.long().clamp(min=0)], table))
    s["live"].copy_(live)
    return dict(ref=ref, table=table, live=s["live"], k=k, v=v)


# ---------------------------------------------------------------------------- the library's calls
def _cache(s):
    from jacobi_block_refiner_amd import xpress
    if "cache" not in s:
        s["cache"] = xpress.Cache(k=s["k"], v=s["v"], table=s["table"], length=s["length"],
                                  ref=s["ref"])
    return xpress, s["cache"]


def _own_attend(s):
    xpress, cache = _cache(s)
    N, B, Hq, D = s["case"]["N"], s["case"]["B"], s["case"]["Hkv"] * s["case"]["G"], s["case"]["D"]
    if "ws" not in s:
        s["ws"] = xpress.attention_workspace(cache, N, B, Hq)
        s["out"] = torch.empty(N * B, Hq * D, dtype=s["q"].dtype, device="cuda")
        s["lse"] = torch.empty(N * B, Hq, device="cuda")
    xpress.block_attention(cache, 0, s["q"], N=N, B=B, Hq=Hq, shared=s["case"]["shared"],
                           out=s["out"], lse=s["lse"], ws=s["ws"])
    return dict(out=s["out"], lse=s["lse"])


def _own_verify(s):
    from jacobi_block_refiner_amd import xpress
    N, B, V = s["case"]["N"], s["case"]["B"], s["case"]["V"]
    if "ws" not in s:
        s["ws"] = xpress.verify_workspace(N, B, V)
        s["out"] = torch.empty(N, B, dtype=torch.int64, device="cuda")
        s["accepted"] = torch.empty(N, dtype=torch.int32, device="cuda")
        s["drop"] = torch.empty(N, dtype=torch.int32, device="cuda")
    xpress.verify_draft(s["logits"], s["blk"], u=s["u"], temperature=s["temperature"],
                        draft_len=s["draft_len"], q=s["q"], out=s["out"], accepted=s["accepted"],
                        drop=s["drop"], ws=s["ws"])
    return dict(out=s["out"], accepted=s["accepted"], drop=s["drop"])


def _own_turn(s):
    xpress, cache = _cache(s)
    case = s["case"]
    width = case["Hkv"] * case["D"]
    if "ws" not in s:
        s["ws"] = xpress.cache_workspace(cache, case["rows"])
        s["lacking"] = torch.empty(1, dtype=torch.int32, device="cuda")
    s["flat"].copy_(s["now"])
    xpress.cache_fork(cache, s["src"], s["dst"])
    xpress.cache_extend(cache, case["B"], N=case["rows"], lacking=s["lacking"], ws=s["ws"])
    for layer in range(case["layers"]):
        new = s["new"][layer]
        xpress.cache_append(cache, layer, new[:, :width], new[:, width:], N=case["rows"],
                            B=case["B"])
    xpress.cache_trim(cache, s["drop"], N=case["rows"])
    return dict(ref=s["ref"], length=s["length"], table=s["table"], k=s["k"], v=s["v"])


def _own_compact(s):
    xpress, cache = _cache(s)
    if "ws" not in s:
        s["ws"] = xpress.cache_workspace(cache, s["case"]["rows"])
    s["flat"].copy_(s["now"])
    xpress.cache_compact(cache, live=s["live"], ws=s["ws"])
    return dict(ref=s["ref"], table=s["table"], live=s["live"], k=s["k"], v=s["v"])


def run(state):
    plain = dict(attend=_attend, verify=_verify, turn=_turn, compact=_compact)
    kernels = dict(attend=_own_attend, verify=_own_verify, turn=_own_turn, compact=_own_compact)
    return (kernels if own else plain)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------- floors
def work(case):
    op = case["op"]
    if op == "attend":
        N, B, Hkv, G, D = (case[k] for k in ("N", "B", "Hkv", "G", "D"))
        mean_own = (max(case["own_max"], B) + B) / 2
        seen = case["shared"] + mean_own - (B - 1) / 2  # of an average query
        keys = case["shared"] + N * mean_own
        return dict(bytes=2 * (2 * keys * Hkv * D + 2 * N * B * Hkv * G * D) + 4 * N * B * Hkv * G,
                    flops=4 * N * B * Hkv * G * D * seen)
    if op == "verify":
        size = dict(none=0, bf16=2, f16=2, f32=4)
        N, B, V = case["N"], case["B"], case["V"]
        # every row of logits; the draft's probabilities only where a draft is refused
        return dict(bytes=N * B * V * size[case["dtype"]] + N * V * size[case["q"]] + 16 * N * B,
                    flops=3 * N * B * V)
    token = 2 * 2 * case["layers"] * case["Hkv"] * case["D"]  # bytes of K and V of one token
    if op == "turn":
        rows, B, page = case["rows"], case["B"], case["page"]
        copied = min(rows, 2 * case["forks"]) * page * (page - 1) / page
        meta = 4 * (case["n_pages"] + rows * (case["shared"] + case["own_max"] + B) / page)
        return dict(bytes=2 * token * (rows * B + copied) + 2 * meta, flops=0)
    live = max(1, int(case["n_pages"] * case["live"]))
    moved = live * (1 - live / case["n_pages"])  # live pages past the front, on average
    return dict(bytes=2 * token * case["page"] * moved + 2 * 4 * (case["n_pages"] + live), flops=0)


# ------------------------------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    """Attention from its definition, a request at a time; the other operators return ids, counts
    and copies, which have no such values."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    N, B, Hkv, G, D, page = (case[k] for k in ("N", "B", "Hkv", "G", "D", "page"))
    out = torch.zeros(N, B, Hkv, G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((N, B, Hkv, G), -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(N, B, Hkv, G, D)
    for n, length in enumerate(s["lengths"]):
        if length == 0:
            continue
        ids = s["table"][n, :-(-length // page)].long()
        k, v = ([pool[0, ids].double().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :length]
                 for pool in (s["k"], s["v"])])
        rows = q[n].permute(1, 0, 2, 3).reshape(Hkv, B * G, D)
        score = torch.matmul(rows, k.transpose(1, 2).contiguous()).view(Hkv, B, G, length)
        score = score / math.sqrt(D)
        hidden = torch.arange(length, device="cuda") > torch.arange(
            length - B, length, device="cuda")[:, None]
        score = score.masked_fill(hidden[None, :, None], -math.inf)
        norm = torch.logsumexp(score, -1)
        p = torch.exp(score - norm[..., None]).view(Hkv, B * G, length)
        out[n] = torch.matmul(p, v).view(Hkv, B, G, D).transpose(0, 1)
        lse[n] = norm.transpose(0, 1)
    return dict(out=out.view(N * B, -1), lse=lse.view(N * B, -1))
