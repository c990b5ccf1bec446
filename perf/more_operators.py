"""What a cache in 4 bits and the report on served tokens cost: K and V quantised as they are written
and read back, attention of blocks over such a cache, and the log probabilities of given tokens with
entropy, rank and top alternatives.

``run`` computes each case in its plain form (elementary torch operations); with ``own`` it makes
the calls that a user makes of ``jacobi_block_refiner_amd.xpress``. Sizes follow the synthetic
workloads of this repository: blocks of 16 slots, 1, 32 and 256 requests, 151936 ids, hidden sizes
4096 and 5120 (32 and 40 heads of 128, 8 of K and V).

A cache in 4 bits holds tiles of 16 tokens of a page and head. A value is one of 0, 0.5, 1, 1.5, 2, 3,
4, 6 (codes 0 to 7; 8 to 15 are their negatives) times 2^(s - 127) with a byte s for 32 channels. A
tile has 8 D bytes of codes, then D/2 of scales. In K token t, channels 2c and 2c + 1 are the low and
high half of byte t D/2 + c, and the scale of group g is byte t D/32 + g. In V channels 32 g + 2 i and
the next of token 4 q + j are byte ((16 q + i) D/32 + g) 4 + j, their scale byte (q D/32 + g) 4 + j.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
RANGE = {"bf16": (-123, 125), "f16": (-23, 13)}  # exponents of a scale


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # store: K and V of the last B tokens of N rows are quantised into one layer, and read back.
        # One block of 16 slots for one request: the smallest call, latency alone.
        dict(name="store_block", op="store", N=1, B=16, Hkv=8, D=128, page=64, before=1000,
             dtype="bf16"),
        # A prompt of one request, rows that begin inside a tile.
        dict(name="store_prompt", op="store", N=1, B=8191, Hkv=8, D=128, page=64, before=37,
             dtype="f16"),
        # read: tokens of a cache as 16-bit values, for a program that moves or inspects them.
        # A few short rows of small heads in small pages.
        dict(name="read_short", op="read", N=4, B=100, Hkv=4, D=64, page=16, before=33, dtype="f16"),
        # Eight rows of 8192 tokens: the whole prefix of a batch that leaves the card.
        dict(name="read_long", op="read", N=8, B=8192, Hkv=8, D=128, page=64, before=0,
             dtype="bf16"),
        # attend: B query tokens for each of N requests over `shared` common positions and up to
        # `own_max` of their own (ragged; the block's own tokens among them).
        # One request decoding, a short conversation.
        dict(name="attend4_single", op="attend", N=1, B=1, Hkv=8, G=4, D=128, page=64, shared=0,
             own_max=1000, dtype="bf16", empty=0),
        # Plain decoding (one token a request) behind a system prompt.
        dict(name="attend4_decode32", op="attend", N=32, B=1, Hkv=8, G=4, D=128, page=64,
             shared=4096, own_max=1024, dtype="bf16", empty=0),
        # Odd everything: 5 requests, 7 slots, groups of 3 heads of 64, a prefix that ends inside
        # a page of 16, one request of no tokens (a padded batch).
        dict(name="attend4_odd", op="attend", N=5, B=7, Hkv=4, G=3, D=64, page=16, shared=777,
             own_max=333, dtype="f16", empty=1),
        # Long contexts of very different lengths, one token each: what 4 bits are for.
        dict(name="attend4_long", op="attend", N=64, B=1, Hkv=8, G=5, D=128, page=64, shared=0,
             own_max=32768, dtype="bf16", empty=0),
        # The 32-block workload scored behind a long prompt: bound by the matrix core.
        dict(name="attend4_block32", op="attend", N=32, B=16, Hkv=8, G=5, D=128, page=64,
             shared=8192, own_max=700, dtype="bf16", empty=0),
        # logprobs: a token a row of logits, at the blocks' temperatures.
        # The token of one request, with 20 alternatives.
        dict(name="logprobs_single", op="logprobs", N=1, B=1, V=151936, top=20, dtype="f32",
             temps="one"),
        # The 32-block workload after its verification: slots without a token among them.
        dict(name="logprobs_batch32", op="logprobs", N=32, B=16, V=151936, top=20, dtype="bf16",
             temps="mixed"),
        # A prompt of 2048 tokens scored, with 5 alternatives each.
        dict(name="logprobs_prompt", op="logprobs", N=1, B=2048, V=151936, top=5, dtype="bf16",
             temps="none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend", "attend", "logprobs", "logprobs"])
    most = {c["name"]: work(c) for c in listed()}
    if op in ("store", "read"):
        cap = most["store_prompt" if op == "store" else "read_long"]["bytes"]
        while True:
            c = dict(op=op, N=_log(rng, 1, 256), B=_log(rng, 1, 8192),
                     Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 128, 256]),
                     page=rng.choice([16, 32, 64, 128]), before=rng.choice([0, _log(rng, 1, 1000)]),
                     dtype=rng.choice(["bf16", "bf16", "f16"]))
            # (the tokens before these are in the pools too)
            if work(c)["bytes"] <= cap and c["N"] * c["before"] <= 32768:
                return c
    if op == "attend":
        while True:
            c = dict(op=op, N=_log(rng, 1, 256),
                     B=rng.choice([1, 1, 1, 2, 4, 5, 8, 13, 16, 16]),
                     Hkv=rng.choice([1, 2, 4, 8, 8]), G=rng.choice([1, 2, 3, 4, 5, 6, 7, 8]),
                     D=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]),
                     shared=rng.choice([0, 0, _log(rng, 1, 8192), _log(rng, 256, 8192)]),
                     own_max=rng.choice([_log(rng, 16, 1500), _log(rng, 16, 32768)]),
                     dtype=rng.choice(["bf16", "bf16", "f16"]), empty=rng.choice([0, 0, 1]))
            w = work(c)
            if (w["flops"] <= most["attend4_block32"]["flops"] * min(1, c["D"] / 128)
                    and w["bytes"] <= most["attend4_long"]["bytes"]
                    and c["N"] * c["own_max"] * c["Hkv"] * c["D"] <= 64 * 32768 * 8 * 128):
                return c
    while True:
        c = dict(op="logprobs", N=_log(rng, 1, 256), B=rng.choice([1, 1, 2, 7, 16, 16]),
                 V=rng.choice([151936, _log(rng, 1000, 151936)]),
                 top=rng.choice([0, 1, 5, 5, 20, 20, rng.randint(2, 64)]),
                 dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                 temps=rng.choice(["none", "one", "mixed"]))
        if work(c)["bytes"] <= most["logprobs_prompt"]["bytes"]:
            return c


# --------------------------------------------------------------------------------------- inputs
def _cpu(seed):
    return torch.Generator().manual_seed(seed)


def _gpu(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantise(x, dtype):
    """Codes (uint8, 0..15) of x [..., D] and exponents (int32) of its groups of 32 channels."""
    lo, hi = RANGE[dtype]
    x = x.float()
    x = torch.where(x.isnan(), 0.0, x).clamp(-3.3e38, 3.3e38)
    groups = x.view(*x.shape[:-1], -1, 32)
    top = groups.abs().amax(-1)
    # the exponent of the largest, one more from 1.75 of its power of two on; less 2, for 4 to 6
    e = ((top.view(torch.int32) + (1 << 21)) >> 23) - 127 - 2
    e = e.clamp(lo, hi)
    y = groups * _pow2(-e)[..., None]
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = code.to(torch.uint8) | (y < 0).to(torch.uint8) << 3
    return code.view(x.shape), e


def _pow2(e):
    """2^e in 32 bits, for exponents of normal numbers."""
    return ((e + 127) << 23).view(torch.float32)


def _bytes(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def _pack(x, dtype, is_v):
    """Tiles of x [..., 16, D]: [..., 17 D / 2] bytes."""
    code, e = _quantise(x, dtype)
    D, lead = x.shape[-1], x.shape[:-2]
    both, scale = _bytes(code), (e + 127).to(torch.uint8)
    if is_v:
        both = both.view(*lead, 4, 4, D // 32, 16).permute(*range(len(lead)), -4, -1, -2, -3)
        scale = scale.view(*lead, 4, 4, D // 32).transpose(-1, -2)
    return torch.cat([both.reshape(*lead, 8 * D), scale.reshape(*lead, D // 2)], -1)


def _pool(case, n_pages, seed, same=None):
    """K and V of one layer: [1, n_pages, Hkv, page / 16, 17 D / 2] bytes each, quantised normal
    values. `same`: (page ids, number of lines) whose first lines are the same values."""
    Hkv, page, D = case["Hkv"], case["page"], case["D"]
    g, dt = _gpu(seed), DTYPES[case["dtype"]]
    pools = []
    step = max(1, (1 << 26) // (Hkv * page * D))
    for is_v in (False, True):
        pool = torch.empty(1, n_pages, Hkv, page // 16, 17 * D // 2, dtype=torch.uint8, device="cuda")
        first = torch.randn(Hkv, page, D, generator=g, device="cuda", dtype=dt)
        for a in range(0, n_pages, step):
            n = min(step, n_pages - a)
            x = torch.randn(n, Hkv, page, D, generator=g, device="cuda", dtype=dt)
            if same is not None:
                to = [p - a for p in same[0] if a <= p < a + n]
                x[to, :, :same[1]] = first[:, :same[1]]
            pool[0, a:a + n] = _pack(x.view(n, Hkv, page // 16, 16, D), case["dtype"], is_v)
        pools.append(pool)
    return pools


def _tables(lengths, shared, page, width, g):
    """Page tables of rows whose first shared//page pages are the same, on pages drawn at random.
    Row n holds lengths[n] tokens (0: no pages). Returns table and ref (CPU, int32)."""
    first = shared // page
    need = [-(-int(n) // page) for n in lengths]
    n_pages = first + sum(max(n - first, 0) for n in need) + 3
    perm = torch.randperm(n_pages, generator=g, dtype=torch.int64)
    table = torch.full((len(need), width), -1, dtype=torch.int64)
    used = first
    for n, k in enumerate(need):
        common = min(first, k)
        table[n, :common] = perm[:common]
        table[n, common:k] = perm[used:used + k - common]
        used += k - common
    ref = torch.bincount(table[table >= 0], minlength=n_pages)
    return table.to(torch.int32), ref.to(torch.int32)


def prepare(case, seed):
    g, op = _cpu(seed), case["op"]
    if op == "logprobs":
        N, B, V = case["N"], case["B"], case["V"]
        logits = torch.randn(N * B, V, generator=_gpu(seed), device="cuda").mul_(2)
        token = torch.randint(V, (N, B), generator=g)
        # most tokens were drawn from their rows: their logits are near the rest's log-sum-exp
        mark = math.log(V) + 1.0 + 1.5 * torch.randn(N * B, generator=g)
        logits[torch.arange(N * B, device="cuda"), token.view(-1).cuda()] = mark.cuda()
        if B == 16:  # blocks after their verification: slots behind the last token hold none
            last = torch.randint(1, B + 1, (N,), generator=g)
            token[torch.arange(B) >= last[:, None]] = -1
        kind = torch.randint(3, (N,), generator=g)
        temps = {"none": None, "one": 0.6 + 0.2 * kind,
                 "mixed": torch.where(kind == 0, torch.zeros(N), 0.5 + 0.25 * kind)}[case["temps"]]
        return dict(case=case, logits=logits.to(DTYPES[case["dtype"]]), token=token.cuda(),
                    temperature=None if temps is None else temps.float().cuda())
    N, B, Hkv, D, page = (case[k] for k in ("N", "B", "Hkv", "D", "page"))
    if op in ("store", "read"):
        shared = 0
        lengths = case["before"] + B - (torch.rand(N, generator=g) * case["before"] * 0.5).long()
    else:
        shared, own_max = case["shared"], case["own_max"]
        # every request holds the prefix and its own tokens, the block of B among them
        lengths = shared + B + (torch.rand(N, generator=g) * max(own_max - B, 1)).long()
        lengths[0] = shared + max(own_max, B)
        if case["empty"] and N > 1:
            lengths[1 + int(torch.randint(N - 1, (1,), generator=g))] = 0
    table, ref = _tables(lengths, shared, page, -(-int(lengths.max()) // page) + 1, g)
    same = None
    if shared % page:  # the rows' common tokens past the last whole shared page
        first = shared // page
        same = ([int(p) for p, n in zip(table[:, first], lengths) if n > first * page], shared % page)
    k, v = _pool(case, len(ref), seed, same)
    s = dict(case=case, k=k, v=v, table=table.cuda(), length=lengths.to(torch.int32).cuda(),
             ref=ref.cuda(), lengths=lengths.tolist())
    # the new values are parts of a fused projection's output
    G = case.get("G", 1)
    if op != "read":
        s["qkv"] = torch.randn(N * B, (G + 2) * Hkv * D, generator=_gpu(seed + 1), device="cuda",
                               dtype=DTYPES[case["dtype"]])
    return s


# --------------------------------------------------------------------------------- plain forms
def _values(tiles, D, is_v):
    """The values of tiles [..., 17 D / 2]: [..., 16, D] in 32 bits."""
    lead = tiles.shape[:-1]
    both, scale = tiles[..., :8 * D], tiles[..., 8 * D:].int()
    if is_v:
        both = both.reshape(*lead, 4, 16, D // 32, 4).permute(*range(len(lead)), -4, -1, -2, -3)
        scale = scale.view(*lead, 4, D // 32, 4).transpose(-1, -2)
    both = both.reshape(*lead, 16, D // 32, 16)
    # the value of every byte's two halves
    level = torch.tensor(LEVELS, device=tiles.device)
    level = torch.cat([level, -level])
    pair = torch.stack([level.repeat(16), level.repeat_interleave(16)], -1)  # [256, 2]
    value = pair[both.int()].view(*lead, 16, D // 32, 32)
    return (value * (scale << 23).view(torch.float32).reshape(*lead, 16, D // 32, 1)).view(*lead, 16, D)


def _gather(pool, table, lo, hi, D, is_v):
    """Tokens lo..hi-1 (lo a multiple of 16) of every row of `table`: [rows, Hkv, hi-lo, D], 32 bits."""
    per = pool.shape[3]
    tile = torch.arange(lo // 16, -(-hi // 16), device=pool.device)
    ids = table[:, tile // per].long().clamp(min=0)
    tiles = pool[0][ids, :, tile % per].transpose(1, 2)  # [rows, Hkv, tiles, bytes]
    x = _values(tiles, D, is_v)
    return x.reshape(*x.shape[:2], -1, D)[:, :, :hi - lo]


def _read(s):
    """The last B tokens of every row, as a row of values a token."""
    case = s["case"]
    N, B, Hkv, D, page = (case[k] for k in ("N", "B", "Hkv", "D", "page"))
    pos = (s["length"].long() - B)[:, None] + torch.arange(B, device="cuda")
    ids = s["table"].long().gather(1, pos // page)
    out = []
    for pool, is_v in ((s["k"], False), (s["v"], True)):
        rows = []
        # the tiles of some tokens at a time, then of each its own line
        step = max(1, (1 << 25) // (16 * Hkv * D))
        for a in range(0, N * B, step):
            p, i = pos.reshape(-1)[a:a + step], ids.reshape(-1)[a:a + step]
            x = _line(pool[0][i, :, p % page // 16], p % 16, D, is_v)
            rows.append(x.to(DTYPES[case["dtype"]]))
        out.append(torch.cat(rows).view(N * B, Hkv * D))
    return dict(k=out[0], v=out[1])


def _line(tiles, t, D, is_v):
    """The values of line t[n] of tiles [n, Hkv, 17 D / 2]: [n, Hkv, D] in 32 bits."""
    n, Hkv = tiles.shape[:2]
    at = torch.arange(n, device=tiles.device)
    both, scale = tiles[..., :8 * D], tiles[..., 8 * D:]
    if is_v:
        both = both.reshape(n, Hkv, 4, 16, D // 32, 4)[at, :, t // 4, :, :, t % 4].transpose(2, 3)
        scale = scale.reshape(n, Hkv, 4, D // 32, 4)[at, :, t // 4, :, t % 4]
    else:
        both = both.reshape(n, Hkv, 16, D // 2)[at, :, t]
        scale = scale.reshape(n, Hkv, 16, D // 32)[at, :, t]
    level = torch.tensor(LEVELS, device=tiles.device)
    level = torch.cat([level, -level])
    both = both.reshape(n, Hkv, D // 32, 16).int()
    value = torch.stack([level[both & 15], level[both >> 4]], -1).view(n, Hkv, D // 32, 32)
    return (value * (scale.int() << 23).view(torch.float32)[..., None]).view(n, Hkv, D)


def _store(s):
    case = s["case"]
    N, B, Hkv, D, page = (case[k] for k in ("N", "B", "Hkv", "D", "page"))
    width = Hkv * D
    pos = ((s["length"].long() - B)[:, None] + torch.arange(B, device="cuda")).view(-1)
    row = torch.arange(N, device="cuda").repeat_interleave(B)
    ids, tile, t = s["table"][row, pos // page].long(), pos % page // 16, pos % 16
    n_pages, per = s["k"].shape[1], page // 16
    for pool, x, is_v in ((s["k"], s["qkv"][:, width:2 * width], False),
                          (s["v"], s["qkv"][:, 2 * width:], True)):
        code, e = _quantise(x.reshape(N * B, Hkv, D), case["dtype"])
        both, scale = _bytes(code), (e + 127).to(torch.uint8)
        codes, scales = pool[0, ..., :8 * D], pool[0, ..., 8 * D:]
        if is_v:
            codes = codes.unflatten(-1, (4, 16, D // 32, 4))
            codes[ids, :, tile, t // 4, :, :, t % 4] = (
                both.view(N * B, Hkv, D // 32, 16).transpose(2, 3))
            scales.unflatten(-1, (4, D // 32, 4))[ids, :, tile, t // 4, :, t % 4] = scale
        else:
            codes.unflatten(-1, (16, D // 2))[ids, :, tile, t] = both
            scales.unflatten(-1, (16, D // 32))[ids, :, tile, t] = scale
    return _read(s)


def _attend(s):
    case = s["case"]
    N, B, Hkv, G, D, shared = (case[k] for k in ("N", "B", "Hkv", "G", "D", "shared"))
    dtype = s["qkv"].dtype
    rows = B * G
    q = s["qkv"][:, :G * Hkv * D].float().view(N, B, Hkv, G, D).permute(0, 2, 1, 3, 4) * D ** -0.5
    q = q.reshape(N, Hkv, rows, D)
    first = shared // 16 * 16  # (what is left of the prefix is read with the requests' own)
    last = (s["length"].long()[:, None] - B + torch.arange(B, device="cuda"))[:, None, :, None, None]
    own_len = max(s["lengths"]) - first
    out = torch.empty(N, Hkv, rows, D, device="cuda")
    lse = torch.empty(N, Hkv, rows, device="cuda")
    if first:
        pre_k = _gather(s["k"], s["table"][:1], 0, first, D, False)[0].transpose(1, 2).contiguous()
        pre_v = _gather(s["v"], s["table"][:1], 0, first, D, True)[0]
    step = max(1, (1 << 28) // (max(own_len, 1) * Hkv * D), (1 << 25) // (own_len * Hkv * rows))
    for a in range(0, N, step):
        n = min(step, N - a)
        table = s["table"][a:a + n]
        own_k = _gather(s["k"], table, first, first + own_len, D, False).transpose(2, 3).contiguous()
        score = q[a:a + n] @ own_k
        del own_k
        if first:
            flat = q[a:a + n].transpose(0, 1).reshape(Hkv, n * rows, D)
            pre = (flat @ pre_k).view(Hkv, n, rows, first).transpose(0, 1)
            score = torch.cat([pre, score], -1)
        pos = torch.arange(first + own_len, device="cuda")
        score.view(n, Hkv, B, G, -1).masked_fill_(pos > last[a:a + n], -math.inf)
        top = score.amax(-1, keepdim=True).clamp(min=-1e30)
        weight = (score - top).exp_()
        total = weight.sum(-1, keepdim=True)
        lse[a:a + n] = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
        own_v = _gather(s["v"], table, first, first + own_len, D, True)
        sums = weight[..., first:] @ own_v
        if first:
            flat = weight[..., :first].transpose(0, 1).reshape(Hkv, n * rows, first)
            sums += (flat @ pre_v).view(Hkv, n, rows, D).transpose(0, 1)
        out[a:a + n] = torch.where(total > 0, sums / total, 0.0)
    out = out.view(N, Hkv, B, G, D).permute(0, 2, 1, 3, 4).reshape(N * B, Hkv * G * D)
    lse = lse.view(N, Hkv, B, G).permute(0, 2, 1, 3).reshape(N * B, Hkv * G)
    return dict(out=out.to(dtype), lse=lse)


def _logprobs(s):
    """Rows without a token: nothing is known of them (0, rank -1, alternatives -1 at -inf)."""
    case = s["case"]
    V, top, B = case["V"], case["top"], case["B"]
    token = s["token"].view(-1)
    x = s["logits"].float()
    t = torch.ones(len(token), device="cuda")
    if s["temperature"] is not None:
        t = s["temperature"].repeat_interleave(B)
    greedy = (t == 0)[:, None]
    peak = x.max(-1, keepdim=True).values
    z = (x - peak) / torch.where(greedy, 1.0, t[:, None])
    weight = z.exp()
    total = weight.sum(-1, keepdim=True, dtype=torch.float64)
    log_total = total.log()
    mean = (weight * z).sum(-1, keepdim=True, dtype=torch.float64) / total
    entropy = torch.where(greedy, 0.0, log_total - mean)[:, 0]
    # the order of the ids: by value, the lowest first among equal ones
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
    key = order * (1 << 32) + (V - 1 - torch.arange(V, device="cuda"))
    best = key.amax(-1, keepdim=True)
    at = token.clamp(min=0)[:, None]
    logprob = torch.where(greedy, torch.where(key.gather(1, at) == best, 0.0, -math.inf),
                          z.gather(1, at).double() - log_total)[:, 0]
    rank = (x > x.gather(1, at)).sum(-1).int()
    none = token < 0
    result = dict(logprob=torch.where(none, 0.0, logprob).float(),
                  entropy=torch.where(none, 0.0, entropy).float(),
                  rank=torch.where(none, -1, rank))
    if top:
        k = min(top, V)
        ids = V - 1 - key.topk(k, -1).values % (1 << 32)
        first = torch.arange(k, device="cuda") == 0
        values = torch.where(greedy, torch.where(first, 0.0, -math.inf),
                             z.gather(1, ids).double() - log_total)
        result["top_ids"] = torch.where(none[:, None], -1, ids)
        result["top_logprobs"] = torch.where(none[:, None], -math.inf, values).float()
    return result


# ---------------------------------------------------------------------------- the library's calls
def _cache(s):
    from jacobi_block_refiner_amd import xpress
    if "cache" not in s:
        s["cache"] = xpress.Cache(k=s["k"], v=s["v"], table=s["table"], length=s["length"],
                                  ref=s["ref"], dtype=DTYPES[s["case"]["dtype"]])
    return xpress, s["cache"]


def _own_read(s):
    xpress, cache = _cache(s)
    case = s["case"]
    N, B, width = case["N"], case["B"], case["Hkv"] * case["D"]
    if "out" not in s:
        s["out"] = [torch.empty(N * B, width, dtype=DTYPES[case["dtype"]], device="cuda")
                    for _ in range(2)]
    xpress.cache_read(cache, 0, s["out"][0], s["out"][1], N=N, B=B)
    return dict(k=s["out"][0], v=s["out"][1])


def _own_store(s):
    xpress, cache = _cache(s)
    case = s["case"]
    width = case["Hkv"] * case["D"]
    xpress.cache_append(cache, 0, s["qkv"][:, width:2 * width], s["qkv"][:, 2 * width:], N=case["N"],
                        B=case["B"])
    return _own_read(s)


def _own_attend(s):
    xpress, cache = _cache(s)
    N, B, Hq, D = s["case"]["N"], s["case"]["B"], s["case"]["Hkv"] * s["case"]["G"], s["case"]["D"]
    if "ws" not in s:
        s["ws"] = xpress.attention_workspace(cache, N, B, Hq)
        s["out"] = torch.empty(N * B, Hq * D, dtype=s["qkv"].dtype, device="cuda")
        s["lse"] = torch.empty(N * B, Hq, device="cuda")
    xpress.block_attention(cache, 0, s["qkv"][:, :Hq * D], N=N, B=B, Hq=Hq, out=s["out"],
                           shared=s["case"]["shared"], lse=s["lse"], ws=s["ws"])
    return dict(out=s["out"], lse=s["lse"])


def _own_logprobs(s):
    from jacobi_block_refiner_amd import xpress
    case = s["case"]
    N, B, V, top = (case[k] for k in ("N", "B", "V", "top"))
    if "ws" not in s:
        s["ws"] = xpress.logprobs_workspace(N * B, V, top)
        s["out"] = dict(logprob=torch.empty(N * B, device="cuda"),
                        entropy=torch.empty(N * B, device="cuda"),
                        rank=torch.empty(N * B, dtype=torch.int32, device="cuda"))
        if top:
            s["out"]["top_ids"] = torch.empty(N * B, top, dtype=torch.int64, device="cuda")
            s["out"]["top_logprobs"] = torch.empty(N * B, top, device="cuda")
    xpress.token_logprobs(s["logits"], s["token"], temperature=s["temperature"], ws=s["ws"],
                          **s["out"])
    return s["out"]


def run(state):
    plain = dict(store=_store, read=_read, attend=_attend, logprobs=_logprobs)
    kernels = dict(store=_own_store, read=_own_read, attend=_own_attend, logprobs=_own_logprobs)
    return (kernels if own else plain)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------- floors
def work(case):
    op = case["op"]
    if op == "logprobs":
        size = dict(bf16=2, f16=2, f32=4)[case["dtype"]]
        rows = case["N"] * case["B"]
        # (rows without a token need not be read: half of a block of 16, in the mean)
        read = rows * (17 / 32 if case["B"] == 16 else 1)
        return dict(bytes=read * case["V"] * size + rows * (20 + 12 * case["top"]),
                    flops=6 * read * case["V"])
    N, B, Hkv, D = (case[k] for k in ("N", "B", "Hkv", "D"))
    held = Hkv * 17 * D / 16  # bytes of K and V of one token
    if op in ("store", "read"):
        wide = 4 * Hkv * D
        both = N * B * (wide + held)
        # (a store's own tokens are read back: what it wrote once more, and the values)
        return dict(bytes=both * (2 if op == "store" else 1), flops=0)
    G = case["G"]
    mean_own = (max(case["own_max"], B) + B) / 2
    seen = case["shared"] + mean_own - (B - 1) / 2  # of an average query
    keys = case["shared"] + N * mean_own
    return dict(bytes=keys * held + 4 * N * B * Hkv * G * D + 4 * N * B * Hkv * G,
                flops=4 * N * B * Hkv * G * D * seen)


# ------------------------------------------------------------------------ the definition, 64 bits
def _where(D, is_v):
    """Byte of every token and channel of a tile, and of its scale: [16, D] each."""
    t, c = torch.arange(16)[:, None], torch.arange(D)[None]
    if is_v:
        code = ((t // 4 * 16 + c % 32 // 2) * (D // 32) + c // 32) * 4 + t % 4
        return code, 8 * D + (t // 4 * (D // 32) + c // 32) * 4 + t % 4
    return t * (D // 2) + c // 2, 8 * D + t * (D // 32) + c // 32


def _exact_tiles(tiles, D, is_v):
    code, scale = (i.to(tiles.device) for i in _where(D, is_v))
    odd = (torch.arange(D, device=tiles.device) % 2).to(torch.uint8)
    c = tiles[..., code] >> (4 * odd) & 15
    # sign, two bits of exponent, one of significand
    sign = 1.0 - 2.0 * (c >> 3).double()
    e, f = (c >> 1 & 3).double(), (c & 1).double()
    size = torch.where(e > 0, (1 + f / 2) * torch.pow(2.0, e - 1), f / 2)
    return sign * size * torch.pow(2.0, tiles[..., scale].double() - 127)


def _exact_quantised(x, dtype):
    """The nearest values of 4 bits, one group of 32 channels after the other in 64 bits."""
    lo, hi = RANGE[dtype]
    g = x.double().view(*x.shape[:-1], -1, 32)
    top = g.abs().amax(-1, keepdim=True)
    frac, e = torch.frexp(top)  # top = frac 2^e, frac in [0.5, 1)
    e = e - 1 + (frac >= 0.875).to(e.dtype) - 2
    step = torch.pow(2.0, torch.where(top > 0, e, lo).clamp(lo, hi).double())
    y = (g / step).clamp(-6, 6)
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    away = (y.abs()[..., None] - level).abs()
    # a tie goes to the even code: the odd ones are a little further
    away = away + 1e-9 * (torch.arange(8, device=x.device) % 2)
    return (torch.copysign(level[away.argmin(-1)], y) * step).view(x.shape)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "logprobs":
        return _exact_logprobs(s)
    N, B, Hkv, D, page = (case[k] for k in ("N", "B", "Hkv", "D", "page"))
    if op == "store":
        width, parts = Hkv * D, []
        for x in (s["qkv"][:, width:2 * width], s["qkv"][:, 2 * width:]):
            done = [_exact_quantised(y, case["dtype"]) for y in x.split(max(1, (1 << 23) // width))]
            parts.append(torch.cat(done))
        return dict(k=parts[0], v=parts[1])
    if op == "read":
        out = [], []
        for n, length in enumerate(s["lengths"]):
            for pool, to, is_v in ((s["k"], out[0], False), (s["v"], out[1], True)):
                ids = s["table"][n, :-(-length // page)].long()
                x = _exact_tiles(pool[0, ids], D, is_v)  # [pages, Hkv, tiles, 16, D]
                x = x.permute(0, 2, 3, 1, 4).reshape(-1, Hkv * D)
                to.append(x[length - B:length])
        return dict(k=torch.cat(out[0]), v=torch.cat(out[1]))
    G = case["G"]
    out = torch.zeros(N, B, Hkv, G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((N, B, Hkv, G), -math.inf, dtype=torch.float64, device="cuda")
    q = s["qkv"][:, :G * Hkv * D].double().view(N, B, Hkv, G, D)
    for n, length in enumerate(s["lengths"]):
        if length == 0:
            continue
        ids = s["table"][n, :-(-length // page)].long()
        k, v = (_exact_tiles(pool[0, ids], D, is_v).permute(1, 0, 2, 3, 4).reshape(Hkv, -1, D)
                [:, :length] for pool, is_v in ((s["k"], False), (s["v"], True)))
        rows = q[n].permute(1, 0, 2, 3).reshape(Hkv, B * G, D)
        score = torch.matmul(rows, k.transpose(1, 2).contiguous()).view(Hkv, B, G, length)
        score = score / math.sqrt(D)
        hidden = torch.arange(length, device="cuda") > torch.arange(
            length - B, length, device="cuda")[:, None]
        score = score.masked_fill(hidden[None, :, None], -math.inf)
        norm = torch.logsumexp(score, -1)
        p = torch.exp(score - norm[..., None]).view(Hkv, B * G, length)
        out[n] = torch.matmul(p, v.contiguous()).view(Hkv, B, G, D).transpose(0, 1)
        lse[n] = norm.transpose(0, 1)
    return dict(out=out.view(N * B, -1), lse=lse.view(N * B, -1))


def _exact_logprobs(s):
    case = s["case"]
    V, top, B = case["V"], case["top"], case["B"]
    names = ["logprob", "entropy"] + (["top_logprobs"] if top else [])
    parts = {name: [] for name in names}
    temps = s["temperature"].tolist() if s["temperature"] is not None else [1.0] * case["N"]
    for n, t in enumerate(temps):
        for a in range(0, B, 64):
            token = s["token"][n, a:a + 64]
            x = s["logits"][n * B + a:n * B + a + len(token)].double()
            if t == 0:
                first = x.argmax(-1, keepdim=True)
                logp = torch.full_like(x, -math.inf).scatter_(1, first, 0.0)
                entropy = torch.zeros(len(x), dtype=torch.float64, device=x.device)
            else:
                logp = torch.log_softmax(x / t, -1)
                entropy = -(logp.exp() * logp).sum(-1)
            none = token < 0
            logprob = logp.gather(1, token.clamp(min=0)[:, None])[:, 0]
            parts["logprob"].append(torch.where(none, 0.0, logprob))
            parts["entropy"].append(torch.where(none, 0.0, entropy))
            if top:
                best = logp.sort(-1, descending=True).values[:, :top]
                parts["top_logprobs"].append(torch.where(none[:, None], -math.inf, best))
    out = {name: torch.cat(parts[name]) for name in names}
    return dict(logprob=out["logprob"], entropy=out["entropy"], rank=None,
                **(dict(top_ids=None, top_logprobs=out["top_logprobs"]) if top else {}))
