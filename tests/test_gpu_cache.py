"""The paged cache's calls on the GPU against the host oracle, bit for bit after every call."""
import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import xpress
from tests.gpu_helpers import log
from tests.serve_oracle import CacheOracle

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    xpress.lib()
    torch.cuda.set_device(0)


def device_cache(o: CacheOracle) -> xpress.Cache:
    return xpress.Cache(k=o.k.cuda(), v=o.v.cuda(), table=torch.from_numpy(o.table).cuda(),
                        length=torch.from_numpy(o.length).cuda(),
                        ref=torch.from_numpy(o.ref).cuda())


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def same(c: xpress.Cache, o: CacheOracle, what: str):
    torch.cuda.synchronize()
    assert np.array_equal(c.length.cpu().numpy(), o.length), what
    assert np.array_equal(c.table.cpu().numpy(), o.table), what
    assert np.array_equal(c.ref.cpu().numpy(), o.ref), what
    assert torch.equal(c.k.cpu().view(torch.int16), o.k.view(torch.int16)), what
    assert torch.equal(c.v.cpu().view(torch.int16), o.v.view(torch.int16)), what
    # the counts are what the tables say
    held = [o.table[r, :o.pages(o.length[r])] for r in range(len(o.length))]
    count = np.bincount(np.concatenate(held).astype(np.int64), minlength=len(o.ref))
    assert np.array_equal(count, o.ref), what


SHAPES = [  # layers, pages, Hkv, page, D, rows, ld, dtype
    (1, 40, 1, 16, 64, 6, 9, torch.bfloat16),
    (3, 75, 2, 32, 128, 9, 11, torch.float16),
    (2, 33, 5, 16, 256, 5, 14, torch.bfloat16),
    (1, 21, 3, 256, 64, 4, 5, torch.float16),
    (2, 1500, 1, 16, 64, 40, 70, torch.bfloat16),  # more pages than the planning workgroup's threads
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"p{s[1]}x{s[3]}D{s[4]}")
@pytest.mark.parametrize("seed", [0, 1])
def test_random_turns(shape, seed):
    layers, n_pages, Hkv, page, D, rows, ld, dtype = shape
    rng = np.random.default_rng(seed)
    o = CacheOracle(layers, n_pages, Hkv, page, D, rows, ld, dtype, seed)
    c = device_cache(o)
    ws = xpress.cache_workspace(c, rows)
    lacking = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    seen = {"cow": 0, "lack": 0, "over": 0, "moved": 0}
    log(f"cache turns {shape} seed {seed}")
    for turn in range(14):
        sub = rng.permutation(rows)[: rng.integers(1, rows + 1)]
        kind = rng.integers(0, 6)
        if kind == 0 and rows > 1:
            half = rows // 2
            perm = rng.permutation(rows)
            n = rng.integers(1, half + 1)
            src, dst = rng.choice(perm[:half], n), perm[half:][:n]
            o.fork(src, dst)
            xpress.cache_fork(c, i32(src), i32(dst))
            same(c, o, f"turn {turn} fork")
        elif kind == 1:
            drop = rng.integers(-2, 3 * page, len(sub)) if rng.random() < 0.8 else None
            o.trim(sub, drop)
            xpress.cache_trim(c, None if drop is None else i32(drop), seq=i32(sub))
            same(c, o, f"turn {turn} trim")
        elif kind == 2:
            live = torch.zeros(1, dtype=torch.int32, device="cuda")
            before = o.table.copy()
            want = o.compact()
            seen["moved"] += int((before != o.table).sum())
            xpress.cache_compact(c, live=live, ws=ws)
            same(c, o, f"turn {turn} compact")
            assert int(live.item()) == want
        # every turn also grows some rows and writes their last tokens
        each = rng.integers(-1, 2 * page + 3, len(sub))
        if rng.random() < 0.3:
            each[:] = int(rng.integers(0, 17))
            got = xpress.cache_extend(c, int(each[0]), lacking=lacking, ws=ws, seq=i32(sub))
        else:
            got = xpress.cache_extend(c, i32(each), lacking=lacking, ws=ws, seq=i32(sub))
        refs = o.ref.copy()
        want = o.extend(sub, each)
        same(c, o, f"turn {turn} extend")
        assert int(got.item()) == want
        seen["lack"] += want > 0
        seen["over"] += want < 0
        seen["cow"] += int((o.ref < refs).sum())
        B = int(rng.integers(1, 20))
        wide = torch.randn(len(sub) * B, 2 * Hkv * D + 8).to(dtype)
        k_new, v_new = wide[:, :Hkv * D], wide[:, Hkv * D:2 * Hkv * D]
        layer = int(rng.integers(layers))
        # rows that share a page are not written through it
        alone = [r for r in sub if all(
            o.ref[o.table[r, p // page]] == 1
            for p in range(max(int(o.length[r]) - B, 0), int(o.length[r])))]
        if not alone:
            continue
        at = np.concatenate([np.arange(B) + B * int(np.nonzero(sub == r)[0][0]) for r in alone])
        k_new, v_new = wide[at][:, :Hkv * D], wide[at][:, Hkv * D:2 * Hkv * D]
        o.append(layer, k_new.reshape(-1, Hkv, D), v_new.reshape(-1, Hkv, D), alone, B)
        dev = wide[at].cuda()
        xpress.cache_append(c, layer, dev[:, :Hkv * D], dev[:, Hkv * D:2 * Hkv * D], B=B,
                            seq=i32(alone))
        same(c, o, f"turn {turn} append")
    log(f"  seen {seen}")


def test_copy_on_write_of_a_shared_partial_page():
    """Two rows of one prompt both grow: each gets a page of its own with the prompt's tokens, and
    the page that nobody holds any more is free."""
    o = CacheOracle(2, 12, 2, 16, 64, 3, 6, torch.bfloat16)
    c = device_cache(o)
    ws = xpress.cache_workspace(c, 3)
    lacking = i32([9])
    for want, add in (([0], [21]),):
        assert o.extend(want, add) == 0
        xpress.cache_extend(c, i32(add), lacking=lacking, ws=ws, seq=i32(want))
    o.fork([0], [1])
    xpress.cache_fork(c, i32([0]), i32([1]))
    same(c, o, "fork")
    assert o.ref[1] == 2
    assert o.extend([1, 0], [1, 2]) == 0
    xpress.cache_extend(c, i32([1, 2]), lacking=lacking, ws=ws, seq=i32([1, 0]))
    same(c, o, "extend")
    assert o.ref[1] == 0 and int(lacking.item()) == 0
    assert o.table[0, 1] == 3 and o.table[1, 1] == 2


def test_nothing_changes_when_pages_are_missing_or_a_row_is_full():
    o = CacheOracle(1, 5, 1, 16, 64, 3, 4, torch.bfloat16)
    c = device_cache(o)
    ws = xpress.cache_workspace(c, 3)
    lacking = i32([9])
    for add, want in (([40, 30, 16], 1), ([80, 80, 0], -1), ([64, 16, 16], 1),
                      ([64, 16, 0], 0), ([1, 0, 0], -1), ([0, 0, 1], 1)):
        got = int(xpress.cache_extend(c, i32(add), lacking=lacking, ws=ws).item())
        assert got == o.extend(range(3), add) == want, add
        same(c, o, str(add))


def test_rows_and_pages_outside_the_cache_are_skipped():
    """List entries outside [0, rows) do nothing; page ids outside the pool are neither counted nor
    written."""
    o = CacheOracle(1, 8, 1, 16, 64, 4, 4, torch.bfloat16)
    c = device_cache(o)
    ws = xpress.cache_workspace(c, 4)
    lacking = i32([9])
    xpress.cache_extend(c, i32([5, 5, 20]), lacking=lacking, ws=ws, seq=i32([-1, 4, 2]))
    assert o.extend([2], [20]) == 0
    same(c, o, "extend")
    xpress.cache_trim(c, i32([3, 3]), seq=i32([1 << 30, 2]))
    o.trim([2], [3])
    same(c, o, "trim")
    xpress.cache_fork(c, i32([-5, 2]), i32([0, 77]))
    same(c, o, "fork")
    new = torch.randn(2, 64).to(torch.bfloat16)
    xpress.cache_append(c, 0, new.cuda(), new.cuda(), B=1, seq=i32([9, 2]))
    o.append(0, new[1:].reshape(1, 1, 64), new[1:].reshape(1, 1, 64), [2], 1)
    same(c, o, "append")
    bad = torch.from_numpy(o.table).cuda()
    bad[2, 0], bad[2, 1] = 99, -7
    c.table.copy_(bad)
    xpress.cache_append(c, 0, new.cuda(), new.cuda(), B=2, seq=i32([2]))
    xpress.cache_trim(c, seq=i32([2]))
    torch.cuda.synchronize()
    assert torch.equal(c.k.cpu().view(torch.int16), o.k.view(torch.int16))
    assert np.array_equal(c.ref.cpu().numpy(), o.ref)
    assert int(c.length[2].item()) == 0 and bool((c.table[2] == -1).all())


def test_list_of_a_row_twice_stays_inside_the_buffers():
    """A row twice in one list is the caller's error: the result is unspecified, but every page id
    and length stays in range and other rows keep theirs."""
    o = CacheOracle(1, 32, 1, 16, 64, 4, 6, torch.bfloat16)
    c = device_cache(o)
    ws = xpress.cache_workspace(c, 4)
    lacking = i32([9])
    xpress.cache_extend(c, i32([30]), lacking=lacking, ws=ws, seq=i32([1]))
    keep = c.table[1].clone()
    xpress.cache_extend(c, 90, lacking=lacking, ws=ws, seq=i32([0, 0, 0]))
    torch.cuda.synchronize()
    t = c.table.cpu().numpy()
    assert t.min() >= -1 and t.max() < 32
    assert torch.equal(c.table[1], keep)
    assert 0 <= int(c.length[0].item()) <= 6 * 16


@pytest.mark.parametrize("page,Hkv,D", [(64, 8, 128)])
def test_offsets_past_32_bits(page, Hkv, D):
    """A layer of 4.6e9 elements (9.2 GB a side): pages at its end are written, copied and moved."""
    n_pages = 70000
    assert n_pages * page * Hkv * D > 1 << 32
    c = xpress.Cache.empty(1, n_pages, Hkv, page, D, rows=3, table_ld=4)
    log("cache past 32 bits")
    ws = xpress.cache_workspace(c, 3)
    lacking, live = i32([9]), i32([9])
    c.ref.fill_(1)
    c.ref[n_pages - 4:] = 0  # the only free pages are the last ones
    xpress.cache_extend(c, i32([page + 9, 0, 0]), lacking=lacking, ws=ws)
    assert int(lacking.item()) == 0
    assert c.table[0].tolist() == [n_pages - 4, n_pages - 3, -1, -1]
    new = torch.randn(page + 9, 2 * Hkv * D, device="cuda").to(torch.bfloat16)
    xpress.cache_append(c, 0, new[:, :Hkv * D], new[:, Hkv * D:], B=page + 9, N=1)
    kk = new[:, :Hkv * D].view(-1, Hkv, D).transpose(0, 1)
    vv = new[:, Hkv * D:].view(-1, Hkv, D).transpose(0, 1)
    assert torch.equal(c.k[0, n_pages - 4], kk[:, :page])
    assert torch.equal(c.v[0, n_pages - 3, :, :9], vv[:, page:])
    xpress.cache_fork(c, i32([0]), i32([1]))
    xpress.cache_extend(c, i32([1]), lacking=lacking, ws=ws, seq=i32([1]))
    assert int(lacking.item()) == 0
    assert c.table[1].tolist() == [n_pages - 4, n_pages - 2, -1, -1]
    assert torch.equal(c.v[0, n_pages - 2, :, :9], vv[:, page:])
    c.ref[:n_pages - 4] = 0
    xpress.cache_compact(c, live=live, ws=ws)
    assert int(live.item()) == 3
    assert c.table[0].tolist() == [0, 1, -1, -1] and c.table[1].tolist() == [0, 2, -1, -1]
    assert torch.equal(c.k[0, 0], kk[:, :page]) and torch.equal(c.v[0, 2, :, :9], vv[:, page:])
    assert c.ref[:4].tolist() == [2, 1, 1, 0] and int(c.ref.sum().item()) == 4
    del c, ws
    torch.cuda.empty_cache()


def test_replaced_tensors_are_the_ones_used():
    c = xpress.Cache.empty(1, 8, 1, 16, 64, 2, 4)
    lacking, ws = torch.full((1,), 9, dtype=torch.int32, device="cuda"), xpress.cache_workspace(c, 2)
    old = c.length
    c.length = torch.zeros_like(old)
    xpress.cache_extend(c, 20, lacking=lacking, ws=ws)
    assert c.length.tolist() == [20, 20] and old.tolist() == [0, 0] and lacking.item() == 0
    with pytest.raises(ValueError):
        c.ref = torch.zeros(7, dtype=torch.int32, device="cuda")
    assert c.ref.numel() == 8  # refused: the one before stays


def test_more_rows_and_pages_than_a_step_of_the_plan():
    """1100 rows and 9500 pages: the rows' needs, the free pages and the live ones take several steps."""
    rng = np.random.default_rng(4)
    rows = 1100
    o = CacheOracle(1, 9500, 1, 16, 64, rows, 20, torch.bfloat16, 4)
    c = device_cache(o)
    ws = xpress.cache_workspace(c, rows)
    lacking, live = torch.zeros(1, dtype=torch.int32, device="cuda"), i32([0])
    every = np.arange(rows)
    for turn, most in enumerate((200, 60, 90)):
        each = np.minimum(rng.integers(0, most, rows), 320 - o.length)
        want = o.extend(every, each)
        xpress.cache_extend(c, i32(each), lacking=lacking, ws=ws)
        same(c, o, f"turn {turn} extend")
        assert int(lacking.item()) == want == (0, 0, 99)[turn]
        drop = np.where(rng.random(rows) < 0.25, rng.integers(0, 150, rows), 0)
        o.trim(every, drop)
        xpress.cache_trim(c, i32(drop))
        src, dst = rng.permutation(rows)[:200].reshape(2, 100)
        o.fork(src, dst)
        xpress.cache_fork(c, i32(src), i32(dst))
        same(c, o, f"turn {turn} trim and fork")
        if turn:
            want = o.compact()
            xpress.cache_compact(c, live=live, ws=ws)
            same(c, o, f"turn {turn} compact")
            assert int(live.item()) == want > 4096
    each = np.minimum(rng.integers(100, 200, rows), 320 - o.length)
    want = o.extend(every, each)
    xpress.cache_extend(c, i32(each), lacking=lacking, ws=ws)
    same(c, o, "too many pages")
    assert int(lacking.item()) == want > 0


def guarded(shape, dtype, fill):
    """A tensor in the middle of a larger one; the larger one's two ends."""
    n = int(np.prod(shape))
    pad = -(-n // 8) * 8
    hold = torch.full((3 * pad,), fill, dtype=dtype, device="cuda")
    return hold[pad:pad + n].view(shape), (hold[:pad], hold[pad + n:])


@pytest.mark.parametrize("n_pages", [24, 5000])
@pytest.mark.parametrize("twice", ["trim", "fork"])
def test_compaction_after_a_row_twice_in_a_list(twice, n_pages):
    """A row twice in a list of trim or fork may release its pages twice and leave counts below 0
    (set here too, since it depends on timing): a compaction then moves pages inside the pools alone,
    and rows whose pages nobody else named keep their tokens."""
    log(f"compaction after a row twice in {twice}, {n_pages} pages")
    k, k_ends = guarded((2, n_pages, 1, 16, 64), torch.bfloat16, 3.0)
    v, v_ends = guarded((2, n_pages, 1, 16, 64), torch.bfloat16, 4.0)
    table, t_ends = guarded((5, 8), torch.int32, -1)
    ref, r_ends = guarded((n_pages,), torch.int32, 0)
    length, l_ends = guarded((5,), torch.int32, 0)
    c = xpress.Cache(k=k, v=v, table=table, length=length, ref=ref)
    ws = xpress.cache_workspace(c, 5)
    lacking, live = i32([9]), i32([9])
    k.copy_(torch.randn(k.shape)), v.copy_(torch.randn(v.shape))
    order = [0, 3, 1, 2, 4]  # row 4's pages are the last ones
    xpress.cache_extend(c, i32([40, 33, 16, 50, 90]), lacking=lacking, ws=ws, seq=i32(order))
    # row 4 moves to the end of the pool, so that it has to come to the front again
    held = table[4, :6].long()
    far = torch.arange(n_pages - 6, n_pages, device="cuda")
    for pool in (k, v):
        pool[:, far] = pool[:, held]
    ref[held], ref[far] = 0, 1
    table[4, :6] = far.int()
    tokens = [(k[:, table[r, :p].long()].clone(), v[:, table[r, :p].long()].clone())
              for r, p in ((3, 3), (4, 6))]
    if twice == "trim":
        xpress.cache_trim(c, i32([40, 40, 40]), seq=i32([0, 0, 0]))
    else:
        xpress.cache_fork(c, i32([1, 1, 1]), i32([0, 0, 0]))
    torch.cuda.synchronize()
    assert int(ref.min()) >= -2
    ref[:3] = torch.tensor([-1, -2, -1], dtype=torch.int32)  # what row 0 held: released twice
    ws.fill_(0x7f)
    xpress.cache_compact(c, live=live, ws=ws)
    torch.cuda.synchronize()
    n = int(live.item())
    assert n == int((ref > 0).sum()) and bool((ref[:n] > 0).all()) and bool((ref[n:] <= 0).all())
    t = table.cpu().numpy()
    assert t.min() >= -1 and t.max() < n_pages
    assert t[3:].max() < n
    for (r, p), (wk, wv) in zip(((3, 3), (4, 6)), tokens):
        at = table[r, :p].long()
        assert torch.equal(k[:, at], wk) and torch.equal(v[:, at], wv), r
    for ends, fill in ((k_ends, 3.0), (v_ends, 4.0), (t_ends, -1), (r_ends, 0), (l_ends, 0)):
        assert all(bool((e == fill).all()) for e in ends)
    # pages of counts below 0 are free: extensions take them
    ref[n] = -1
    xpress.cache_extend(c, 30, lacking=lacking, ws=ws, seq=i32([4]))
    assert int(lacking.item()) == 0 and int(length[4]) == 120
    assert table[4, 6:].tolist() == [n, n + 1] and ref[n:n + 3].tolist() == [1, 1, 0]


@pytest.mark.parametrize("why", ["no pages", "a full row"])
def test_a_turn_without_room_changes_nothing(why):
    """Rows that share a prompt, one table or the pool too small for the next block: extension, append
    and trim leave every row, count and page as it was, also captured and replayed, and the same
    graph goes on once there is room."""
    B, n_pages, ld = 6, 24, 6
    o = CacheOracle(2, n_pages, 2, 16, 64, 4, ld, torch.bfloat16, 5)
    o.extend([0], [40])
    o.fork([0, 0], [1, 2])
    o.extend([1, 2], [9, 13])
    if why == "a full row":
        o.extend([3], [ld * 16 - B + 1])
    else:
        o.ref[o.ref == 0] = 1  # held by rows that are not in the batch
    c = device_cache(o)
    ws = xpress.cache_workspace(c, 4)
    lacking, drop = i32([0]), i32([2, 0, 5, 1])
    new = torch.randn(4 * B, 2 * 2 * 64, device="cuda").to(torch.bfloat16)

    def turn():
        xpress.cache_extend(c, B, N=4, lacking=lacking, ws=ws)
        for layer in range(2):
            xpress.cache_append(c, layer, new[:, :128], new[:, 128:], N=4, B=B, lacking=lacking)
        xpress.cache_trim(c, drop, N=4, lacking=lacking)

    def state():
        return [getattr(c, name).clone() for name in ("table", "length", "ref", "k", "v")]

    before = state()
    turn()
    torch.cuda.synchronize()
    assert (int(lacking.item()) < 0) == (why == "a full row") and int(lacking.item()) != 0
    assert all(torch.equal(a, b) for a, b in zip(before, state()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert int(lacking.item()) != 0
        assert all(torch.equal(a, b) for a, b in zip(before, state()))
    if why == "a full row":  # freed while lacking is not 0: the plain call
        xpress.cache_trim(c, seq=i32([3]))
        o.trim([3], None)
    else:
        held = [int(p) for r in range(4) for p in o.table[r, :o.pages(o.length[r])]]
        o.ref[[p for p in range(n_pages) if p not in held]] = 0
        c.ref.copy_(torch.from_numpy(o.ref))
    graph.replay()
    torch.cuda.synchronize()
    assert int(lacking.item()) == o.extend(range(4), [B] * 4) == 0
    for layer in range(2):
        kv = new.cpu().view(-1, 2, 2, 64)
        o.append(layer, kv[:, 0], kv[:, 1], range(4), B)
    o.trim(range(4), drop.tolist())
    same(c, o, "with room")


def test_more_missing_pages_than_32_bits_hold():
    """4096 rows that ask for 2^20 pages each, in a pool without any: 2^32 pages are missing, not none."""
    rows, ld = 4096, 1 << 20
    c = xpress.Cache.empty(1, 8, 1, 16, 64, rows=rows, table_ld=ld)  # a table of 17 GB
    log("extension by 2^32 pages")
    c.ref.fill_(1)
    ws, lacking = xpress.cache_workspace(c, rows), i32([9])
    xpress.cache_extend(c, ld * 16, lacking=lacking, ws=ws)
    assert int(lacking.item()) == 2 ** 31 - 1
    xpress.cache_extend(c, 3 * 16, lacking=lacking, ws=ws)
    assert int(lacking.item()) == 3 * rows
    assert bool((c.length == 0).all()) and c.ref.tolist() == [1] * 8
    assert all(bool((part == -1).all()) for part in c.table.split(512))
    del c
    torch.cuda.empty_cache()


def test_a_single_token_of_any_row_stride():
    """One row of one token: K of its own, V and q out of wider rows, whose strides mean nothing."""
    c = xpress.Cache.empty(1, 2, 2, 16, 64, 1, 2)
    ws, lacking = xpress.cache_workspace(c, 1), i32([9])
    xpress.cache_extend(c, 1, lacking=lacking, ws=ws)
    k = torch.randn(1, 128, device="cuda").to(torch.bfloat16)
    v = torch.randn(1, 128 + 3, device="cuda").to(torch.bfloat16)[:, :128]
    q = torch.randn(1, 256 + 5, device="cuda").to(torch.bfloat16)[:, :256]
    xpress.cache_append(c, 0, k, v, B=1)
    p = int(c.table[0, 0])
    assert torch.equal(c.k[0, p, :, 0], k.view(2, 64)) and torch.equal(c.v[0, p, :, 0], v.view(2, 64))
    out = torch.empty(1, 256 + 1, dtype=torch.bfloat16, device="cuda")[:, :256]
    xpress.block_attention(c, 0, q, B=1, Hq=4, out=out, ws=xpress.attention_workspace(c, 1, 1, 4))
    assert torch.equal(out.view(2, 2, 64), v.view(2, 1, 64).expand(2, 2, 64))
