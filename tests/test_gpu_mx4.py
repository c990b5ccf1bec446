"""The cache of 4 bits on the GPU: what an append leaves and a read gives, the page calls, and attention
over it, against 64-bit oracles."""
import math

import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import xpress
from tests import mx4_oracle as mx4
from tests.gpu_helpers import log
from tests.serve_oracle import CacheOracle, attention, attention_bounds
from tests.test_gpu_attention import Case

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    xpress.lib()
    torch.cuda.set_device(0)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def odd_values(n, width, dtype, g):
    """Values of many sizes, ties, zeros, subnormals, infinities and NaN among them."""
    x = torch.randn(n, width, generator=g)
    groups = x.view(n, -1, 32)
    span = (-23, 15) if dtype == torch.float16 else (-126, 126)
    groups *= torch.pow(2.0, torch.randint(*span, groups.shape[:2], generator=g).float())[..., None]
    half_steps = torch.randint(-28, 29, groups.shape, generator=g) / 4
    kind = torch.randint(6, groups.shape[:2], generator=g)[..., None]
    groups[:] = torch.where(kind == 0, half_steps, groups)
    groups[:] = torch.where(kind == 1, 0.0, groups)
    few = torch.rand(groups.shape, generator=g)
    groups[:] = torch.where((kind == 2) & (few < 0.05), math.nan, groups)
    groups[:] = torch.where((kind == 2) & (few > 0.97), math.inf, groups)
    groups[:] = torch.where((kind == 2) & (few > 0.985), -math.inf, groups)
    tiny = torch.finfo(dtype).tiny * torch.rand(groups.shape, generator=g)
    groups[:] = torch.where(kind == 3, tiny, groups)
    return x.to(dtype)


SHAPES = [  # Hkv, page, D, rows' lengths, B
    (1, 16, 64, [1], 1),
    (3, 16, 64, [40, 0, 17, 5, 33], 7),  # rows shorter than the block: its first tokens are skipped
    (2, 64, 128, [64, 130, 77], 64),
    (8, 32, 128, [16, 32, 200], 16),
    (1, 256, 256, [300, 257], 33),
    (5, 16, 256, [9, 50], 9),
]


class Held:
    """A cache of 4 bits with rows of `lengths` tokens on pages in random order, random bytes in it."""

    def __init__(self, Hkv, page, D, lengths, dtype, layers=2, seed=0, spare=2):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        self.n_pages = sum(need) + spare
        shape = (layers, self.n_pages, Hkv, page // 16, 17 * D // 2)
        self.k, self.v = (torch.randint(256, shape, generator=g, dtype=torch.uint8) for _ in range(2))
        perm = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = np.full((len(lengths), max(max(need), 1) + 1), -1, np.int32)
        for r, n in enumerate(need):
            self.table[r, :n] = [perm.pop() for _ in range(n)]
        self.lengths, self.page, self.D, self.dtype, self.Hkv = lengths, page, D, dtype, Hkv
        self.c = xpress.Cache(k=self.k.cuda(), v=self.v.cuda(), table=i32(self.table),
                              length=i32(lengths), ref=i32(np.ones(self.n_pages)), dtype=dtype)

    def set(self, layer, is_v, r, pos, x):
        """Writes the nearest values of x [Hkv, D] into the host's bytes."""
        pool, p, t = (self.v if is_v else self.k), self.table[r, pos // self.page], pos % 16
        tiles = pool[layer, p, :, pos % self.page // 16]
        code, e = mx4.quantise(x, self.dtype)
        for c in range(self.D):
            byte, odd = mx4.code_byte(self.D, t, c, is_v)
            tiles[:, byte] = (tiles[:, byte] & (15 if odd else 240)) | (code[:, c] << 4 * odd).to(torch.uint8)
        for s in range(self.D // 32):
            tiles[:, mx4.scale_byte(self.D, t, s, is_v)] = (e[:, s] + 127).to(torch.uint8)


def same_values(a, b, D, is_v):
    """Equal bytes, but for the sign of a 0."""
    va, vb = mx4.pool_values(a, D, is_v), mx4.pool_values(b, D, is_v)
    return torch.equal(va.nan_to_num(9), vb.nan_to_num(9))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_what_an_append_leaves_and_a_read_gives(i, dtype):
    Hkv, page, D, lengths, B = SHAPES[i]
    log(f"append {SHAPES[i]} {dtype}")
    x = Held(Hkv, page, D, lengths, dtype, seed=i)
    N, width = len(lengths), Hkv * D
    g = torch.Generator().manual_seed(i)
    new = torch.cat([odd_values(N * B, 2 * width, dtype, g), torch.zeros(N * B, 8, dtype=dtype)], 1)
    d = new.cuda()
    xpress.cache_append(x.c, 1, d[:, :width], d[:, width:2 * width], B=B)
    for r, n in enumerate(lengths):
        for b in range(B):
            pos = n - B + b
            if pos >= 0:
                for is_v in (False, True):
                    part = new[r * B + b, is_v * width:(is_v + 1) * width].view(Hkv, D)
                    x.set(1, is_v, r, pos, part)
    torch.cuda.synchronize()
    # nothing but those tokens changed, in either layer, and they are what the oracle says
    assert torch.equal(x.c.k[0].cpu(), x.k[0]) and torch.equal(x.c.v[0].cpu(), x.v[0])
    assert same_values(x.c.k.cpu(), x.k, D, False) and same_values(x.c.v.cpu(), x.v, D, True)
    # read back: the last B tokens, zeros before a row's first
    hold = torch.full((N * B, 2 * width + 16), 5.0, dtype=dtype, device="cuda")
    xpress.cache_read(x.c, 1, hold[:, :width], hold[:, width:2 * width], B=B)
    got = hold.cpu()
    assert bool((got[:, 2 * width:] == 5).all())
    for r, n in enumerate(lengths):
        for b in range(B):
            for is_v in (False, True):
                part = new[r * B + b, is_v * width:(is_v + 1) * width].view(Hkv, D)
                want = mx4.values(*mx4.quantise(part, dtype)) if n - B + b >= 0 else torch.zeros(Hkv, D)
                assert torch.equal(got[r * B + b, is_v * width:(is_v + 1) * width].double(),
                                   want.double().flatten()), (r, b, is_v)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_reading_ranges_of_rows_in_any_order(bits, dtype):
    """Positions before, inside and behind a row, rows outside the cache, another layer."""
    Hkv, page, D, lengths, B = 2, 32, 128, [70, 0, 33, 100], 40
    x = Held(Hkv, page, D, lengths, dtype, seed=3)
    g = torch.Generator().manual_seed(1)
    if bits == 16:
        shape = (2, x.n_pages, Hkv, page, D)
        k, v = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
        x.c = xpress.Cache(k=k.cuda(), v=v.cuda(), table=x.c.table, length=x.c.length, ref=x.c.ref)
    else:
        for pool in (x.k, x.v):  # scales of the type's own range
            pool[..., 8 * D:] = torch.randint(110, 140, pool[..., 8 * D:].shape, generator=g,
                                              dtype=torch.uint8)
        x.c.k.copy_(x.k)
        x.c.v.copy_(x.v)
        k, v = mx4.pool_values(x.k, D, False), mx4.pool_values(x.v, D, True)
    for rows, first in (([3, -1, 2, 9], [90, 0, -10, 5]), ([0, 1, 2, 3], [31, 0, 1 << 30, -(1 << 31)])):
        out = torch.full((2, 4 * B, Hkv * D), 7.0, dtype=dtype, device="cuda")
        xpress.cache_read(x.c, 1, out[0], out[1], B=B, seq=i32(rows), first=i32(first))
        got = out.cpu().view(2, 4, B, Hkv, D)
        for i, (r, f) in enumerate(zip(rows, first)):
            for b in range(B):
                for pool, y in ((k, got[0]), (v, got[1])):
                    want = torch.zeros(Hkv, D, dtype=torch.float64)
                    if 0 <= r < 4 and 0 <= f + b < lengths[r]:
                        want = pool[1, x.table[r, (f + b) // page], :, (f + b) % page].double()
                    assert torch.equal(y[i, b].double(), want), (i, b)


def test_appends_that_do_nothing():
    """No room, rows outside the cache, pages outside the pool: no byte changes."""
    x = Held(2, 16, 64, [20, 30], torch.bfloat16, seed=5)
    new = torch.randn(8, 128, device="cuda").bfloat16()
    xpress.cache_append(x.c, 0, new, new, B=4, lacking=i32([3]))
    xpress.cache_append(x.c, 0, new, new, B=4, seq=i32([-1, 2]))
    x.c.table.fill_(-5)
    xpress.cache_append(x.c, 0, new, new, B=4)
    torch.cuda.synchronize()
    assert torch.equal(x.c.k.cpu(), x.k) and torch.equal(x.c.v.cpu(), x.v)


@pytest.mark.parametrize("shape", [(1, 40, 1, 16, 64, 6, 9, torch.bfloat16),
                                   (3, 75, 2, 32, 128, 9, 11, torch.float16),
                                   (2, 33, 5, 16, 256, 5, 14, torch.bfloat16)],
                         ids=lambda s: f"p{s[1]}x{s[3]}D{s[4]}")
def test_random_turns(shape):
    """Forks, extensions with copies of shared pages, appends, trims and compactions: the tables as the
    16-bit oracle's, the values the nearest of what was written."""
    layers, n_pages, Hkv, page, D, rows, ld, dtype = shape
    rng = np.random.default_rng(7)
    g = torch.Generator().manual_seed(7)
    o = CacheOracle(layers, n_pages, Hkv, page, D, rows, ld, dtype)
    o.k.zero_()
    o.v.zero_()
    c = xpress.Cache.empty(layers, n_pages, Hkv, page, D, rows, ld, dtype=dtype, bits=4)
    assert c.k.shape == (layers, n_pages, Hkv, page // 16, 17 * D // 2) and c.page == page
    c.k.zero_()
    c.v.zero_()
    ws, lacking = xpress.cache_workspace(c, rows), i32([7])
    live = i32([0])
    for step in range(25):
        op = rng.integers(5)
        some = rng.permutation(rows)[:rng.integers(1, rows + 1)]
        if op == 0 and len(some) > 1:
            n = len(some) // 2
            o.fork(some[:n], some[n:2 * n])
            xpress.cache_fork(c, i32(some[:n]), i32(some[n:2 * n]))
        elif op == 1:
            drop = rng.integers(0, 40, len(some))
            o.trim(some, drop)
            xpress.cache_trim(c, i32(drop), seq=i32(some))
        elif op == 2 and step % 2:
            n = o.compact()
            xpress.cache_compact(c, live=live, ws=ws)
            assert int(live.item()) == n
        else:
            B = int(rng.integers(1, 24))
            want = o.extend(some, [B] * len(some))
            xpress.cache_extend(c, B, seq=i32(some), lacking=lacking, ws=ws)
            assert int(lacking.item()) == want
            if want == 0:
                for layer in range(layers):
                    new = torch.randn(len(some) * B, 2 * Hkv * D, generator=g).to(dtype)
                    held = mx4.values(*mx4.quantise(new.view(-1, 2 * Hkv, D), dtype)).to(dtype)
                    o.append(layer, held[:, :Hkv], held[:, Hkv:], some, B)
                    d = new.cuda()
                    xpress.cache_append(c, layer, d[:, :Hkv * D], d[:, Hkv * D:], seq=i32(some), B=B)
        torch.cuda.synchronize()
        assert np.array_equal(c.length.cpu().numpy(), o.length), step
        assert np.array_equal(c.table.cpu().numpy(), o.table), step
        assert np.array_equal(c.ref.cpu().numpy(), o.ref), step
        held = [(o.table[r, t // page], t % page) for r in range(rows) for t in range(o.length[r])]
        if held:
            p, line = (torch.tensor([h[i] for h in held]) for i in (0, 1))
            for pool, want, is_v in ((c.k, o.k, False), (c.v, o.v, True)):
                got = mx4.pool_values(pool.cpu(), D, is_v)
                assert torch.equal(got[:, p, :, line], want[:, p, :, line].double()), (step, is_v)


class Case4(Case):
    """Rows as in Case, held in 4 bits; the lines past a row's end, and pages nobody holds, are bytes
    of 255 or random ones."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        g = torch.Generator().manual_seed(99)
        self.pools = []
        for name, is_v in (("k", False), ("v", True)):
            x = getattr(self, name)
            dead = x.isnan().any(-1)  # [layers, pages, Hkv, page]
            code, e = mx4.quantise(x.unflatten(3, (-1, 16)), self.dtype)
            code[dead.unflatten(3, (-1, 16))] = 15
            e[dead.unflatten(3, (-1, 16))] = 128
            some = (torch.rand(dead.shape, generator=g) < 0.5).unflatten(3, (-1, 16))
            some &= dead.unflatten(3, (-1, 16))
            code[some] = torch.randint(16, code[some].shape, generator=g)
            e[some] = torch.randint(-127, 129, e[some].shape, generator=g)
            self.pools.append(mx4.pack(code, e, is_v))
            live = torch.where(dead[..., None], 0.0, mx4.pool_values(self.pools[-1], self.D, is_v))
            setattr(self, name, live.to(self.dtype))

    def cache(self):
        return xpress.Cache(k=self.pools[0].cuda(), v=self.pools[1].cuda(), dtype=self.dtype,
                            table=torch.from_numpy(self.table).cuda(),
                            length=torch.tensor(self.lengths, dtype=torch.int32, device="cuda"),
                            ref=torch.zeros(self.k.shape[1], dtype=torch.int32, device="cuda"))


CASES = [
    # lengths, shared, B, Hkv, G, D, page
    dict(lengths=[1], shared=0, B=1, Hkv=1, G=1, D=64, page=16),
    dict(lengths=[1, 2, 15, 16, 17, 31, 32, 33], shared=0, B=1, Hkv=2, G=4, D=128, page=16),
    dict(lengths=[5, 0, 3, 64, 65], shared=0, B=4, Hkv=2, G=3, D=64, page=16),
    dict(lengths=[100, 37, 129], shared=32, B=16, Hkv=2, G=4, D=128, page=32),
    dict(lengths=[300, 0, 290, 288, 401], shared=277, B=7, Hkv=1, G=5, D=128, page=64),
    dict(lengths=[64, 64, 64], shared=64, B=1, Hkv=2, G=1, D=64, page=64),
    dict(lengths=[700, 650], shared=600, B=16, Hkv=1, G=8, D=256, page=128),
    dict(lengths=[500, 3, 17], shared=450, B=5, Hkv=1, G=2, D=64, page=256),  # rows end in the prefix
    dict(lengths=[1025], shared=0, B=16, Hkv=2, G=7, D=128, page=16),
    dict(lengths=[260] * 9, shared=256, B=2, Hkv=3, G=1, D=64, page=32),
    dict(lengths=[90, 91, 92, 93], shared=80, B=33, Hkv=1, G=9, D=64, page=16),  # 297 rows a request
    dict(lengths=[420 + 3 * i for i in range(40)], shared=384, B=16, Hkv=1, G=1, D=64, page=32),
    dict(lengths=[70] * 70, shared=64, B=2, Hkv=1, G=5, D=128, page=64),
    dict(lengths=[1300, 1301], shared=1279, B=64, Hkv=1, G=4, D=128, page=128),
    dict(lengths=[60] * 11, shared=43, B=16, Hkv=1, G=3, D=64, page=16),  # less than a tile
    dict(lengths=[150, 160, 170, 180, 0], shared=130, B=30, Hkv=1, G=4, D=256, page=32),
    # decoding: few query rows a request
    dict(lengths=[1500, 7, 0, 900, 1], shared=0, B=1, Hkv=2, G=8, D=128, page=64),
    dict(lengths=[1500, 7, 0, 900, 1], shared=0, B=1, Hkv=2, G=1, D=64, page=16),
    dict(lengths=[900, 2, 513], shared=0, B=1, Hkv=1, G=5, D=256, page=32),
    dict(lengths=[4000, 31, 33], shared=0, B=2, Hkv=1, G=8, D=128, page=16),
    dict(lengths=[1000, 1001, 999], shared=0, B=4, Hkv=1, G=8, D=64, page=32),
    dict(lengths=[1000, 1001, 3], shared=0, B=8, Hkv=1, G=4, D=256, page=64),
    # many query rows a head (D 128): the shared part in wide items
    dict(lengths=[400, 0, 395, 17, 300, 399, 396, 401] * 2, shared=390, B=16, Hkv=2, G=8, D=128, page=16),
    dict(lengths=[200 + i for i in range(9)], shared=192, B=57, Hkv=1, G=4, D=128, page=64),
    dict(lengths=[1300 - 40 * i for i in range(16)], shared=640, B=16, Hkv=1, G=8, D=128, page=128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention_against_the_definition(i, dtype):
    log(f"attention over 4 bits, case {i} {CASES[i]} {dtype}")
    x = Case4(**CASES[i], dtype=dtype, seed=i)
    c = x.cache()
    x.check(x.run(c), what="shared")
    if x.shared:
        x.check(x.run(c, shared=0), what="not shared")
        x.check(x.run(c, shared=x.shared - 1), what="shared, one less")
    x.check(x.run(c, lse=False), what="no lse")


def test_rows_in_any_order_and_rows_outside():
    for B, G in ((3, 2), (1, 1), (16, 4)):
        x = Case4(lengths=[80, 33, 0, 47, 95], shared=32, B=B, Hkv=2, G=G, D=128, page=16, seed=3)
        c = x.cache()
        order = [4, 1, 3]
        x.check(x.run(c, seq=i32(order), rows=order), rows=order, what="a list")
        out, lse = x.run(c, seq=i32([4, -1, 9]), rows=[4, 0, 0])
        assert bool((out[B:] == 0).all()) and bool((lse[B:] == -math.inf).all())
        x.check((out[:B], lse[:B]), rows=[4], what="rows outside are empty")


def test_page_ids_outside_the_pool_and_lengths_past_the_table():
    for B, G in ((2, 2), (16, 5)):
        x = Case4(lengths=[80, 90], shared=0, B=B, Hkv=1, G=G, D=64, page=16, seed=7)
        c = x.cache()
        c.table[0, 1], c.table[0, 2] = -9, 1 << 30
        out, lse = x.run(c)
        x.q = x.q[B:]
        x.check((out[B:], lse[B:]), rows=[1], what="the other row")
        y = Case4(lengths=[80, 96], shared=0, B=B, Hkv=1, G=G, D=64, page=16, seed=8)
        c = y.cache()
        c.table = c.table[:, :6].contiguous()
        c.length[1] = 1 << 30  # the table holds 96
        y.check(y.run(c), what="clamped")


@pytest.mark.parametrize("B,G,D", [(1, 4, 128), (4, 4, 64), (16, 4, 128)])
def test_large_scores(B, G, D):
    """Scores of some hundreds, and keys that grow along the row: the maximum moves in every tile."""
    x = Case4(lengths=[400, 333], shared=256, B=B, Hkv=1, G=G, D=D, page=32, seed=4, q_scale=16.0)
    x.check(x.run(x.cache()), what="large")
    x.check(x.run(x.cache(), shared=0), what="large, alone")
    x.check(x.run(x.cache(), scale=0.01), scale=0.01, what="scale 0.01")
    y = Case4(lengths=[600], shared=0, B=B, Hkv=1, G=G, D=D, page=16, seed=5)
    grown = torch.zeros(1, y.k.shape[1], 1, 16, D)
    for j in range(600):
        grown[0, y.table[0, j // 16], :, j % 16] = y.q[0, :D].float() * (j / 100.0)
    y.pools[0] = mx4.pool_of(grown, y.dtype, False)
    y.k = mx4.pool_values(y.pools[0], D, False).to(y.dtype)
    y.check(y.run(y.cache(), scale=0.125), scale=0.125, what="growing")
    y.q.neg_()
    y.check(y.run(y.cache(), scale=0.125), scale=0.125, what="falling")


@pytest.mark.parametrize("B,G,shared", [(1, 4, 0), (1, 4, 400), (16, 4, 400), (16, 16, 400)])
def test_streams_workspaces_and_captured_calls(B, G, shared):
    """Another stream, a workspace full of NaN, the same bits twice; replays of a captured call read
    lengths and tables as they are then, with eager work in between."""
    x = Case4(lengths=[500, 480, 0], shared=shared, B=B, Hkv=2, G=G, D=128, page=64, seed=9, n_layers=3,
              layer=2)
    c = x.cache()
    N = 3
    ws = xpress.attention_workspace(c, N, B, x.Hq)
    ws.fill_(0xFF)
    a = x.run(c, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = x.run(c, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    x.check(a, what="first")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q = x.wide.cuda()[:, :x.Hq * x.D]
    out = torch.empty(N * B, x.Hq * x.D, dtype=x.dtype, device="cuda")
    lse = torch.empty(N * B, x.Hq, device="cuda")

    def call():
        xpress.block_attention(c, 2, q, B=B, Hq=x.Hq, out=out, lse=lse, shared=shared, ws=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in ([500, 480, 0], [430, 2, 401], [499, 480, 450], [500, 480, 0]):
        x.lengths = lengths
        x.table[2] = x.table[1]  # (a row of the others' pages)
        c.table.copy_(torch.from_numpy(x.table))
        c.length.copy_(i32(lengths))
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = (out.cpu().view(N * B, x.Hq, x.D), lse.cpu())
        x.check(got, what=f"replay {lengths}")
        ws.fill_(0xFF)
        eager = x.run(c, ws=ws)
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])


@pytest.mark.parametrize("shared", [0, 16500])
def test_more_pages_than_an_item_holds(shared):
    x = Case4(lengths=[20000, 17001, 16501], shared=shared, B=2, Hkv=1, G=2, D=64, page=16, seed=60)
    x.check(x.run(x.cache()), what=f"many pages, shared {shared}")


def test_many_short_requests():
    """More requests than workgroups: rows of no, one and a few tokens among longer ones."""
    for B, G, D, page in ((1, 4, 128, 16), (3, 5, 64, 64), (1, 8, 256, 32)):
        lengths = [(37 * i) % 90 for i in range(140)] + [300, 1, 0, 64, 65]
        x = Case4(lengths=lengths, shared=0, B=B, Hkv=2, G=G, D=D, page=page, seed=70)
        x.check(x.run(x.cache()), what=f"{len(lengths)} requests, D {D}")


@pytest.mark.parametrize("D,ld", [(64, 2048), (128, 2048), (256, 512)])
@pytest.mark.parametrize("B,G,shared", [(16, 4, 0), (16, 3, 0), (13, 3, 100), (33, 1, 70), (2, 2, 0)])
def test_blocks_under_tables_for_long_contexts(D, ld, B, G, shared):
    """Requests of 17 to 64 query rows a head in several waves, where the tables could hold much more
    than they do."""
    N, Hkv = 8, 4
    lengths = [shared + n for n in (1, 40, 0, 33, 300, 97, 64, 31)]
    lengths[2] = 0
    x = Case4(lengths=lengths, shared=shared, B=B, Hkv=Hkv, G=G, D=D, page=16, seed=80)
    wide = np.full((N, ld), -1, np.int32)
    wide[:, :x.table.shape[1]] = x.table
    x.table = wide
    c = x.cache()
    x.check(x.run(c), what=f"D {D}, {B * G} rows")
    x.check(x.run(c, shared=0), what="not shared")
    order = [6, 1, 4]
    x.check(x.run(c, seq=i32(order), rows=order), rows=order, what="a list")


@pytest.mark.parametrize("N,B,G,shared", [(4100, 1, 2, 0), (4100, 1, 2, 64), (5, 1, 2, 0)])
def test_rows_of_whole_runs_of_tiles(N, B, G, shared):
    """Rows of exactly 64 and 128 tiles of 32 tokens, and one token more or less, which one wave walks
    through where there are very many requests; among them as many short ones as it takes."""
    Hkv, D, page = 2, 64, 64
    long = [2048, 2049, 2047, 4096, 4097]
    at = [0, 1, N // 2, N - 2, N - 1] if N > 5 else range(5)
    lengths = [(7 * i) % 4 + shared for i in range(N)]
    for r, n in zip(at, long):
        lengths[r] = n + shared
    log(f"rows of whole runs of tiles, {N} requests, shared {shared}")
    g = torch.Generator().manual_seed(2)
    pages = -(-(4097 + shared) // page)
    shape = (1, pages, Hkv, page, D)
    pools = [mx4.pool_of(torch.randn(shape, generator=g), torch.bfloat16, v) for v in (False, True)]
    k, v = (mx4.pool_values(p, D, is_v).float() for p, is_v in zip(pools, (False, True)))
    # every row's tokens are the first of the same pages
    c = xpress.Cache(k=pools[0].cuda(), v=pools[1].cuda(), length=i32(lengths), ref=i32(np.ones(pages)),
                     table=torch.arange(pages, dtype=torch.int32, device="cuda").repeat(N, 1))
    q = torch.randn(N * B, Hkv * G * D, generator=g).bfloat16()
    out = torch.empty(N * B, Hkv * G * D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(N * B, Hkv * G, device="cuda")
    ws = xpress.attention_workspace(c, N, B, Hkv * G)
    ws.fill_(0xFF)
    xpress.block_attention(c, 0, q.cuda(), B=B, Hq=Hkv * G, N=N, out=out, lse=lse, shared=shared, ws=ws)
    rows = sorted({*at, *range(0, N, max(1, N // 40))})
    pick = [r * B + b for r in rows for b in range(B)]
    want, wl, mass, size = attention(k[0], v[0], np.tile(np.arange(pages), (N, 1)), lengths, page,
                                     q[pick], rows, B, Hkv * G, D ** -0.5)
    bound, lse_bound = attention_bounds(want, mass, size, 4200, D, torch.bfloat16)
    got = out.cpu().double().view(N * B, Hkv * G, D)
    assert bool(((got[pick] - want).abs() <= bound).all())
    sees = wl > -math.inf
    assert bool((lse.cpu()[pick][~sees] == -math.inf).all())
    assert bool(((lse.cpu()[pick].double() - wl).abs() <= lse_bound + wl.abs() * 2.0 ** -22)[sees].all())
    assert not bool(got.isnan().any())


def test_long_row_in_a_big_pool():
    """Pages past byte 2^32 of a layer, written and attended to."""
    n_pages, Hkv, page, D = 140000, 8, 64, 128
    c = xpress.Cache.empty(1, n_pages, Hkv, page, D, rows=2, table_ld=40, bits=4)
    assert c.k[0].numel() > 1 << 32
    log("attention over 4 bits past 32 bits")
    g = torch.Generator().manual_seed(1)
    ids = n_pages - 1 - torch.randperm(60, generator=g)
    lengths = [30 * 64 - 5, 30 * 64 - 60]
    c.table[0, :30], c.table[1, :30] = ids[:30].int().cuda(), ids[30:].int().cuda()
    c.length.copy_(i32(lengths))
    held = torch.zeros(2, 60, Hkv, page, D)
    new = torch.randn(2, 1920, Hkv, 2 * D, generator=g).bfloat16()
    for r, n in enumerate(lengths):
        kv = new[r, :n].cuda()
        k, v = (kv[..., i * D:(i + 1) * D].reshape(n, Hkv * D) for i in (0, 1))
        xpress.cache_append(c, 0, k, v, B=n, seq=i32([r]))
        val = mx4.values(*mx4.quantise(new[r, :n].unflatten(-1, (2, D)), torch.bfloat16)).float()
        for t in range(n):
            held[:, 30 * r + t // 64, :, t % 64] = val[t].transpose(0, 1)
    table = np.full((2, 40), -1, np.int64)
    table[0, :30], table[1, :30] = np.arange(30), np.arange(30, 60)
    for B in (1, 16):
        q = torch.randn(2 * B, 8 * D, generator=g).to(torch.bfloat16)
        out = torch.empty(2 * B, 8 * D, dtype=torch.bfloat16, device="cuda")
        xpress.block_attention(c, 0, q.cuda(), B=B, Hq=8, out=out,
                               ws=xpress.attention_workspace(c, 2, B, 8))
        want, _, mass, size = attention(held[0], held[1], table, lengths, page, q, [0, 1], B, 8, D ** -0.5)
        bound, _ = attention_bounds(want, mass, size, 1920, D, torch.bfloat16)
        assert bool(((out.cpu().double().view(2 * B, 8, D) - want).abs() <= bound).all())
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("B", [1, 2, 17])
def test_more_rows_than_a_grid_has_in_its_second_direction(B):
    """70,001 rows of one head: appended to and read."""
    N, D, dtype = 70001, 64, torch.bfloat16
    g = torch.Generator().manual_seed(B)
    pool = torch.zeros(1, 2 * N, 1, 1, 17 * D // 2, dtype=torch.uint8, device="cuda")
    length = torch.randint(1, 33, (N,), generator=g, dtype=torch.int32)
    c = xpress.Cache(k=pool, v=pool.clone(), table=torch.randperm(2 * N, generator=g).int().view(N, 2).cuda(),
                     length=length.cuda(), ref=torch.ones(2 * N, dtype=torch.int32, device="cuda"),
                     dtype=dtype)
    new = torch.randn(2, N * B, D, generator=g).to(dtype)
    d, out = new.cuda(), torch.full((2, N * B, D), 7.0, dtype=dtype, device="cuda")
    xpress.cache_append(c, 0, d[0], d[1], B=B)
    xpress.cache_read(c, 0, out[0], out[1], B=B)
    want = mx4.values(*mx4.quantise(new, dtype)).view(2, N, B, D)
    held = torch.arange(B)[None] >= B - length[:, None]
    assert torch.equal(out.cpu().view(2, N, B, D).double(), want * held[None, :, :, None])


@pytest.mark.parametrize("bits", [4, 16])
def test_a_row_read_twice_and_reads_at_once(bits):
    """The same row several times in a list, two reads on streams of their own beside an append to other
    rows, and replays of a captured read over rows that grow."""
    Hkv, page, D, lengths, B, dtype = 3, 32, 128, [300, 200, 64], 50, torch.float16
    width = Hkv * D
    x = Held(Hkv, page, D, lengths, dtype, seed=8)
    g = torch.Generator().manual_seed(2)
    if bits == 16:
        shape = (2, x.n_pages, Hkv, page, D)
        k, v = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
        x.c = xpress.Cache(k=k, v=v, table=x.c.table, length=x.c.length, ref=x.c.ref)
    first = torch.randn(lengths[0], 2 * width, generator=g).to(dtype).cuda()
    xpress.cache_append(x.c, 1, first[:, :width], first[:, width:], seq=i32([0]), B=lengths[0])
    whole = torch.empty_like(first)
    xpress.cache_read(x.c, 1, whole[:, :width], whole[:, width:], seq=i32([0]), B=lengths[0])
    torch.cuda.synchronize()
    starts = [250, 13, 250]
    outs = [torch.zeros(3 * B, 2 * width, dtype=dtype, device="cuda") for _ in range(2)]
    seq, at = i32([0] * 3), i32(starts)
    streams = [torch.cuda.Stream() for _ in range(3)]
    new = torch.randn(2 * B, 2 * width, generator=g).to(dtype).cuda()
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        with torch.cuda.stream(s):
            xpress.cache_read(x.c, 1, o[:, :width], o[:, width:], seq=seq, first=at, B=B)
    with torch.cuda.stream(streams[2]):
        xpress.cache_append(x.c, 1, new[:, :width], new[:, width:], seq=i32([1, 2]), B=B)
    torch.cuda.synchronize()
    for o in outs:
        for i, f in enumerate(starts):
            assert torch.equal(o.view(3, B, -1)[i], whole[f:f + B])
    graph, o = torch.cuda.CUDAGraph(), outs[0]
    last = i32([1])
    with torch.cuda.graph(graph):
        xpress.cache_read(x.c, 1, o[:B, :width], o[:B, width:], seq=last, B=B)
    for n in (200, 180, 49, 0, 200):
        x.c.length[1] = n
        o.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        xpress.cache_read(x.c, 1, outs[1][:B, :width], outs[1][:B, width:], seq=last, B=B)
        assert torch.equal(o[:B].view(torch.int16), outs[1][:B].view(torch.int16)) and bool((o[B:] == 3).all())
        assert bool((o[:max(0, B - n)] == 0).all())
