"""Block attention over the paged cache against attention from its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import xpress
from tests.gpu_helpers import log
from tests.serve_oracle import attention, attention_bounds

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    xpress.lib()
    torch.cuda.set_device(0)


class Case:
    """Rows of `lengths` tokens whose first `shared` are the same, on pages drawn at random; the
    lines past a row's end, and pages nobody holds, are NaN."""

    def __init__(self, lengths, shared, B, Hkv, G, D, page, dtype=torch.bfloat16, seed=0, q_scale=1.0,
                 n_layers=1, layer=0, pad=8):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.shared, self.B, self.Hq, self.page = lengths, shared, B, Hkv * G, page
        self.D, self.dtype, self.layer = D, dtype, layer
        need = [-(-n // page) for n in lengths]
        ld = max(max(need), -(-shared // page), 1) + 1
        first = shared // page
        perm = rng.permutation(sum(need) + first + 3)
        n_pages = len(perm)
        common, used = perm[:first], first
        self.table = np.full((len(lengths), ld), -1, np.int32)
        pools = torch.full((2, n_pages, Hkv, page, D), math.nan)
        prefix = torch.randn(2, Hkv, max(shared, 1), D, generator=g)
        for r, n in enumerate(lengths):
            for j in range(need[r]):
                if j < first:
                    p = common[j]
                else:
                    p, used = perm[used], used + 1
                self.table[r, j] = p
                lines = min(page, n - j * page)
                if j >= first or r == max(range(len(lengths)), key=lambda x: lengths[x]):
                    pools[:, p, :, :lines] = torch.randn(2, Hkv, lines, D, generator=g)
                both = max(0, min(lines, shared - j * page))
                if both:
                    pools[:, p, :, :both] = prefix[:, :, j * page:j * page + both]
        pools = pools.to(dtype)
        full = torch.full((n_layers, n_pages, Hkv, page, D), 3.0).to(dtype)
        self.k, self.v = full.clone(), full.clone()
        self.k[layer], self.v[layer] = pools[0], pools[1]
        # q and out are slices of wider rows
        self.wide = (torch.randn(len(lengths) * B, self.Hq * D + pad, generator=g) * q_scale).to(dtype)
        self.q = self.wide[:, :self.Hq * D]
        self.pad = pad

    def cache(self):
        return xpress.Cache(k=self.k.cuda(), v=self.v.cuda(),
                            table=torch.from_numpy(self.table).cuda(),
                            length=torch.tensor(self.lengths, dtype=torch.int32, device="cuda"),
                            ref=torch.zeros(self.k.shape[1], dtype=torch.int32, device="cuda"))

    def run(self, cache, shared=None, seq=None, rows=None, scale=None, lse=True, q=None, ws=None):
        rows = list(range(len(self.lengths))) if rows is None else rows
        N = len(rows)
        q = self.wide.cuda()[:N * self.B, :self.Hq * self.D] if q is None else q
        hold = torch.full((N * self.B, self.Hq * self.D + self.pad), 5.0, dtype=self.dtype,
                          device="cuda")
        out = hold[:, :self.Hq * self.D]
        l = torch.full((N * self.B, self.Hq), 7.0, device="cuda") if lse else None
        ws = xpress.attention_workspace(cache, N, self.B, self.Hq) if ws is None else ws
        xpress.block_attention(cache, self.layer, q, B=self.B, Hq=self.Hq, N=N, seq=seq, out=out,
                               lse=l, shared=self.shared if shared is None else shared, ws=ws,
                               scale=scale)
        torch.cuda.synchronize()
        assert bool((hold[:, self.Hq * self.D:] == 5.0).all())  # nothing past a row's end
        return out.cpu().view(N * self.B, self.Hq, self.D), None if l is None else l.cpu()

    def check(self, got, rows=None, scale=None, what=""):
        rows = list(range(len(self.lengths))) if rows is None else rows
        scale = self.D ** -0.5 if scale is None else scale
        out, lse, mass, size = attention(self.k[self.layer], self.v[self.layer], self.table,
                                         self.lengths, self.page, self.q[:len(rows) * self.B],
                                         rows, self.B, self.Hq, scale)
        bound, lse_bound = attention_bounds(out, mass, size, max(self.lengths), self.D, self.dtype)
        err = (got[0].double() - out).abs()
        worst = float((err / bound).max())
        log(f"  {what}: worst error {worst:.3f} of the bound")
        assert not bool(got[0].isnan().any()), what
        assert bool((err <= bound).all()), (what, worst)
        if got[1] is not None:
            empty = lse == -math.inf
            assert bool((got[1][empty] == -math.inf).all()), what
            off = (got[1].double() - lse).abs()[~empty]
            assert bool((off <= (lse_bound + lse.abs() * 2.0 ** -22)[~empty]).all()), (
                what, float(off.max()))


CASES = [
    # lengths, shared, B, Hkv, G, D, page
    dict(lengths=[1], shared=0, B=1, Hkv=1, G=1, D=64, page=16),
    dict(lengths=[5, 0, 3, 64, 65], shared=0, B=4, Hkv=2, G=3, D=64, page=16),
    dict(lengths=[100, 37, 129], shared=32, B=16, Hkv=2, G=4, D=128, page=32),
    dict(lengths=[300, 0, 290, 288, 401], shared=277, B=7, Hkv=1, G=5, D=128, page=64),
    dict(lengths=[64, 64, 64], shared=64, B=1, Hkv=2, G=1, D=64, page=64),
    dict(lengths=[700, 650], shared=600, B=16, Hkv=1, G=8, D=256, page=128),
    dict(lengths=[500, 3, 17], shared=450, B=5, Hkv=1, G=2, D=64, page=256),  # rows end in the prefix
    dict(lengths=[1025], shared=0, B=16, Hkv=2, G=7, D=128, page=16),
    dict(lengths=[260] * 9, shared=256, B=2, Hkv=3, G=1, D=64, page=32),
    dict(lengths=[90, 91, 92, 93], shared=80, B=33, Hkv=1, G=9, D=64, page=16),  # 297 rows a request
    # many query rows a head: the shared part in wide items, whole tiles, a part of one, rows that
    # end inside the prefix, rows without tokens, a last item of few rows
    dict(lengths=[420 + 3 * i for i in range(40)], shared=384, B=16, Hkv=1, G=1, D=64, page=32),
    dict(lengths=[400, 0, 395, 17, 300, 399, 396, 401], shared=390, B=13, Hkv=2, G=6, D=128, page=16),
    dict(lengths=[70] * 70, shared=64, B=2, Hkv=1, G=5, D=128, page=64),
    dict(lengths=[1300, 1301], shared=1279, B=64, Hkv=1, G=4, D=128, page=128),
    dict(lengths=[60] * 11, shared=43, B=16, Hkv=1, G=3, D=64, page=16),  # less than a tile
    dict(lengths=[150, 160, 170, 180, 0], shared=130, B=30, Hkv=1, G=4, D=256, page=32),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_definition(i, dtype):
    log(f"attention case {i} {CASES[i]} {dtype}")
    x = Case(**CASES[i], dtype=dtype, seed=i)
    c = x.cache()
    x.check(x.run(c), what="shared")
    # the same rows attended alone
    x.check(x.run(c, shared=0), what="not shared")
    if x.shared > 1:
        x.check(x.run(c, shared=x.shared - 1), what="shared, one less")


def test_rows_in_any_order_and_rows_outside():
    x = Case(lengths=[80, 33, 0, 47, 95], shared=32, B=3, Hkv=2, G=2, D=128, page=16, seed=3)
    c = x.cache()
    order = [4, 1, 3]
    seq = torch.tensor(order, dtype=torch.int32, device="cuda")
    x.check(x.run(c, seq=seq, rows=order), rows=order, what="a list")
    seq = torch.tensor([4, -1, 9], dtype=torch.int32, device="cuda")
    out, lse = x.run(c, seq=seq, rows=[4, 0, 0])
    assert bool((out[3:] == 0).all()) and bool((lse[3:] == -math.inf).all())
    x.check((out[:3], lse[:3]), rows=[4], what="rows outside are empty")


def test_large_scores_and_other_scales():
    """Scores of some hundreds: one key takes all the weight in most rows; running maxima grow along
    the row."""
    x = Case(lengths=[400, 333], shared=256, B=4, Hkv=1, G=4, D=128, page=32, seed=4, q_scale=16.0)
    x.check(x.run(x.cache()), what="large")
    x.check(x.run(x.cache(), scale=0.01), scale=0.01, what="scale 0.01")
    # keys that grow along the row: the maximum moves in every tile
    y = Case(lengths=[600], shared=0, B=2, Hkv=1, G=2, D=64, page=16, seed=5)
    for j in range(600):
        p = y.table[0, j // 16]
        y.k[0, p, :, j % 16] = (y.q[0, :64].float() * (j / 100.0)).to(y.dtype)
    y.check(y.run(y.cache(), scale=0.125), what="growing")
    y.q.neg_()
    y.check(y.run(y.cache(), scale=0.125), what="falling")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_values_of_later_tokens_do_not_reach_earlier_queries(D, bad):
    """K and V of the block's last token are infinite or NaN: queries before it are as if it were
    not there, the last query is not finite."""
    x = Case(lengths=[75, 40, 64], shared=32, B=6, Hkv=2, G=3, D=D, page=16, seed=6)
    x.pad = 8
    good = x.run(x.cache())
    x.check(good, what="before")
    for r, n in enumerate(x.lengths):
        p = x.table[r, (n - 1) // 16]
        x.v[0, p, :, (n - 1) % 16] = bad
        x.k[0, p, :, (n - 1) % 16, : D // 2] = bad
    got = x.run(x.cache())
    early = [t for t in range(18) if t % 6 != 5]
    assert not bool(got[0][early].isnan().any())
    scale = D ** -0.5
    out, lse, mass, size = attention(
        torch.nan_to_num(x.k[0], 0, 0, 0), torch.nan_to_num(x.v[0], 0, 0, 0), x.table, x.lengths, 16,
        x.q, range(3), 6, x.Hq, scale)
    bound, _ = attention_bounds(out, mass, size, 75, D, x.dtype)
    assert bool(((got[0].double() - out).abs() <= bound)[early].all())
    if math.isnan(bad):
        assert bool(got[0][5::6].isnan().all())


def test_page_ids_outside_the_pool_stay_inside_it():
    """Ids outside the pool are the caller's error: the affected request's result is unspecified, the
    others' is right."""
    x = Case(lengths=[80, 90], shared=0, B=2, Hkv=1, G=2, D=64, page=16, seed=7)
    c = x.cache()
    c.table[0, 1], c.table[0, 2] = -9, 1 << 30
    out, lse = x.run(c)
    x.q = x.q[2:]
    x.check((out[2:], lse[2:]), rows=[1], what="the other row")


def test_lengths_past_the_table_are_clamped():
    x = Case(lengths=[80, 96], shared=0, B=2, Hkv=1, G=1, D=64, page=16, seed=8)
    c = x.cache()
    c.table = c.table[:, :6].contiguous()
    c = xpress.Cache(k=c.k, v=c.v, table=c.table, length=c.length, ref=c.ref)
    c.length[1] = 1 << 30  # the table holds 96
    x.check(x.run(c), what="clamped")


@pytest.mark.parametrize("layer", [0, 2])
def test_layers_streams_and_workspaces(layer):
    """Another stream, another layer, a workspace of another call's, twice the same bits."""
    x = Case(lengths=[500, 480, 0], shared=400, B=16, Hkv=2, G=4, D=128, page=64, seed=9,
             n_layers=3, layer=layer)
    c = x.cache()
    ws = xpress.attention_workspace(c, 3, 16, 8)
    ws.fill_(0xFF)  # NaN everywhere: nothing is read that was not written
    a = x.run(c, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = x.run(c, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    x.check(a, what="first")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x.check(x.run(c, lse=False, ws=ws), what="no lse")


def test_long_row_in_a_big_pool():
    """Pages past element 2^32 of a layer."""
    n_pages, Hkv, page, D = 70000, 8, 64, 128
    c = xpress.Cache.empty(1, n_pages, Hkv, page, D, rows=2, table_ld=40)
    log("attention past 32 bits")
    g = torch.Generator().manual_seed(1)
    ids = n_pages - 1 - torch.randperm(60, generator=g)
    lengths = [30 * 64 - 5, 30 * 64 - 60]
    kv = torch.randn(2, 60, Hkv, page, D, generator=g).to(torch.bfloat16)
    c.k[0, ids.cuda()], c.v[0, ids.cuda()] = kv[0].cuda(), kv[1].cuda()
    table = torch.full((2, 40), -1, dtype=torch.int32)
    table[0, :30], table[1, :30] = ids[:30], ids[30:]
    small = np.full((2, 40), -1, np.int64)
    small[0, :30], small[1, :30] = np.arange(30), np.arange(30, 60)
    c.table.copy_(table)
    c.length.copy_(torch.tensor(lengths, dtype=torch.int32))
    q = torch.randn(4, 8 * D, generator=g).to(torch.bfloat16)
    out = torch.empty(4, 8 * D, dtype=torch.bfloat16, device="cuda")
    xpress.block_attention(c, 0, q.cuda(), B=2, Hq=8, out=out,
                           ws=xpress.attention_workspace(c, 2, 2, 8))
    want, _, mass, size = attention(kv[0], kv[1], small, lengths, page, q, [0, 1], 2, 8, D ** -0.5)
    bound, _ = attention_bounds(want, mass, size, 1920, D, torch.bfloat16)
    assert bool(((out.cpu().double().view(4, 8, D) - want).abs() <= bound).all())
    del c
    torch.cuda.empty_cache()


def test_a_captured_call_follows_the_lengths():
    """Replays of a captured call read lengths and tables as they are then; eager work in between."""
    x = Case(lengths=[200, 180, 190], shared=128, B=4, Hkv=2, G=2, D=128, page=32, seed=11)
    c = x.cache()
    q = x.wide.cuda()[:, :x.Hq * x.D]
    out = torch.empty(12, x.Hq * x.D, dtype=x.dtype, device="cuda")
    lse = torch.empty(12, x.Hq, device="cuda")
    ws = xpress.attention_workspace(c, 3, 4, x.Hq)

    def call():
        xpress.block_attention(c, 0, q, B=4, Hq=x.Hq, out=out, lse=lse, shared=128, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in ([200, 180, 190], [150, 0, 131], [199, 180, 2], [200, 180, 190]):
        x.lengths = lengths
        c.length.copy_(torch.tensor(lengths, dtype=torch.int32))
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = (out.cpu().view(12, x.Hq, x.D), lse.cpu())
        x.check(got, what=f"replay {lengths}")
        eager = x.run(c, ws=ws)
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])


# Many query rows a head (2048 and more, D 128), where the shared part has items of its own kind.
MANY_ROWS = [
    dict(lengths=[400, 0, 395, 17, 300, 399, 396, 401] * 2, shared=390, B=16, Hkv=2, G=8, D=128, page=16),
    dict(lengths=[200 + i for i in range(9)], shared=192, B=57, Hkv=1, G=4, D=128, page=64),  # 2052 rows
    dict(lengths=[1300 - 40 * i for i in range(16)], shared=640, B=16, Hkv=1, G=8, D=128, page=128),
    dict(lengths=[70] * 128, shared=64, B=4, Hkv=1, G=4, D=128, page=16),  # one tile of keys
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(MANY_ROWS)))
def test_many_query_rows(i, dtype):
    c = MANY_ROWS[i]
    x = Case(**c, dtype=dtype, seed=40 + i)
    cache = x.cache()
    x.check(x.run(cache), what=f"many rows {i} {dtype}")
    x.check(x.run(cache, lse=False), what="no lse")


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_many_query_rows_with_values_that_are_not_finite(bad):
    """The last token of rows that end past the prefix is infinite or NaN: the queries before it do
    not see it. (A row that ends inside the prefix shares its last token with the others.)"""
    N, B = 16, 16
    lengths = [90 + 3 * i for i in range(N - 2)] + [40, 0]
    x = Case(lengths=lengths, shared=64, B=B, Hkv=1, G=8, D=128, page=16, seed=50)
    for r, n in enumerate(lengths):
        if n > 64:
            p = x.table[r, (n - 1) // 16]
            x.v[0, p, :, (n - 1) % 16] = bad
            x.k[0, p, :, (n - 1) % 16, :64] = bad
    got = x.run(x.cache())
    early = [t for t in range(N * B) if t % B != B - 1]
    assert not bool(got[0][early].isnan().any())
    out, lse, mass, size = attention(
        torch.nan_to_num(x.k[0], 0, 0, 0), torch.nan_to_num(x.v[0], 0, 0, 0), x.table, lengths, 16,
        x.q, range(N), B, x.Hq, 128 ** -0.5)
    bound, _ = attention_bounds(out, mass, size, max(lengths), 128, x.dtype)
    assert bool(((got[0].double() - out).abs() <= bound)[early].all())
    if math.isnan(bad):
        assert bool(got[0][B - 1:(N - 2) * B:B].isnan().all())


@pytest.mark.parametrize("shared", [0, 16500])
def test_more_pages_than_an_item_holds(shared):
    """Rows of more than a thousand small pages are split whatever their number."""
    x = Case(lengths=[20000, 17001, 16501], shared=shared, B=2, Hkv=1, G=2, D=64, page=16, seed=60)
    x.check(x.run(x.cache()), what=f"many pages, shared {shared}")


# Many requests of few query rows at D 256, without a prefix: two workgroups a CU.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("B,G,page", [(1, 4, 16), (3, 2, 64), (16, 4, 32)])
def test_many_requests_of_wide_heads(B, G, page, dtype):
    lengths = [(37 * i) % 90 for i in range(140)] + [300, 1, 0, 64, 65]
    x = Case(lengths=lengths, shared=0, B=B, Hkv=2, G=G, D=256, page=page, dtype=dtype, seed=70)
    x.check(x.run(x.cache()), what=f"{len(lengths)} requests, D 256")
    bad = Case(lengths=lengths, shared=0, B=B, Hkv=2, G=G, D=256, page=page, dtype=dtype, seed=71)
    if B > 1:  # the last token is not finite: the queries before it do not see it
        for r, n in enumerate(lengths):
            if n:
                bad.v[0, bad.table[r, (n - 1) // page], :, (n - 1) % page] = math.inf
        got = bad.run(bad.cache())
        bad.v = torch.nan_to_num(bad.v, 0, 0, 0)
        early = [t for t in range(len(lengths) * B) if t % B != B - 1]
        out, lse, mass, size = attention(bad.k[0].nan_to_num(0), bad.v[0], bad.table, lengths, page,
                                         bad.q, range(len(lengths)), B, bad.Hq, 256 ** -0.5)
        bound, _ = attention_bounds(out, mass, size, max(lengths), 256, dtype)
        assert bool(((got[0].double() - out).abs() <= bound)[early].all())


@pytest.mark.parametrize("lengths,B,G,D,page", [
    ([0, 400, 395, 17, 300, 399], 5, 3, 64, 16), ([70, 300, 290], 16, 4, 128, 32),
    ([3, 0, 0, 310, 309], 2, 2, 256, 64), ([0] * 5 + [250, 350, 0, 299] * 3, 64, 4, 128, 16),  # wide
    ([100, 0, 30], 4, 2, 128, 16)])  # no row sees the whole prefix
def test_a_first_request_that_ends_inside_the_prefix(lengths, B, G, D, page):
    x = Case(lengths=lengths, shared=270, B=B, Hkv=2 if B < 64 else 1, G=G, D=D, page=page, seed=80)
    x.check(x.run(x.cache()), what=f"short first row, D {D}")
    rows = list(range(len(lengths)))[::-1]
    x.check(x.run(x.cache(), seq=torch.tensor(rows, dtype=torch.int32, device="cuda"), rows=rows),
            rows=rows, what="the other way round")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_first_query_that_sees_the_prefix_alone(bad, dtype):
    """Many query rows, rows of prefix + B - 1 tokens: a block's first query sees the shared part and
    nothing else, and the later tokens of its block, infinite or NaN, do not reach it (nor the queries
    before them)."""
    N, B = 16, 16
    lengths = [79] * 8 + [79 + i for i in range(8)]  # 64 shared tokens
    x = Case(lengths=lengths, shared=64, B=B, Hkv=1, G=8, D=128, page=16, dtype=dtype, seed=51)
    assert len(lengths) * B * 8 >= 1536
    for r, n in enumerate(lengths):
        p = x.table[r, (n - 1) // 16]
        x.v[0, p, :, (n - 1) % 16] = bad
        x.k[0, p, :, (n - 1) % 16, :64] = bad
    got = x.run(x.cache())
    early = [t for t in range(N * B) if t % B != B - 1]
    assert not bool(got[0][early].isnan().any())
    out, lse, mass, size = attention(
        torch.nan_to_num(x.k[0], 0, 0, 0), torch.nan_to_num(x.v[0], 0, 0, 0), x.table, lengths, 16,
        x.q, range(N), B, x.Hq, 128 ** -0.5)
    bound, lse_bound = attention_bounds(out, mass, size, max(lengths), 128, dtype)
    assert bool(((got[0].double() - out).abs() <= bound)[early].all())
    assert bool(((got[1].double() - lse).abs() <= lse_bound + lse.abs() * 2.0 ** -22)[early].all())
    if math.isnan(bad):
        assert bool(got[0][B - 1::B].isnan().all())


@pytest.mark.parametrize("gap", [9.0, 12.3, 17.0, 18.0])
@pytest.mark.parametrize("D,N,B,G,lengths,shared", [
    (64, 1, 1, 1, [60000], 0), (128, 1, 2, 2, [60000], 0), (256, 1, 1, 2, [60000], 0),
    (128, 2, 64, 12, [30000, 30040], 29000),  # wide items
    (64, 3, 2, 2, [40000, 39000, 100], 30000)])
def test_a_key_far_ahead_of_many_others(D, N, B, G, lengths, shared, gap):
    """fp16: one key's weight is e^gap times each of the others', and its value is 0 where theirs are 1:
    what many small weights add up to is kept."""
    page, Hq = 64, G
    scale = D ** -0.5
    most = max(lengths)
    pages = -(-most // page)
    g = torch.Generator().manual_seed(9)
    # a query's first component is 8: the keys' first component alone makes the scores
    k = torch.zeros(1, pages, 1, page, D)
    k[..., 0] = (torch.rand(1, pages, 1, page, generator=g) * 0.02).half().float()
    k[0, 0, 0, 0, 0] = gap / scale / 8
    v = torch.ones(1, pages, 1, page, D)
    v[..., 1::2] = 1 + 0.25 * torch.rand(1, pages, 1, page, D // 2, generator=g)
    v[0, 0, 0, 0] = 0
    k, v = k.half(), v.half()
    q = torch.zeros(N * B, Hq * D)
    q[:, ::D] = 8
    q = q.half()
    table = np.tile(np.arange(pages, dtype=np.int32), (N, 1))  # the rows' own tokens are the same too
    c = xpress.Cache(k=k.cuda(), v=v.cuda(), table=torch.from_numpy(table).cuda(),
                     length=torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                     ref=torch.full((pages,), N, dtype=torch.int32, device="cuda"))
    out = torch.empty(N * B, Hq * D, dtype=torch.float16, device="cuda")
    lse = torch.empty(N * B, Hq, device="cuda")
    xpress.block_attention(c, 0, q.cuda(), B=B, Hq=Hq, N=N, out=out, lse=lse, shared=shared,
                           ws=xpress.attention_workspace(c, N, B, Hq))
    # all heads and most queries see nearly the same: the definition for one head of each row's ends
    for i, n in enumerate(lengths):
        for b in {0, B - 1}:
            want, wl, mass, size = attention(k[0], v[0], table, [n - (B - 1 - b)] * N, page,
                                             q[:1, :D], [i], 1, 1, scale)
            bound, lse_bound = attention_bounds(want, mass, size, most, D, torch.float16)
            t = i * B + b
            got = out[t].cpu().double().view(Hq, D)
            worst = float(((got - want[0]).abs() / bound[0]).max())
            log(f"  far ahead D {D} gap {gap} row {i} query {b}: {worst:.3f} of the bound")
            assert worst <= 1, (i, b)
            assert float((lse[t].cpu().double() - wl[0]).abs().max()) <= float(
                (lse_bound + wl.abs() * 2.0 ** -22).max())


@pytest.mark.parametrize("D", [64, 128])
def test_products_near_the_lowest_value(D):
    """Rows whose only product q.k is -1e29 (a value like any other), and -1e32 (as masked)."""
    c = xpress.Cache.empty(1, 4, 1, 16, D, 3, 2)
    ws, lacking = xpress.cache_workspace(c, 3), torch.zeros(1, dtype=torch.int32, device="cuda")
    xpress.cache_extend(c, 1, lacking=lacking, ws=ws)
    q, k = torch.zeros(3, D, device="cuda"), torch.zeros(3, D, device="cuda")
    v = torch.arange(3 * D, device="cuda").view(3, D).bfloat16()
    q[:, 5] = torch.tensor([1e14, 1e16, 1.0])
    k[:, 5] = torch.tensor([-1e15, -1e16, torch.finfo(torch.bfloat16).min])
    xpress.cache_append(c, 0, k.bfloat16(), v, B=1)
    out, lse = torch.full((3, D), 3.0, device="cuda").bfloat16(), torch.zeros(3, 1, device="cuda")
    for scale in (D ** -0.5, 1.0):
        xpress.block_attention(c, 0, q.bfloat16(), B=1, Hq=1, out=out, lse=lse, scale=scale,
                               ws=xpress.attention_workspace(c, 3, 1, 1))
        assert torch.equal(out[0], v[0]) and not out[1:].any()
        assert lse[1:].flatten().tolist() == [-math.inf] * 2
        want = -1e29 * scale  # (two bf16 roundings and two of the product)
        assert abs(float(lse[0]) / want - 1) <= 2 * 2.0 ** -8 + 2.0 ** -20


# (fp16's products end at 65504^2)
@pytest.mark.parametrize("dtype,size", [
    *((torch.bfloat16, x) for x in (1e3, 3e5, 1e7, 1e9, 1e11, 1e20, 1e28)),
    *((torch.float16, x) for x in (1e3, 3e5, 1e7, 1e9))])
@pytest.mark.parametrize("D,N,B,G,own,shared", [(64, 2, 1, 1, 40, 0), (128, 3, 4, 2, 700, 0),
                                                (256, 2, 3, 1, 100, 70), (128, 2, 16, 48, 90, 150)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(size, sign, D, N, B, G, own, shared, dtype):
    """Products q.k of up to `size`, exact in 32 bits, hundreds apart or equal: the largest share all."""
    page, keys = 16, shared + own
    g = torch.Generator().manual_seed(3)
    pages = -(-keys // page)
    # eight bits each of q and k: the products are exact, their product with log2(e) is not
    a = 129 / 128 * 2.0 ** math.floor(math.log2(size) / 2)
    steps = torch.randint(1, 5, (pages * page,), generator=g).float()
    if sign < 0:
        steps = 5 - steps
    steps += 11 / 32
    k = torch.zeros(1, pages, 1, page, D)
    k[0, :, 0, :, 3] = (sign * steps * 2.0 ** math.floor(math.log2(size / a / 5))).view(pages, page)
    v = torch.randn(1, pages, 1, page, D, generator=g)
    k, v = k.to(dtype), v.to(dtype)
    q = torch.zeros(N * B, G * D)
    q[:, 3::D] = a
    assert bool(q.to(dtype).float().eq(q).all()) and float(k.float().abs().max()) * a <= size * 1.01
    c = xpress.Cache(k=k.cuda(), v=v.cuda(),
                     table=torch.arange(pages, dtype=torch.int32, device="cuda").repeat(N, 1),
                     length=torch.full((N,), keys, dtype=torch.int32, device="cuda"),
                     ref=torch.full((pages,), N, dtype=torch.int32, device="cuda"))
    out = torch.empty(N * B, G * D, dtype=dtype, device="cuda")
    lse = torch.empty(N * B, G, device="cuda")
    xpress.block_attention(c, 0, q.to(dtype).cuda(), B=B, Hq=G, out=out, lse=lse, shared=shared,
                           scale=1.0, ws=xpress.attention_workspace(c, N, B, G))
    kk = k[0, :, 0, :, 3].double().flatten() * a
    vv = v[0, :, 0].double().reshape(-1, D)
    for b in range(B):
        see = keys - B + b + 1
        s = kk[:see]
        p = torch.exp(s - s.max())
        assert int((p > 1e-30).sum()) == int((p == 1).sum())
        want = (p / p.sum()) @ vv[:see]
        mass = (p / p.sum()) @ vv[:see].abs()
        # the result's rounding, that of a common weight, 32-bit sums
        half = torch.finfo(dtype).eps / 2
        bound = half * want.abs() + mass * (half * (1 + half) + (keys + 8) * 2.0 ** -24) + 2.0 ** -24
        rows = slice(b, None, B)
        got = out.view(N * B, G, D)[rows].cpu().double()
        assert bool(((got - want).abs() <= bound).all()), b
        lw = float(s.max() + math.log(p.sum()))
        assert bool(((lse[rows].cpu().double() - lw).abs() <= abs(lw) * 2.0 ** -22 + 2.0 ** -20).all()), b
