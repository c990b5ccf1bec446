"""Attention over 4 bits with few query rows: the ways in which its pairs of request and head are cut into
parts, each asserted to be the one that the call takes."""
import math

import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import xpress
from tests import few_plan
from tests import mx4_oracle as mx4
from tests.gpu_helpers import log
from tests.serve_oracle import attention, attention_bounds
from tests.test_gpu_mx4 import Case4, _gpu, i32  # noqa: F401 (a fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


class Rows:
    """N rows over the same pages, each in an order of its own behind `shared` common tokens."""

    def __init__(self, lengths, Hkv, D, dtype, *, shared=0, page=16, table=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        N, self.page, self.D, self.Hkv, self.dtype = len(lengths), page, D, Hkv, dtype
        self.lengths, self.shared = lengths, shared
        first, need = shared // page, -(-max(lengths) // page)
        pages = need + 13
        shape = (1, pages, Hkv, page, D)
        pools = [mx4.pool_of(torch.randn(shape, generator=g), dtype, v) for v in (False, True)]
        self.k, self.v = (mx4.pool_values(p, D, v)[0].float() for p, v in zip(pools, (False, True)))
        self.table = np.full((N, max(need, table or 0)), -1, np.int32)
        for r in range(N):
            order = first + (np.arange(need - first) * 5 + 7 * r) % (pages - first)
            if shared % page and need > first:  # the page that the prefix ends in
                order[0] = first
            self.table[r, :need] = np.concatenate([np.arange(first), order])[:need]
            self.table[r, -(-lengths[r] // page):] = -1
        self.c = xpress.Cache(k=pools[0].cuda(), v=pools[1].cuda(), table=i32(self.table), dtype=dtype,
                              length=i32(lengths), ref=i32(np.ones(pages)))

    def run(self, q, B, Hq, seq=None):
        N = len(self.lengths) if seq is None else len(seq)
        out = torch.full((N * B, Hq * self.D), 5.0, dtype=self.dtype, device="cuda")
        lse = torch.full((N * B, Hq), 5.0, device="cuda")
        ws = xpress.attention_workspace(self.c, N, B, Hq)
        ws.fill_(0xFF)
        xpress.block_attention(self.c, 0, q, B=B, Hq=Hq, N=N, seq=None if seq is None else i32(seq), out=out,
                               lse=lse, shared=self.shared, ws=ws)
        torch.cuda.synchronize()
        return out.cpu().double().view(N, B, Hq, self.D), lse.cpu().double().view(N, B, Hq)

    def check(self, B, G, picked, what):
        """All rows at once: the picked ones against the definition, and every one against a call of a few
        rows (each is off by no more than its bound, so the two by no more than both)."""
        N, Hq, D = len(self.lengths), self.Hkv * G, self.D
        g = torch.Generator().manual_seed(1)
        q = torch.randn(N * B, Hq * D, generator=g).to(self.dtype)
        d = q.cuda()
        out, lse = self.run(d, B, Hq)
        again, lse_again = self.run(d, B, Hq)
        assert torch.equal(out, again) and torch.equal(lse, lse_again)
        tokens = [r * B + b for r in picked for b in range(B)]
        want, wl, mass, size = attention(self.k, self.v, self.table, self.lengths, self.page, q[tokens], picked,
                                         B, Hq, D ** -0.5)
        bound, lse_bound = attention_bounds(want, mass, size, max(self.lengths), D, self.dtype)
        got, gl = out[picked].reshape(want.shape), lse[picked].reshape(wl.shape)
        assert not bool(got.isnan().any())
        worst = float(((got - want).abs() / bound).max())
        log(f"  {what}: worst error {worst:.3f} of the bound")
        assert worst <= 1, what
        sees = wl > -math.inf
        assert bool((gl[~sees] == -math.inf).all())
        assert bool(((gl - wl).abs() <= lse_bound + wl.abs() * 2.0 ** -22 + 2.0 ** -18)[sees].all())
        most = float(self.v.abs().max())
        half = torch.finfo(self.dtype).eps / 2
        for at in range(0, N, 16):
            seq = list(range(at, min(at + 16, N)))
            few, few_lse = self.run(d[at * B:], B, Hq, seq)
            far = (few - out[seq]).abs()
            assert bool((far <= 2 * (half * few.abs() + most * (half * (1 + half) + 2.0 ** -10))).all()), at
            assert torch.equal(few_lse == -math.inf, lse[seq] == -math.inf)
            far = torch.where(few_lse == -math.inf, 0.0, (few_lse - lse[seq]).abs())
            assert float(far.max()) <= 2.0 ** -10


def uneven(N, long, shared=0):
    """Rows of no, one and a few tokens, and some long ones among them."""
    lengths = [shared + (0, 1, 5, 31, 32, 33, 64, 70)[(3 * i) % 8] for i in range(N)]
    at = [0, 1, N // 3, N // 2, N - 2, N - 1]
    for r, n in zip(at, long):
        lengths[r] = shared + n
    return lengths, at + [2, 3, 4, 5, 7, N // 2 + 1, N - 3]


# D, rows a request, K heads, query heads of each, tokens of a block, tokens that a table holds
BY_PART = [
    (64, 400, 8, 4, 1, 0),  # one token a request, a wave a part
    (64, 230, 14, 5, 6, 0),  # 30 rows: two row tiles
    (64, 200, 8, 4, 16, 1024),  # 64 rows: two waves a part
    (128, 300, 8, 5, 1, 0),
    (128, 210, 10, 4, 8, 0),
    (128, 140, 8, 3, 16, 512),
    (256, 300, 8, 4, 1, 0),
    (256, 150, 8, 4, 5, 0),  # 20 rows: two waves a part
    (256, 80, 8, 4, 16, 512),  # 64 rows: four
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("D,N,Hkv,G,B,table", BY_PART)
def test_more_pairs_than_parts(D, N, Hkv, G, B, table, dtype):
    """Each part says which pair begins in it and goes on, and none where it has no tiles."""
    page, R = 16, B * G
    log(f"more pairs than parts: D {D}, {N} x {Hkv} pairs, {R} rows {dtype}")
    lengths, picked = uneven(N, [900, 901, 640, 1, 513, 880])
    x = Rows(lengths, Hkv, D, dtype, page=page, table=table // page, seed=D + R)
    assert N <= few_plan.REQUESTS and N * Hkv > few_plan.parts(D, R)
    assert few_plan.taken(D, R, N, Hkv, x.table.shape[1] * page)
    x.check(B, G, picked, f"D {D}")


@pytest.mark.parametrize("D,Hkv,G", [(64, 8, 4), (128, 8, 4), (256, 8, 4)])
def test_parts_without_tiles(D, Hkv, G):
    """More pairs than parts, of one tile each but for a few: the least that a part takes leaves the last
    parts without any; and no row with a token at all."""
    N = few_plan.parts(D, G) // Hkv + 1
    lengths, picked = [(3 * i) % 33 for i in range(N)], [0, 1, 10, 11, N - 1]
    x = Rows(lengths, Hkv, D, torch.bfloat16)
    assert N * Hkv > few_plan.parts(D, G)
    x.check(1, G, picked, f"one tile each, D {D}")
    x = Rows([1] * N, Hkv, D, torch.bfloat16)
    x.c.length.zero_()
    out, lse = x.run(torch.ones(N, Hkv * G * D, dtype=torch.bfloat16, device="cuda"), 1, Hkv * G)
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("D,Hkv,G,B,dtype,shared", [
    (64, 1, 4, 16, torch.float16, 0), (64, 2, 4, 5, torch.bfloat16, 64), (128, 1, 4, 8, torch.float16, 0),
    (128, 1, 3, 16, torch.bfloat16, 0), (128, 2, 2, 8, torch.bfloat16, 128), (256, 1, 4, 5, torch.float16, 0),
    (256, 1, 3, 16, torch.bfloat16, 0), (256, 1, 5, 1, torch.float16, 64)])
def test_a_pair_a_part(D, Hkv, G, B, dtype, shared):
    """More requests than are cut: one or two row tiles, one to four waves a part."""
    N, page, R = 4097, 16, B * G
    log(f"a pair a part: D {D}, {R} rows, shared {shared}, {dtype}")
    lengths, picked = uneven(N, [300, 301, 64, 1, 65, 130], shared)
    lengths[5] = 0
    x = Rows(lengths, Hkv, D, dtype, shared=shared, page=page, seed=D + R)
    assert N > few_plan.REQUESTS
    assert few_plan.taken(D, R, N, Hkv, x.table.shape[1] * page - shared)
    x.check(B, G, picked, f"D {D}")


@pytest.mark.parametrize("D,ld", [(64, 8192), (128, 2048)])
@pytest.mark.parametrize("B,G,shared", [(13, 3, 100), (33, 1, 70), (16, 4, 192)])
def test_own_parts_of_two_waves_beside_a_shared_part(D, ld, B, G, shared):
    """Requests of 33 to 64 query rows a head under tables for long contexts, all and in a list."""
    N, Hkv, page, R = 8, 4, 16, B * G
    lengths = [shared + n for n in (1, 40, 0, 33, 300, 97, 64, 31)]
    lengths[2] = 0
    x = Case4(lengths=lengths, shared=shared, B=B, Hkv=Hkv, G=G, D=D, page=page, seed=81)
    wide = np.full((N, ld), -1, np.int32)
    wide[:, :x.table.shape[1]] = x.table
    x.table = wide
    assert few_plan.waves(D, R) == 2 and shared >= 64
    order = [6, 1, 4]
    assert few_plan.taken(D, R, len(order), Hkv, ld * page - shared // 64 * 64)
    c = x.cache()
    x.check(x.run(c), what=f"D {D}, {R} rows")
    x.check(x.run(c, seq=i32(order), rows=order), rows=order, what="a list")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("N,Hkv,G,B,table", [(400, 2, 4, 1, 0), (110, 2, 5, 3, 0), (100, 1, 4, 8, 0),
                                             (40, 2, 4, 16, 4096)])
def test_own_parts_behind_wide_items(N, Hkv, G, B, table, dtype):
    """So many query rows that the shared part is a launch of its own, in wide items."""
    D, page, shared, R = 128, 16, 200, B * G
    log(f"own parts behind wide items: {N} x {Hkv} pairs, {R} rows {dtype}")
    lengths, picked = uneven(N, [600, 601, 64, 1, 65, 330], shared)
    lengths[5], lengths[7] = 0, 100  # a row that does not hold the prefix
    x = Rows(lengths, Hkv, D, dtype, shared=shared, page=page, table=table // page, seed=R)
    assert N * R >= 1536 and few_plan.taken(D, R, N, Hkv, x.table.shape[1] * page - 192)
    x.check(B, G, picked, f"{R} rows")


def test_two_captured_calls_share_a_workspace():
    """Decoding and blocks, cut in different ways, replayed in turn with eager calls between them."""
    Hkv, D, G, dtype = 4, 128, 4, torch.bfloat16
    lengths, _ = uneven(520, [900, 901, 640, 1, 513, 880])
    x = Rows(lengths, Hkv, D, dtype)
    Hq = Hkv * G
    calls = []
    for N, B in ((520, 1), (300, 4)):
        assert (N * Hkv > few_plan.parts(D, B * G)) == (B == 1)
        q = torch.randn(N * B, Hq * D, generator=torch.Generator().manual_seed(B)).to(dtype).cuda()
        calls.append((N, B, q, torch.zeros(N * B, Hq * D, dtype=dtype, device="cuda")))
    ws = max((xpress.attention_workspace(x.c, N, B, Hq) for N, B, _, _ in calls), key=torch.Tensor.numel)
    want = [x.run(q, B, Hq, list(range(N)))[0] for N, B, q, _ in calls]
    graphs = []
    for N, B, q, out in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            xpress.block_attention(x.c, 0, q, B=B, Hq=Hq, N=N, out=out, ws=ws)
    for turn in (0, 1, 1, 0, 1, 0):
        out = calls[turn][3].fill_(3.0)
        torch.cuda.synchronize()
        graphs[turn].replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu().double().view(want[turn].shape), want[turn]), turn
        other = x.run(calls[turn][2], calls[turn][1], Hq, list(range(calls[turn][0])))[0]
        assert torch.equal(other, want[turn])
        ws.fill_(0xFF if turn else 0x01)
