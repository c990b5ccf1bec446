"""Draft verification on the GPU against its definition in 64 bits: ids and counts are equal."""
import math

import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import xpress
from tests.gpu_helpers import log
from tests.serve_oracle import verify

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    xpress.lib()
    torch.cuda.set_device(0)


def run(logits, blk, *, q=None, ws=None, **lists):
    N, B = blk.shape
    dev = {k: None if v is None else torch.as_tensor(v).cuda() for k, v in lists.items()}
    out = torch.full((N, B), 77, dtype=torch.int64, device="cuda")
    accepted = torch.full((N,), 77, dtype=torch.int32, device="cuda")
    drop = torch.full((N,), 77, dtype=torch.int32, device="cuda")
    ws = xpress.verify_workspace(N, B, logits.shape[1]) if ws is None else ws
    xpress.verify_draft(logits, torch.as_tensor(blk).cuda(), q=q, out=out, accepted=accepted,
                        drop=drop, ws=ws, **dev)
    torch.cuda.synchronize()
    assert torch.equal(drop, B - 1 - accepted)
    return out.cpu().numpy(), accepted.cpu().numpy()


def draw(N, B, V, seed, agree=0.7):
    """Logits that mostly agree with the drafts, drafts, uniform numbers, temperatures, lengths."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((N * B, V)).astype(np.float32) * 2
    blk = rng.integers(0, V, (N, B))
    for n in range(N):
        for s in range(B - 1):
            if rng.random() < agree:
                x[n * B + s, blk[n, s + 1]] = math.log(V) + 4 + rng.standard_normal()
    u = rng.random((N, B)).astype(np.float32)
    temperature = rng.choice([0.0, 0.5, 1.0, 1.7], N).astype(np.float32)
    return rng, x, blk, u, temperature, rng.integers(0, B, N).astype(np.int32)


def strided(x, dtype, pad):
    """x as a GPU tensor whose rows start at any element."""
    hold = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=dtype, device="cuda")
    hold[:, :x.shape[1]] = torch.as_tensor(x).cuda().to(dtype)
    return hold[:, :x.shape[1]]


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,B,V,pad", [(1, 2, 7, 0), (3, 5, 1000, 3), (9, 16, 5003, 0),
                                       (2, 16, 50257, 0), (1, 64, 333, 1), (4, 1, 100, 0),
                                       (5, 3, 1, 2), (70, 4, 257, 0)])
def test_point_drafts(N, B, V, pad, dtype):
    log(f"verify N={N} B={B} V={V} pad={pad} {dtype}")
    for seed in range(3):
        _, x, blk, u, temperature, lengths = draw(N, B, V, seed)
        t = strided(x, dtype, pad)
        for dl in (None, lengths):
            want = verify(f64(t), blk, dl, None, temperature, u)
            got = run(t, blk, u=u, temperature=temperature, draft_len=dl)
            assert np.array_equal(got[1], want[1]), seed
            assert np.array_equal(got[0], want[0]), seed


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["qbf16", "qf16", "qf32"])
@pytest.mark.parametrize("N,B,V,pad", [(3, 5, 1000, 1), (8, 16, 5003, 0), (1, 16, 50257, 3),
                                       (40, 2, 65, 0)])
def test_drawn_drafts(N, B, V, pad, q_dtype):
    log(f"verify with q N={N} B={B} V={V} {q_dtype}")
    for seed in range(3):
        rng, x, blk, u, temperature, lengths = draw(N, B, V, 10 + seed)
        t = strided(x, torch.bfloat16, pad)
        noisy = x.reshape(N, B, V)[:, :-1].reshape(-1, V) + rng.standard_normal((N * (B - 1), V))
        q = torch.softmax(torch.as_tensor(noisy), -1).numpy()
        q = strided(q, q_dtype, 2 * pad)
        want = verify(f64(t), blk, lengths, f64(q), temperature, u)
        got = run(t, blk, q=q, u=u, temperature=temperature, draft_len=lengths)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0]), seed


@pytest.mark.parametrize("q_dtype", [None, torch.float32], ids=["point", "drawn"])
@pytest.mark.parametrize("V", [97, 8200, 20011])
def test_many_draws(q_dtype, V):
    """Many blocks, a refusal in most, weights of exactly nothing between the others (masked ids, and
    ids where the drafts' probability is the larger): every token is the definition's."""
    N, B = 60000 // V + 40, 2
    rng, x, blk, u, _, _ = draw(N, B, V, 77, agree=0.2)
    x[:, rng.random(V) < 0.4] = -math.inf
    t = strided(x, torch.float32, 1)
    q = None
    if q_dtype is not None:
        noisy = x.reshape(N, B, V)[:, 0] + 0.5 * rng.standard_normal((N, V)).astype(np.float32)
        q = strided(torch.softmax(torch.as_tensor(noisy), -1).numpy(), q_dtype, 3)
    temperature = rng.choice([0.7, 1.0], N).astype(np.float32)
    want = verify(f64(t), blk, None, None if q is None else f64(q), temperature, u)
    got = run(t, blk, q=q, u=u, temperature=temperature)
    assert (want[1] == 0).sum() > N / 10
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


def test_greedy_without_lists():
    """No temperature: argmax, lowest id on ties (also of -0 and +0)."""
    x = np.zeros((8, 900), np.float32) - 1
    x[:, 700] = x[:, 30] = x[:, 899] = 2.5
    x[5, 30] = -1
    x[6] = -0.0
    x[6, 450:] = 0.0
    blk = np.array([[0, 30, 30, 700], [0, 30, 700, 0]])
    out, accepted = run(strided(x, torch.bfloat16, 0), blk)
    assert out.tolist() == [[30, 30, 30, -1], [30, 700, 0, 30]]
    assert accepted.tolist() == [2, 3]


def test_rows_without_weight_infinities_and_nan():
    inf, nan = math.inf, math.nan
    V = 300
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6 * 2, V)).astype(np.float32)
    x[0] = -inf                      # nothing to draw from
    x[2] = nan
    x[4] = -inf
    x[4, 17] = -3.0                  # one id left
    x[6, 5] = x[6, 250] = inf        # two ids share all
    x[8, ::2] = nan
    x[10] = np.float32(torch.finfo(torch.bfloat16).min)  # the lowest value is a value
    blk = np.array([[0, 3], [0, 3], [0, 17], [0, 5], [0, 9], [0, 299]])
    u = np.array([[.5, .5], [.5, .5], [.99, .5], [.75, .75], [.9, .5], [.001, .999]], np.float32)
    for temperature in (None, np.full(6, 0.8, np.float32)):
        t = strided(x, torch.bfloat16, 0)
        want = verify(f64(t), blk, None, None, temperature, u)
        got = run(t, blk, u=u, temperature=temperature)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert got[0][:2].tolist() == [[-1, -1]] * 2
    assert got[0][3].tolist() == [250, -1]
    assert got[0][2, 0] == 17


def test_ends_of_the_unit_interval_and_drafts_outside():
    """u = 0 takes the first id with weight, u just below 1 the last; an id outside [0, V) never
    stands; a point draft that holds all the weight always does."""
    V = 2000
    x = np.full((4 * 2, V), -40.0, np.float32)
    x[0, 100] = x[0, 1900] = 0
    x[2] = x[0]
    x[4, 7] = 60.0
    x[6, 7] = 0.0
    blk = np.array([[0, 100], [0, 100], [0, 7], [0, V]])
    last = np.float32(1 - 2.0 ** -24)
    u = np.array([[last, 0], [last, last], [last, .5], [0, .5]], np.float32)
    t = strided(x, torch.float32, 0)
    temperature = np.ones(4, np.float32)
    want = verify(f64(t), blk, None, None, temperature, u)
    got = run(t, blk, u=u, temperature=temperature)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    # weights of exactly nothing: masked everywhere but two ids
    x[x == -40] = -math.inf
    t = strided(x, torch.float32, 0)
    got = run(t, blk, u=u, temperature=temperature)
    assert got[0].tolist() == [[1900, -1], [1900, -1], [7, got[0][2, 1]], [7, -1]]
    # the draft's probabilities equal the target's: what is left is nothing, the target is drawn
    q = torch.zeros(4, V, device="cuda")
    q[0, 100] = q[0, 1900] = 1.0
    got = run(t, blk, u=u, temperature=temperature, q=q)
    assert got[0][0].tolist() == [100, -1]


@pytest.mark.parametrize("bad", [-1.0, math.nan])
def test_temperatures_that_are_none(bad):
    _, x, blk, u, _, _ = draw(4, 3, 500, 1)
    t = strided(x, torch.float16, 0)
    got = run(t, blk, u=u, temperature=np.full(4, bad, np.float32))
    want = run(t, blk)
    assert np.array_equal(got[0], want[0])


def test_draws_follow_the_distribution():
    """20,000 draws from 6 ids, first token only: frequencies within 5 standard deviations of p,
    whichever probabilities the drafts came from."""
    V, N = 6, 20000
    rng = np.random.default_rng(3)
    logit = np.array([0.0, 1.0, -1.0, 2.0, 0.5, -3.0], np.float32)
    p = np.exp(logit.astype(np.float64))
    p /= p.sum()
    x = torch.as_tensor(np.tile(logit, (2 * N, 1))).cuda()
    q1 = rng.random(V)
    q1 = torch.as_tensor(q1 / q1.sum(), dtype=torch.float32)
    for q in (None, q1.expand(N, V).contiguous().cuda()):
        d = rng.choice(V, N, p=(q1.double() / q1.double().sum()).numpy()) if q is not None else np.full(N, 3)
        blk = np.stack([np.zeros(N, np.int64), d], 1)
        out, _ = run(x, blk, q=q, u=rng.random((N, 2)).astype(np.float32),
                     temperature=np.ones(N, np.float32))
        f = np.bincount(out[:, 0], minlength=V) / N
        assert (np.abs(f - p) <= 5 * np.sqrt(p * (1 - p) / N)).all(), f


def test_workspace_contents_streams_and_replays():
    """Twice the same ids whatever the workspace holds; a captured call picks up new logits; another
    stream."""
    N, B, V = 12, 8, 30011
    _, x, blk, u, temperature, lengths = draw(N, B, V, 2)
    _, x2, _, _, _, _ = draw(N, B, V, 9)
    t = strided(x, torch.bfloat16, 5)
    ws = xpress.verify_workspace(N, B, V)
    ws.fill_(0xFF)
    lists = dict(u=u, temperature=temperature, draft_len=lengths)
    want = run(t, blk, ws=ws, **lists)
    assert np.array_equal(run(t, blk, ws=ws, **lists)[0], want[0])
    dev = {k: torch.as_tensor(v).cuda() for k, v in lists.items()}
    b = torch.as_tensor(blk).cuda()
    out = torch.empty(N, B, dtype=torch.int64, device="cuda")
    acc = torch.empty(N, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        xpress.verify_draft(t, b, out=out, accepted=acc, ws=ws, **dev)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xpress.verify_draft(t, b, out=out, accepted=acc, ws=ws, **dev)
    first = t.clone()
    second = torch.as_tensor(x2).cuda().to(torch.bfloat16)
    for src in (first, second, first, second):
        t.copy_(src)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu().numpy(), acc.cpu().numpy()
        w = verify(f64(t), blk, lengths, None, temperature, u)
        assert np.array_equal(got[0], w[0]) and np.array_equal(got[1], w[1])


@pytest.mark.parametrize("drawn", [False, True], ids=["point", "drawn"])
@pytest.mark.parametrize("V", [1000, 20011])
def test_numbers_next_to_the_border(V, drawn):
    """u is p(d) / q(d) rounded to 32 bits, or a few steps beside it: the test is decided in 64 bits."""
    N, B = 41, 2
    rng, x, blk, u, _, _ = draw(N, B, V, 31, agree=1.0)
    t = strided(x, torch.float32, 0)
    temperature = rng.choice([0.7, 1.0, 1.6], N).astype(np.float32)
    q = None
    if drawn:
        noisy = x.reshape(N, B, V)[:, 0] + rng.standard_normal((N, V)) * 0.3
        q = strided(torch.softmax(torch.as_tensor(noisy), -1).numpy(), torch.float32, 0)
    y = f64(t).reshape(N, B, V)[:, 0] / temperature.astype(np.float64)[:, None]
    p = np.exp(y - y.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    i = np.arange(N)
    border = p[i, blk[:, 1]] / (1 if q is None else f64(q)[i, blk[:, 1]])
    steps = np.tile(np.array([0, 1, -1, 2, -3], np.int32), 9)[:N]
    u[:, 0] = np.minimum(border, 1 - 2.0 ** -20).astype(np.float32)
    u[:, 0] = (u[:, 0].view(np.int32) + steps).view(np.float32)
    want = verify(f64(t), blk, None, None if q is None else f64(q), temperature, u)
    got = run(t, blk, q=q, u=u, temperature=temperature)
    assert 0 < want[1].sum() < N
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


@pytest.mark.parametrize("V", [524289, 700001])
def test_long_vocabularies(V):
    rng, x, blk, u, _, _ = draw(3, 2, V, 12, agree=0.5)
    x[1, V - 2] = x[3, V - 1] = 14.0  # most of the weight at the end
    for dtype in (torch.bfloat16, torch.float32):
        t = strided(x, dtype, 1)
        for temperature in (np.array([0, 1, 0.5], np.float32), np.array([1, 0.8, 0], np.float32)):
            want = verify(f64(t), blk, None, None, temperature, u)
            got = run(t, blk, u=u, temperature=temperature)
            assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


def test_infinite_logits_in_several_chunks_and_infinite_temperature():
    inf, V = math.inf, 20011
    rng = np.random.default_rng(8)
    x = rng.standard_normal((8, V)).astype(np.float32)
    x[0, [5, 9000, 20010]] = inf
    x[2, [8191, 8192]] = inf
    x[2, 100:200] = math.nan
    blk = np.array([[0, 7], [0, 8192], [0, 3], [0, 4]])
    temperature = np.array([1, 1, inf, inf], np.float32)
    x[6, ::3] = -inf
    u = np.array([[0.5, 0.6], [0.4, 0.2], [0.9, 0.37], [0.5, 0.999]], np.float32)
    t = strided(x, torch.float32, 0)
    flat = f64(t)
    flat[4:] = np.where(np.isneginf(flat[4:]), -inf, 0)  # equal weights at an infinite temperature
    want = verify(flat, blk, None, None, np.ones(4, np.float32), u)
    got = run(t, blk, u=u, temperature=temperature)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])
