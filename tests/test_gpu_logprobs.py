"""Token log probabilities on the GPU against their definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import xpress
from tests.gpu_helpers import log

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    xpress.lib()
    torch.cuda.set_device(0)


def oracle(x, token, t, top):
    """One row: (logprob, entropy, rank, ids, values, slack of a log probability, of the entropy)."""
    V = len(x)
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max()
    order = np.lexsort((np.arange(V), -x))
    greedy = not t > 0
    logp = np.full(V, -np.inf)
    entropy, slack, eslack = 0.0, 0.0, 0.0
    if greedy:
        if m > -np.inf:
            logp[order[0]] = 0.0
    elif m > -np.inf:
        with np.errstate(invalid="ignore", over="ignore"):
            z = np.where(x == m, 0.0, (x - m) / t if m < np.inf else -np.inf)
            z = np.where(x == -np.inf, -np.inf, z)
            w = np.exp(z)
        S = w.sum()
        logp = z - math.log(S)
        logp[logp < -3.4028236e38] = -np.inf  # half a step past the lowest 32-bit number
        p = w / S
        lz = np.where(p > 0, -z, 0.0)
        entropy = float(math.log(S) + (p * lz).sum())
        # 32 bits: an exponent is off by three roundings (the difference, its scale, their product), a
        # weight by 2 more units, a chunk's sum by 40 additions; joined and finished in 64
        u, z1, z2 = 2.0 ** -24, float((p * lz).sum()), float((p * lz * lz).sum())
        slack = u * (3 * z1 + 44)
        eslack = slack + u * (3 * z2 + 47 * z1)
    ids = np.full(top, -1)
    values = np.full(top, -np.inf)
    ids[:min(top, V)] = order[:top]
    values[:min(top, V)] = logp[order[:top]]
    if 0 <= token < V:
        return logp[token], entropy, int((x > x[token]).sum()), ids, values, slack, eslack
    return -np.inf, entropy, -1, ids, values, slack, eslack


def outputs(rows, top):
    d = dict(logprob=torch.full((rows,), 3.0, device="cuda"),
             entropy=torch.full((rows,), 3.0, device="cuda"),
             rank=torch.full((rows,), 3, dtype=torch.int32, device="cuda"))
    if top:
        d["top_ids"] = torch.full((rows, top), 3, dtype=torch.int64, device="cuda")
        d["top_logprobs"] = torch.full((rows, top), 3.0, device="cuda")
    return d


def check(x, token, temperature, top, got, what="", entropy=True):
    """x: [N*B, V] as it was given; token [N, B]; temperature [N] or None."""
    N, B = token.shape
    got = {k: v.cpu().double().numpy() for k, v in got.items()}
    half = 2.0 ** -24
    worst = 0.0
    for r in range(N * B):
        tok = int(token[r // B, r % B])
        where = f"{what} row {r}"
        if tok < 0:
            assert got["logprob"][r] == 0 and got["entropy"][r] == 0 and got["rank"][r] == -1, where
            if top:
                assert (got["top_ids"][r] == -1).all() and (got["top_logprobs"][r] == -np.inf).all()
            continue
        t = 1.0 if temperature is None else float(np.float32(temperature[r // B]))
        l, e, rank, ids, values, slack, eslack = oracle(x[r].double().numpy(), tok, t, top)
        for name, want, give in (("logprob", l, slack), ("entropy", e, eslack))[:1 + entropy]:
            far = 0.0 if got[name][r] == want else abs(got[name][r] - want)
            bound = half * abs(want) + give if math.isfinite(want) else 0.0
            assert far <= bound, (where, name, got[name][r], want, bound)
            worst = max(worst, far / bound if bound else 0.0)
        assert got["rank"][r] == rank, where
        if top:
            assert np.array_equal(got["top_ids"][r], ids), (where, got["top_ids"][r], ids)
            same = got["top_logprobs"][r] == values
            with np.errstate(invalid="ignore"):
                far = np.abs(got["top_logprobs"][r] - values)
            assert (same | (far <= half * np.abs(values) + slack)).all(), where
    log(f"  {what}: worst error {worst:.3f} of the bound")


def run(x, token, temperature, top, pad=0, shift=0, ws=None):
    """x [N*B, V] on the device with a row stride of V + pad, `shift` elements past an alignment."""
    rows, V = x.shape
    hold = torch.full((rows * (V + pad) + shift,), 99.0, dtype=x.dtype, device="cuda")
    view = hold[shift:].view(rows, V + pad)[:, :V]
    view.copy_(x)
    out = outputs(rows, top)
    ws = xpress.logprobs_workspace(rows, V, top) if ws is None else ws
    ws.fill_(0xFF)
    t = None if temperature is None else torch.tensor(temperature, device="cuda")
    xpress.token_logprobs(view, token.cuda(), temperature=t, ws=ws, **out)
    torch.cuda.synchronize()
    return out


def logits(rows, V, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, V, generator=g) * 2
    if kind == "ties":  # few values
        x = torch.randint(-2, 3, (rows, V), generator=g).float()
    elif kind == "equal":
        x = torch.full((rows, V), -1.5)
    elif kind == "rising":
        x = torch.arange(V).float().expand(rows, V) * (8.0 / V)
    elif kind == "falling":
        x = -torch.arange(V).float().expand(rows, V) * (8.0 / V)
    elif kind == "large":
        x = x * (1e4 if dtype == torch.float16 else 1e30)
    return x.to(dtype).contiguous()


SIZES = [(1, 1, 0), (5, 7, 3), (31, 4, 1), (32, 8, 0), (33, 64, 5), (100, 64, 7), (8191, 20, 1),
         (8192, 5, 0), (8200, 64, 3), (20011, 20, 0), (151936, 20, 2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,top,pad", SIZES)
def test_against_the_definition(V, top, pad, dtype):
    log(f"log probabilities V={V} top={top} {dtype}")
    N, B = 3, 2
    x = logits(N * B, V, dtype, V)
    token = torch.tensor([[0, V - 1], [-1, V // 2], [V, V // 3]])
    for shift in (0, 1, 3):
        check(x, token, None, top, run(x, token, None, top, pad, shift), f"V {V} shift {shift}")
    temps = [0.7, 0.0, 2.5]
    check(x, token, temps, top, run(x, token, temps, top, pad), f"V {V} temperatures")


@pytest.mark.parametrize("kind", ["ties", "equal", "rising", "falling", "large"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [77, 30000])
def test_rows_of_many_kinds(V, dtype, kind):
    x = logits(4, V, dtype, 5, kind)
    token = torch.tensor([[3, V - 1], [0, 40]])
    for top in (0, 1, 20, 64):
        for temps in (None, [0.0, 0.5]):
            check(x, token, temps, top, run(x, token, temps, top, 3, 1), f"{kind} top {top} {temps}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
def test_logits_that_are_not_finite(dtype):
    V = 9000
    x = logits(10, V, dtype, 6)
    x[0, 5:] = -math.inf
    x[1] = -math.inf  # no weight at all
    x[2, ::7] = math.nan
    x[3] = math.nan
    x[4, [10, 8500]] = math.inf
    x[5, 3] = math.inf
    x[6, 100:] = -math.inf
    x[6, :100] = math.nan
    x[6, 42] = 1.0  # one id alone
    x[7, ::3] = -math.inf
    x[8, 0] = -0.0
    x[8, 1:] = 0.0
    x[9, 8999] = math.inf
    x[9, 17] = math.nan
    token = torch.tensor([[2], [0], [7], [9], [8500], [4], [42], [0], [1], [17]])
    for temps in (None, [0.8] * 10, [0.0] * 10):
        for top in (0, 3, 64):
            check(x, token, temps, top, run(x, token, temps, top), f"not finite {temps and temps[0]}")
    token = torch.tensor([[6], [1], [6], [1], [2], [3], [0], [1], [0], [8999]])
    check(x, token, None, 8, run(x, token, None, 8), "not finite, other tokens")


def test_temperatures_of_any_value():
    V = 1000
    x = logits(9, V, torch.float32, 7)
    token = torch.arange(9)[:, None] * 11
    temps = [math.inf, 1e-40, -1.0, math.nan, 1e30, 1e-3, 0.0, 3e38, 1e-6]
    check(x, token, temps, 10, run(x, token, temps, 10), "temperatures")
    x[:, ::2] = -math.inf
    check(x, token, temps, 10, run(x, token, temps, 10), "temperatures, half the ids")


def test_best_groups_that_lie_together():
    """Very many ids whose best are far apart by the same step: more keys than the list of the
    selection holds."""
    V = 256 * 32 * 64 + 100
    g = torch.Generator().manual_seed(8)
    x = torch.randn(2, V, generator=g)
    at = torch.arange(63)[:, None] + 256 * torch.arange(64)[None]  # groups of 63 of 256 threads
    x[:, at.reshape(-1) * 32 + 5] = 10 + torch.rand(2, 63 * 64, generator=g)
    token = torch.tensor([[5], [77]])
    check(x, token, None, 64, run(x, token, None, 64), "together")
    check(x, token, None, 3, run(x, token, None, 3), "together, three")


def test_a_part_of_the_outputs_and_no_tokens():
    V, top = 5000, 4
    x = logits(6, V, torch.bfloat16, 9).cuda()
    token = torch.tensor([[1, 2, 3], [4, -1, 6]])
    full = run(x.cpu(), token, None, top)
    ws = xpress.logprobs_workspace(6, V, top)
    for name in ("logprob", "entropy", "rank"):
        out = outputs(6, 0)
        xpress.token_logprobs(x, token.cuda(), ws=ws, **{name: out[name]})
        assert torch.equal(out[name], full[name])
    out = outputs(6, top)
    xpress.token_logprobs(x, ws=ws, entropy=out["entropy"], top_ids=out["top_ids"],
                          top_logprobs=out["top_logprobs"])
    every = torch.tensor([[1, 2, 3], [4, 5, 6]])
    whole = run(x.cpu(), every, None, top)
    for name in ("entropy", "top_ids", "top_logprobs"):
        assert torch.equal(out[name], whole[name])
    with pytest.raises(xpress.XpressError, match="token is NULL"):
        xpress.token_logprobs(x, ws=ws, logprob=out["logprob"])
    with pytest.raises(ValueError, match="together"):
        xpress.token_logprobs(x, ws=ws, top_ids=out["top_ids"])
    with pytest.raises(ValueError, match="top"):
        xpress.token_logprobs(x, ws=ws, top_ids=out["top_ids"], top_logprobs=out["top_logprobs"][:, :2])
    with pytest.raises(TypeError, match="ws"):
        xpress.token_logprobs(x, ws=ws.cpu())


def test_streams_and_captured_calls():
    """The same bits on another stream and in replays, whose tokens and logits change, with eager work in
    between."""
    N, B, V, top = 4, 3, 40000, 20
    x = logits(N * B, V, torch.bfloat16, 10).cuda()
    token = torch.randint(V, (N, B)).cuda()
    temps = torch.tensor([0.5, 0.0, 1.0, 2.0], device="cuda")
    ws, mine = xpress.logprobs_workspace(N * B, V, top), outputs(N * B, top)
    other = outputs(N * B, top)

    def call(out, ws=ws):
        xpress.token_logprobs(x, token, temperature=temps, ws=ws, **out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(mine)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(mine)
    for rep in range(4):
        g = torch.Generator().manual_seed(rep)
        x.copy_(torch.randn(N * B, V, generator=g).mul_(3))
        token.copy_(torch.randint(-1 if rep else 0, V, (N, B), generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ws.fill_(0xFF)
        call(other)
        torch.cuda.synchronize()
        for name in mine:
            assert torch.equal(mine[name], other[name]), (rep, name)
        check(x.cpu(), token.cpu(), temps.cpu(), top, mine, f"replay {rep}")


@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, 0x7f81), (torch.float16, 0x7c01),
                                        (torch.float32, 0x7f800001)], ids=["bf16", "f16", "f32"])
def test_signalling_nans(dtype, bits):
    V, top = 20000, 20
    x = logits(4, V, dtype, 11)
    word = torch.int32 if dtype == torch.float32 else torch.int16
    raw = x.view(word)
    g = torch.Generator().manual_seed(3)
    raw[0, torch.randint(V, (50,), generator=g)] = bits
    raw[1, ::2] = bits
    raw[2, 8192:] = bits | (-1 << (31 if dtype == torch.float32 else 15))
    raw[3] = bits
    token = torch.tensor([[5, 7], [9, 11]])
    for temps in (None, [0.0, 0.7]):
        for t in (0, top):
            check(x, token, temps, t, run(x, token, temps, t, 1, 1), f"signalling {temps} {t}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
def test_vocabularies_that_are_masked(dtype):
    """A few allowed ids among -inf or the type's lowest value; chunks of nothing else."""
    V, top = 151936, 20
    x = logits(6, V, dtype, 12)
    allowed = [range(0), range(7), range(100000, 100040), range(0, V, 9973), range(8192, 16384), range(V - 3, V)]
    low = torch.finfo(dtype).min
    for r, ids in enumerate(allowed):
        keep = torch.zeros(V, dtype=torch.bool)
        keep[list(ids)] = True
        x[r] = torch.where(keep, x[r], low if r % 2 else -math.inf)
    token = torch.tensor([[0, 3], [100002, 9973], [9000, V - 1]])
    for temps in (None, [0.6, 0.0, 1.5]):
        check(x, token, temps, top, run(x, token, temps, top), f"masked {temps}")


def test_two_calls_at_once_and_rows_past_32_bits():
    """Two streams with a workspace each; rows whose last element lies past 2^32 bytes."""
    V, top, ld = 1000, 5, 1 << 29
    hold = torch.empty(5 * ld, dtype=torch.bfloat16, device="cuda")
    view = hold.view(5, ld)[:, :V]
    x = logits(5, V, torch.bfloat16, 13)
    view.copy_(x)
    token = torch.tensor([[1], [2], [3], [4], [999]])
    d = token.cuda()
    outs = [outputs(5, top) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [xpress.logprobs_workspace(5, V, top) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, ws in zip(streams, outs, spaces):
            with torch.cuda.stream(s):
                xpress.token_logprobs(view, d, ws=ws, **o)
    torch.cuda.synchronize()
    for o in outs:
        check(x, token, None, top, o, "at once")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_very_many_equal_ids_behind_others(dtype):
    """More groups whose best are equal than the selection's list holds, beginning far into the row, with
    fewer better ones than there are places, as many, and more."""
    V = 400000
    g = torch.Generator().manual_seed(15)
    x = (-5 - torch.rand(4, V, generator=g)).to(dtype)
    x[:, 200000:] = 1.0
    for r, better in enumerate((0, 10, 64, 200)):
        at = torch.randperm(V, generator=g)[:better]
        x[r, at] = (2 + torch.rand(better, generator=g)).to(dtype)
    token = torch.tensor([[200000], [5], [V - 1], [399000]])
    for top in (1, 64):
        check(x, token, None, top, run(x, token, None, top, 5, 1), f"equal behind others {dtype} {top}")


def test_best_ids_that_share_groups():
    """All ids of a few groups before all others: more keys at the end than are counted without a search."""
    V, top = 151936, 64
    x = logits(2, V, torch.float32, 16) - 30
    for group in range(60):
        x[0, 32 * 70 * group:32 * 70 * group + 32] += 40
    x[1, 1000:5000] += 40
    token = torch.tensor([[0], [1234]])
    for t in (top, 20, 1):
        check(x, token, None, t, run(x, token, None, t), f"shared groups {t}")
