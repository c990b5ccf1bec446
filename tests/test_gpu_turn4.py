"""Whole turns with a cache of 4 bits and the tokens' log probabilities: every call of a decoded prompt
against plain oracles; and such a turn captured and replayed."""
import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import synth, upload, xpress
from jacobi_block_refiner_amd.draft_turn import Decoder, Target, main
from tests import mx4_oracle as mx4
from tests.gpu_helpers import log
from tests.serve_oracle import attention, attention_bounds, verify
from tests.test_gpu_logprobs import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("samples,prompt,page,temperature,top", [(1, 3, 16, 0.0, 0), (3, 41, 32, 1.0, 5)])
def test_turns_with_a_cache_of_4_bits(samples, prompt, page, temperature, top, monkeypatch):
    inp = synth.make_inputs(1).rounded_bf16()
    B, turns, most = inp.wl.B, 4, prompt + 5 * inp.wl.B
    target = Target(inp.wl.V, inp.wl.H, most=most)
    dec = Decoder(target, upload.weights(inp), samples, page=page, most=most - B, bits=4, top=top,
                  temperature=temperature)
    assert dec.cache.k.dtype == torch.uint8
    # what every row holds, written beside the calls
    kept = torch.zeros(2, len(target.layers), samples, target.Hkv, most, target.D)
    append, attend = xpress.cache_append, xpress.block_attention
    worst = [0.0]

    def shadowed_append(cache, layer, k, v, *, N, B, lacking):
        append(cache, layer, k, v, N=N, B=B, lacking=lacking)
        for side, x in ((0, k), (1, v)):
            held = mx4.values(*mx4.quantise(x.cpu().view(N, B, target.Hkv, target.D), torch.bfloat16))
            for i in range(N):
                at = int(cache.length[i]) - B
                rows = slice(None) if N == 1 else i  # (the prompt is every row's)
                kept[side, layer, rows, :, at:at + B] = held[i].transpose(0, 1).float()

    def checked_attend(cache, layer, q, *, N, B, Hq, shared, out, ws):
        attend(cache, layer, q, N=N, B=B, Hq=Hq, shared=shared, out=out, ws=ws)
        lengths = cache.length[:N].tolist()
        want, _, mass, size = attention(kept[0, layer], kept[1, layer], [[i] for i in range(N)], lengths,
                                        most, q.cpu(), range(N), B, Hq, target.D ** -0.5)
        bound, _ = attention_bounds(want, mass, size, most, target.D, torch.bfloat16)
        far = (out.cpu().double().view(want.shape) - want).abs() / bound
        worst[0] = max(worst[0], float(far.max()))
        assert worst[0] <= 1, (layer, N, B)
        return out

    monkeypatch.setattr(xpress, "cache_append", shadowed_append)
    monkeypatch.setattr(xpress, "block_attention", checked_attend)
    dec.prompt(torch.randint(inp.wl.V, (prompt,), generator=torch.Generator().manual_seed(3)).cuda())
    for turn in range(turns):
        t = dec.turn()
        assert int(dec.lacking.item()) == 0
        temps = np.full(samples, temperature, np.float32)
        out, accepted = verify(t.logits.double().cpu().numpy(), t.blk.cpu().numpy(), None, None, temps,
                               t.u.cpu().numpy())
        assert np.array_equal(out, t.out.cpu().numpy())
        assert np.array_equal(accepted, t.accepted.cpu().numpy())
        got = dict(logprob=t.logprob, entropy=t.entropy, rank=t.rank)
        if top:
            got.update(top_ids=t.top_ids, top_logprobs=t.top_logprobs)
        check(t.logits.cpu(), t.out.cpu(), temps, top,
              {k: v.reshape(samples * B, *v.shape[2:]) for k, v in got.items()}, f"turn {turn}")
    log(f"turns over 4 bits: attention's worst error {worst[0]:.3f} of the bound")
    # one sample kept and compacted, then read back: the values that were written
    keep = samples - 1
    n = int(dec.cache.length[keep])
    dec.keep(keep)
    width = target.Hkv * target.D
    k, v = (torch.empty(n, width, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    seq = torch.tensor([keep], dtype=torch.int32, device="cuda")
    for layer in range(len(target.layers)):
        xpress.cache_read(dec.cache, layer, k, v, B=n, seq=seq)
        for side, x in ((0, k), (1, v)):
            want = kept[side, layer, keep, :, :n].transpose(0, 1).reshape(n, width)
            assert torch.equal(x.cpu().float(), want), (layer, side)


def test_a_captured_turn_replayed():
    """Extension, append, attention, verification, log probabilities and trim in one graph, on new inputs
    each replay, against the same calls one by one."""
    N, B, Hq, Hkv, D, V, P, top = 4, 4, 4, 2, 64, 9000, 50, 3
    g = torch.Generator(device="cuda").manual_seed(0)

    def fresh():
        c = xpress.Cache.empty(1, 40, Hkv, 16, D, N, 10, bits=4)
        c.k.fill_(0x7a), c.v.fill_(0x7b)
        x = {a: torch.zeros(N * B, n, device="cuda", dtype=torch.bfloat16)
             for a, n in (("q", Hq * D), ("k", Hkv * D), ("v", Hkv * D), ("logits", V))}
        x["blk"] = torch.zeros(N, B, dtype=torch.int64, device="cuda")
        x["u"] = torch.zeros(N, B, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        o = dict(att=torch.zeros(N * B, Hq * D, dtype=torch.bfloat16, device="cuda"),
                 out=torch.zeros(N, B, dtype=torch.int64, device="cuda"),
                 accepted=torch.zeros(N, **i32), drop=torch.zeros(N, **i32), lacking=torch.zeros(1, **i32),
                 logprob=torch.zeros(N * B, device="cuda"), rank=torch.zeros(N * B, **i32),
                 top_ids=torch.zeros(N * B, top, dtype=torch.int64, device="cuda"),
                 top_logprobs=torch.zeros(N * B, top, device="cuda"))
        ws = (xpress.cache_workspace(c, N), xpress.attention_workspace(c, N, B, Hq),
              xpress.verify_workspace(N, B, V), xpress.logprobs_workspace(N * B, V, top))
        xpress.cache_extend(c, P, N=1, lacking=o["lacking"], ws=ws[0])
        rows = torch.arange(N, **i32)
        xpress.cache_fork(c, torch.zeros_like(rows[1:]), rows[1:])
        temperature = torch.tensor([0.0, 1.0, 0.5, 2.0], device="cuda")

        def turn():
            xpress.cache_extend(c, B, N=N, lacking=o["lacking"], ws=ws[0])
            xpress.cache_append(c, 0, x["k"], x["v"], N=N, B=B, lacking=o["lacking"])
            xpress.block_attention(c, 0, x["q"], N=N, B=B, Hq=Hq, shared=P, out=o["att"], ws=ws[1])
            xpress.verify_draft(x["logits"], x["blk"], u=x["u"], temperature=temperature, out=o["out"],
                                accepted=o["accepted"], drop=o["drop"], ws=ws[2])
            xpress.token_logprobs(x["logits"], o["out"], temperature=temperature, ws=ws[3],
                                  logprob=o["logprob"], rank=o["rank"], top_ids=o["top_ids"],
                                  top_logprobs=o["top_logprobs"])
            xpress.cache_trim(c, o["drop"], N=N, lacking=o["lacking"])

        return c, x, o, turn

    (ce, xe, oe, eager), (cg, xg, og, captured) = fresh(), fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    for rep in range(5):
        new = {a: torch.randn(b.shape, generator=g, device="cuda").to(b.dtype) for a, b in xe.items()
               if b.dtype == torch.bfloat16}
        new["blk"] = torch.randint(V, (N, B), generator=g, device="cuda")
        new["u"] = torch.rand(N, B, generator=g, device="cuda")
        row = torch.arange(N * B, device="cuda").view(N, B)[:, :-1]
        new["logits"][row.reshape(-1), new["blk"][:, 1:].reshape(-1)] = 9.0
        for x in (xe, xg):
            for a, b in new.items():
                x[a].copy_(b)
        eager()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in oe:
            assert torch.equal(oe[name], og[name]), (rep, name)
        for name in ("table", "length", "ref", "k", "v"):
            assert torch.equal(getattr(ce, name), getattr(cg, name)), (rep, name)
        check(xe["logits"].cpu(), oe["out"].cpu(), [0.0, 1.0, 0.5, 2.0], top,
              dict(logprob=oe["logprob"], rank=oe["rank"], top_ids=oe["top_ids"],
                   top_logprobs=oe["top_logprobs"], entropy=torch.zeros(N * B)), f"replay {rep}",
              entropy=False)


def test_the_command_runs(capsys):
    main(["--samples", "2", "--turns", "3", "--prompt", "40", "--bits", "4", "--logprobs"])
    said = capsys.readouterr().out.splitlines()
    assert len(said) == 3 and said[-1].startswith("pages after")
    assert all("log probability -" in x for x in said[:2])
