"""Whole turns: several samples of one prompt decoded with all calls together (draft_turn), against
plain oracles; and a captured turn replayed."""
import math

import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import synth, upload, xpress
from jacobi_block_refiner_amd.draft_turn import Decoder, Target, main
from tests.gpu_helpers import log
from tests.serve_oracle import verify

pytestmark = pytest.mark.gpu


def plain(target, ids):
    """Logits of a whole sequence without a cache, attention in float32."""
    n = ids.numel()

    def attend(layer, q, k, v):
        Hq, Hkv, D = target.Hq, target.Hkv, target.D
        q, k, v = (x.float().view(n, -1, D).transpose(0, 1) for x in (q, k, v))
        k, v = (x.repeat_interleave(Hq // Hkv, 0).contiguous() for x in (k, v))
        s = (q.contiguous() @ k.transpose(1, 2).contiguous()) * D ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=s.device).triu(1), -math.inf)
        return (s.softmax(-1) @ v).transpose(0, 1).reshape(n, Hq * D).to(torch.bfloat16)

    return target.forward(ids, torch.arange(n, device=ids.device), attend)[1]


@pytest.mark.parametrize("samples,prompt,page,temperature", [(1, 3, 16, 0.0), (3, 41, 16, 1.0),
                                                             (5, 130, 64, 0.7)])
def test_turns_against_a_forward_without_a_cache(samples, prompt, page, temperature):
    inp = synth.make_inputs(1).rounded_bf16()
    B, turns = inp.wl.B, 6
    target = Target(inp.wl.V, inp.wl.H, most=prompt + turns * B + B)
    dec = Decoder(target, upload.weights(inp), samples, page=page, most=prompt + turns * B,
                  temperature=temperature)
    ids = torch.randint(inp.wl.V, (prompt,), generator=torch.Generator().manual_seed(3)).cuda()
    dec.prompt(ids)
    text = [ids.tolist() for _ in range(samples)]
    seen, stood = [], 0
    for _ in range(turns):
        t = dec.turn()
        assert int(dec.lacking.item()) == 0
        out, accepted = verify(t.logits.double().cpu().numpy(), t.blk.cpu().numpy(), None, None,
                               np.full(samples, temperature, np.float32), t.u.cpu().numpy())
        assert np.array_equal(out, t.out.cpu().numpy())
        assert np.array_equal(accepted, t.accepted.cpu().numpy())
        for i in range(samples):
            assert int(t.blk[i, 0]) == text[i][-1]  # the anchor
            for s in range(accepted[i] + 1):
                seen.append((i, len(text[i]) - 1 + s, t.logits[i * B + s]))
            text[i] += [int(x) for x in out[i] if x >= 0]
        stood += int(accepted.sum())
        assert dec.cache.length.tolist() == [len(x) - 1 for x in text]
    log(f"turns: {stood} of {samples * turns * (B - 1)} drafts stood")
    assert 0 < stood
    # Both sides round the same 29 values to bf16, at most one step apart where a sum's last bits
    # differ: sqrt(29 * 2 / 3) * 2^-8 = 0.017 of a row's norm, three times that for the layers' gain.
    full = [plain(target, torch.tensor(x, device="cuda")) for x in text]
    for i, at, got in seen:
        want = full[i][at].float()
        assert (got.float() - want).norm() <= 0.05 * want.norm(), (i, at)
    # one sample kept: its pages move to the front, with the same tokens in them
    keep = samples // 2
    n = int(dec.cache.length[keep])

    def lines():
        pages = dec.cache.table[keep, : -(-n // page)].long()
        k, v = (x[:, pages].transpose(2, 3).flatten(1, 2)[:, :n] for x in (dec.cache.k, dec.cache.v))
        return k.clone(), v.clone()

    before = lines()
    assert dec.keep(keep) == -(-n // page)
    assert all(torch.equal(a, b) for a, b in zip(before, lines()))
    assert dec.cache.length.tolist() == [n if i == keep else 0 for i in range(samples)]
    assert dec.cache.ref.sum().item() == -(-n // page) == (dec.cache.ref > 0).sum().item()


def test_a_captured_turn_replayed():
    """Extension, append, attention, verification and trim in one graph, on new inputs each replay,
    against the same calls one by one; other work and synchronizations between the replays."""
    N, B, Hq, Hkv, D, V, P = 4, 4, 4, 2, 64, 9000, 50
    g = torch.Generator(device="cuda").manual_seed(0)

    def fresh():
        c = xpress.Cache.empty(1, 40, Hkv, 16, D, N, 10)
        c.k.fill_(0.25), c.v.fill_(0.5)
        x = dict(q=torch.zeros(N * B, Hq * D), k=torch.zeros(N * B, Hkv * D),
                 v=torch.zeros(N * B, Hkv * D), logits=torch.zeros(N * B, V))
        x = {a: b.to("cuda", torch.bfloat16) for a, b in x.items()}
        x["blk"] = torch.zeros(N, B, dtype=torch.int64, device="cuda")
        x["u"] = torch.zeros(N, B, device="cuda")
        o = dict(att=torch.zeros(N * B, Hq * D, dtype=torch.bfloat16, device="cuda"),
                 out=torch.zeros(N, B, dtype=torch.int64, device="cuda"),
                 accepted=torch.zeros(N, dtype=torch.int32, device="cuda"),
                 drop=torch.zeros(N, dtype=torch.int32, device="cuda"),
                 lacking=torch.zeros(1, dtype=torch.int32, device="cuda"))
        ws = (xpress.cache_workspace(c, N), xpress.attention_workspace(c, N, B, Hq),
              xpress.verify_workspace(N, B, V))
        # a shared prompt
        xpress.cache_extend(c, P, N=1, lacking=o["lacking"], ws=ws[0])
        rows = torch.arange(N, dtype=torch.int32, device="cuda")
        xpress.cache_fork(c, torch.zeros_like(rows[1:]), rows[1:])
        temperature = torch.tensor([0.0, 1.0, 0.5, 2.0], device="cuda")

        def turn():
            xpress.cache_extend(c, B, N=N, lacking=o["lacking"], ws=ws[0])
            xpress.cache_append(c, 0, x["k"], x["v"], N=N, B=B)
            xpress.block_attention(c, 0, x["q"], N=N, B=B, Hq=Hq, shared=P, out=o["att"], ws=ws[1])
            xpress.verify_draft(x["logits"], x["blk"], u=x["u"], temperature=temperature,
                                out=o["out"], accepted=o["accepted"], drop=o["drop"], ws=ws[2])
            xpress.cache_trim(c, o["drop"], N=N)

        return c, x, o, turn

    ce, xe, oe, eager = fresh()
    cg, xg, og, turn = fresh()
    torch.cuda.synchronize()
    start = cg.length.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    assert torch.equal(cg.length, start)  # recording ran nothing
    for rep in range(5):
        for name, t in xe.items():
            if name == "blk":
                t.copy_(torch.randint(V, t.shape, device="cuda", generator=g))
            elif name == "u":
                t.copy_(torch.rand(t.shape, device="cuda", generator=g))
            else:
                t.copy_(torch.randn(t.shape, device="cuda", generator=g))
            xg[name].copy_(t)
        # some drafts stand: their logits are far above the rest
        sure = torch.arange(N, device="cuda")[:, None] >= torch.arange(B - 1, device="cuda")
        for x in (xe, xg):
            l = x["logits"].view(N, B, V)[:, :-1]
            l.scatter_(2, x["blk"][:, 1:, None], torch.where(sure, 60.0, -9.0)[:, :, None].bfloat16())
        eager()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in oe:
            assert torch.equal(oe[name], og[name]), (rep, name)
        for name in ("table", "length", "ref", "k", "v"):
            assert torch.equal(getattr(ce, name), getattr(cg, name)), (rep, name)
        assert oe["accepted"].tolist() == [1, 2, 3, 3], rep


def test_the_command_runs(capsys):
    main(["--samples", "2", "--turns", "3", "--prompt", "40", "--greedy"])
    said = capsys.readouterr().out.splitlines()
    assert len(said) == 3 and said[0].startswith("sample 0:") and said[-1].startswith("pages after")


def test_a_decoder_whose_table_is_full():
    """Turns past the decoder's tokens: the turn that finds no room raises and leaves the cache and the
    anchors as they were."""
    inp = synth.make_inputs(1).rounded_bf16()
    target = Target(inp.wl.V, inp.wl.H, most=64)
    dec = Decoder(target, upload.weights(inp), 3, page=16, most=30, temperature=0.0)
    dec.prompt(torch.randint(inp.wl.V, (25,), generator=torch.Generator().manual_seed(5)).cuda())

    def state():
        c = dec.cache
        return [x.clone() for x in (c.table, c.length, c.ref, c.k.view(torch.int16),
                                    c.v.view(torch.int16), dec.anchor, dec.am1, dec.h, dec.base)]

    with pytest.raises(RuntimeError, match="table is full"):
        for _ in range(40):
            before = state()
            dec.turn()
    assert all(torch.equal(a, b) for a, b in zip(before, state()))
    room = dec.cache.table.shape[1] * 16
    assert room - dec.B < int(dec.cache.length.max()) <= room
    with pytest.raises(RuntimeError, match="table is full"):
        dec.turn()
    assert all(torch.equal(a, b) for a, b in zip(before, state()))


def test_a_pool_with_room_for_every_table():
    """Samples whose first block fits in the prompt's page: each copies it while it is still there."""
    inp = synth.make_inputs(1).rounded_bf16()
    B, N, prompt = inp.wl.B, 4, 3
    target = Target(inp.wl.V, inp.wl.H, most=64)
    dec = Decoder(target, upload.weights(inp), N, page=16, most=16 - B, temperature=0.0)
    assert dec.cache.table.shape[1] == 1 and prompt - 1 + B <= 16
    dec.prompt(torch.arange(prompt).cuda())
    t = dec.turn()
    assert int(dec.lacking.item()) == 0
    assert (dec.cache.length == prompt + t.accepted).all() and dec.cache.ref.sum().item() == N
    assert sorted(dec.cache.table.flatten().tolist()) == [1, 2, 3, 4] and int(dec.cache.ref[0]) == 0


def test_a_prompt_too_short_or_too_long():
    inp = synth.make_inputs(1).rounded_bf16()
    target = Target(inp.wl.V, inp.wl.H, most=64)
    dec = Decoder(target, upload.weights(inp), 2, page=16, most=20)
    for n in (0, 1):
        with pytest.raises(ValueError, match="two tokens"):
            dec.prompt(torch.zeros(n, dtype=torch.int64, device="cuda"))
    with pytest.raises(RuntimeError, match="table is full"):
        dec.prompt(torch.zeros(dec.cache.table.shape[1] * 16 + 2, dtype=torch.int64, device="cuda"))
    assert not dec.cache.length.any() and not dec.cache.ref.any()
