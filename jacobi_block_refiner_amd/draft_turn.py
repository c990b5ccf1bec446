"""Speculative decoding of several samples of one prompt, with the library's calls together.

A small random target model (its dense products are plain torch) keeps its K and V in a paged cache.
The prompt is run once and forked to every sample; then each turn drafts a block with the refiner,
runs the target over the block and keeps what the target confirms:

    xpress_jacobi_step -> xpress_cache_extend
    -> (xpress_cache_append_if, xpress_block_attention) a layer
    -> xpress_verify_draft -> xpress_cache_trim_if

At the end all samples but one are freed and the pool is compacted.

    python -m jacobi_block_refiner_amd.draft_turn [--samples 4] [--turns 8] [--prompt 200] [--greedy]
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

from . import synth, upload, xpress

__all__ = ["Target", "Decoder", "Turn"]


def _normed(x):
    x32 = x.float()
    return (x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Target:
    """A decoder-only model of random bf16 weights: grouped-query attention and a gated MLP a layer,
    learned positions. Its attention and its cache are the library's."""

    def __init__(self, V: int, H: int, *, layers: int = 2, Hq: int = 4, Hkv: int = 2, D: int = 64,
                 most: int = 1024, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(device, torch.bfloat16)

        self.V, self.H, self.Hq, self.Hkv, self.D, self.most = V, H, Hq, Hkv, D, most
        self.embed, self.place = w(V, H) * H ** 0.5, w(most, H) * H ** 0.5
        self.layers = [dict(qkv=w((Hq + 2 * Hkv) * D, H), out=w(H, Hq * D), up=w(4 * H, H),
                            gate=w(4 * H, H), down=w(H, 4 * H)) for _ in range(layers)]
        self.head = self.embed / H ** 0.5  # tied: a token is likely to follow itself, so drafts stand

    def forward(self, ids: torch.Tensor, at: torch.Tensor, attend) -> tuple[torch.Tensor, torch.Tensor]:
        """ids, at (positions): [tokens]. attend(layer, q, k, v) gives the attention's result.
        Returns the last hidden states and the logits."""
        x = self.embed[ids] + self.place[at.clamp(max=self.most - 1)]
        nq, nk = self.Hq * self.D, self.Hkv * self.D
        for i, p in enumerate(self.layers):
            q, k, v = (_normed(x) @ p["qkv"].t()).split([nq, nk, nk], dim=1)
            x = x + attend(i, q, k, v) @ p["out"].t()
            y = _normed(x)
            x = x + (torch.nn.functional.silu(y @ p["gate"].t()) * (y @ p["up"].t())) @ p["down"].t()
        h = _normed(x)
        return h, h @ self.head.t()


@dataclass
class Turn:
    """What a turn did: the block, the target's logits, and what stood (all on the device)."""

    blk: torch.Tensor  # [N, B]: the anchor and the drafts
    logits: torch.Tensor  # [N*B, V]
    u: torch.Tensor  # [N, B]
    out: torch.Tensor  # [N, B]: the accepted drafts, one more token, -1
    accepted: torch.Tensor  # [N]


class Decoder:
    """The samples of one prompt: their cache, the refiner's inputs and the buffers of a turn."""

    def __init__(self, target: Target, refiner: xpress.Weights, samples: int, *, page: int = 16,
                 most: int = 512, temperature: float = 1.0, seed: int = 0):
        d = refiner.dims
        if (d["H"], d["V"]) != (target.H, target.V):
            raise ValueError("the refiner and the target differ in hidden size or vocabulary")
        self.target, self.refiner, self.N, self.B = target, refiner, samples, d["B"]
        dev = target.embed.device
        N, B, V = self.N, self.B, target.V
        ld = -(-(most + B) // page)
        # every row's table full, and the prompt's last page while every sample copies it
        self.cache = xpress.Cache.empty(len(target.layers), ld * N + 1, target.Hkv, page, target.D, N,
                                        ld, device=dev)
        self.shared = 0

        def empty(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device=dev)

        self.blk, self.out = empty(N, B, dtype=torch.int64), empty(N, B, dtype=torch.int64)
        self.accepted, self.drop, self.lacking, self.live = empty(N), empty(N), empty(1), empty(1)
        self.temperature = torch.full((N,), temperature, device=dev)
        self.rng = torch.Generator(device=dev).manual_seed(seed)
        self.step_ws = xpress.alloc_workspace(N, B, d["r"], V, 0, B, dev)
        self.cache_ws = xpress.cache_workspace(self.cache, N)
        self.attention_ws = xpress.attention_workspace(self.cache, N, B, target.Hq)
        self.verify_ws = xpress.verify_workspace(N, B, V, dev)

    def _run(self, ids: torch.Tensor, N: int, B: int, ws: torch.Tensor):
        """The target over B more tokens of rows 0..N-1; ids: [N*B]."""
        xpress.cache_extend(self.cache, B, N=N, lacking=self.lacking, ws=self.cache_ws)
        end = self.cache.length[:N].to(torch.int64)
        at = (end[:, None] - B + torch.arange(B, device=end.device)).reshape(-1)

        def attend(layer, q, k, v):
            xpress.cache_append(self.cache, layer, k, v, N=N, B=B, lacking=self.lacking)
            return xpress.block_attention(self.cache, layer, q, N=N, B=B, Hq=self.target.Hq,
                                          shared=self.shared, out=torch.empty(
                                              q.shape, dtype=q.dtype, device=q.device),
                                          ws=ws)

        return self.target.forward(ids, at, attend)

    def prompt(self, ids: torch.Tensor) -> None:
        """Runs a prompt (all tokens but the last, which is the first anchor) and forks it to every
        sample."""
        N, B = self.N, self.B
        P = ids.numel() - 1
        if P < 1:
            raise ValueError("a prompt has two tokens at least: the anchor and the one before it")
        ws = xpress.attention_workspace(self.cache, 1, P, self.target.Hq)
        h, logits = self._run(ids[:-1], 1, P, ws)
        self._check_room()
        rows = torch.arange(N, dtype=torch.int32, device=ids.device)
        xpress.cache_fork(self.cache, torch.zeros_like(rows[1:]), rows[1:])
        self.shared = self.reach = P
        self.anchor, self.am1 = ids[-1].repeat(N), ids[-2].repeat(N)
        # the refiner's view of the slots to come: the last state and logits, over the block
        self.h = h[-1].repeat(N, B, 1)
        self.base = logits[-1].repeat(N * (B - 1), 1)

    def turn(self) -> Turn:
        """One turn of all samples. Raises where a row's table is full; the cache and the anchors are
        then as they were."""
        N, B, V = self.N, self.B, self.target.V
        xpress.jacobi_step(self.refiner, self.h, self.base, self.anchor, self.am1, self.blk, K=B,
                           flags=xpress.INIT_FROM_BASE | xpress.STOP_AT_FIXED_POINT, ws=self.step_ws)
        h, logits = self._run(self.blk.view(-1), N, B, self.attention_ws)
        u = torch.rand(N, B, device=h.device, generator=self.rng)
        xpress.verify_draft(logits, self.blk, u=u, temperature=self.temperature, out=self.out,
                            accepted=self.accepted, drop=self.drop, ws=self.verify_ws)
        xpress.cache_trim(self.cache, self.drop, N=N, lacking=self.lacking)
        # tokens of the longest row at most: the host waits for the card only where they might not fit
        self.reach += B
        if self.reach > self.cache.table.shape[1] * self.cache.k.shape[3]:
            self._check_room()
        # the extra token is the next anchor; the state it was drawn from serves the next block
        a = self.accepted.to(torch.int64)[:, None]
        self.anchor, self.am1 = self.out.gather(1, a)[:, 0], self.blk.gather(1, a)[:, 0]
        self.h = h.view(N, B, -1).gather(1, a[:, :, None].expand(N, 1, h.shape[1])).repeat(1, B, 1)
        base = logits.view(N, B, V).gather(1, a[:, :, None].expand(N, 1, V))
        self.base = base.expand(N, B - 1, V).reshape(N * (B - 1), V).contiguous()
        return Turn(self.blk.clone(), logits, u, self.out.clone(), self.accepted.clone())

    def keep(self, sample: int) -> int:
        """Frees every sample but one and compacts the pool; the pages that are left."""
        others = torch.tensor([i for i in range(self.N) if i != sample], dtype=torch.int32,
                              device=self.blk.device)
        if others.numel():
            xpress.cache_trim(self.cache, None, seq=others)
        xpress.cache_compact(self.cache, live=self.live, ws=self.cache_ws)
        return int(self.live.item())

    def _check_room(self) -> None:
        lacking = int(self.lacking.item())
        if lacking:
            raise RuntimeError("a row's table is full" if lacking < 0 else
                               f"the pool lacks {lacking} pages")


def main(argv=None) -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--samples", type=int, default=4)
    p.add_argument("--turns", type=int, default=8)
    p.add_argument("--prompt", type=int, default=200)
    p.add_argument("--greedy", action="store_true")
    a = p.parse_args(argv)
    inp = synth.make_inputs(1).rounded_bf16()
    most = a.prompt + a.turns * inp.wl.B
    target = Target(inp.wl.V, inp.wl.H, most=most + inp.wl.B)
    dec = Decoder(target, upload.weights(inp), a.samples, most=most,
                  temperature=0.0 if a.greedy else 1.0)
    ids = torch.randint(inp.wl.V, (a.prompt,), generator=torch.Generator().manual_seed(1))
    dec.prompt(ids.cuda())
    text = [[] for _ in range(a.samples)]
    for _ in range(a.turns):
        t = dec.turn()
        for row, new in zip(text, t.out.tolist()):
            row += [x for x in new if x >= 0]
    for i, row in enumerate(text):
        print(f"sample {i}: {len(row)} tokens in {a.turns} turns: {row[:12]}")
    print(f"pages after keeping sample 0: {dec.keep(0)}")


if __name__ == "__main__":
    main()
