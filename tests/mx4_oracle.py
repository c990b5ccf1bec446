"""Plain 64-bit oracle of the 4-bit cache: the nearest values of a group, and where a tile's bytes lie,
one statement a token and channel. CPU torch only; nothing here is shared with the library."""
from __future__ import annotations

import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
LIMITS = {torch.bfloat16: (-123, 125), torch.float16: (-23, 13)}


def quantise(x, dtype):
    """x [..., D]: codes (0..15) and the exponents of its groups of 32 channels."""
    lo, hi = LIMITS[dtype]
    g = torch.nan_to_num(x.double(), nan=0.0, posinf=1e300, neginf=-1e300).unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    # the power of two of which the largest is 3.5 to 7 times
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0) / 3.5))
    e = torch.where(torch.pow(2.0, e + 1) * 3.5 <= top, e + 1, e)  # (a logarithm may round across)
    e = torch.where(torch.pow(2.0, e) * 3.5 > top, e - 1, e).clamp(lo, hi)
    e = torch.where(top > 0, e, float(lo))
    y = g / torch.pow(2.0, e)[..., None]
    away = (y.abs().clamp(max=6.0)[..., None] - LEVELS).abs()
    best = away.amin(-1, keepdim=True)
    tied = away == best  # two neighbours at most: the even code of them
    even = tied & (torch.arange(8) % 2 == 0)
    code = torch.where(tied.sum(-1) > 1, even.int().argmax(-1), away.argmin(-1))
    code = code + 8 * (y < 0)
    return code.flatten(-2), e.to(torch.int64)


def values(code, e):
    """What codes and exponents stand for, in 64 bits."""
    size = LEVELS[code % 8] * torch.where(code >= 8, -1.0, 1.0)
    return (size.unflatten(-1, (-1, 32)) * torch.pow(2.0, e.double())[..., None]).flatten(-2)


def code_byte(D, t, c, is_v):
    """Byte of channel c of token t in a tile, and whether it is the byte's high half."""
    if not is_v:
        return t * (D // 2) + c // 2, c % 2
    q, j, g, i = t // 4, t % 4, c // 32, c % 32 // 2
    return ((16 * q + i) * (D // 32) + g) * 4 + j, c % 2


def scale_byte(D, t, g, is_v):
    return 8 * D + ((t // 4 * (D // 32) + g) * 4 + t % 4 if is_v else t * (D // 32) + g)


def _maps(D, is_v):
    byte = torch.tensor([[code_byte(D, t, c, is_v)[0] for c in range(D)] for t in range(16)])
    scale = torch.tensor([[scale_byte(D, t, g, is_v) for g in range(D // 32)] for t in range(16)])
    return byte, scale


def pack(code, e, is_v):
    """Tiles of codes [..., 16, D] and exponents [..., 16, D/32]: [..., 17 D / 2] bytes."""
    D, lead = code.shape[-1], code.shape[:-2]
    byte, scale = _maps(D, is_v)
    tile = torch.zeros(*lead, 17 * D // 2, dtype=torch.int64)
    for odd in (0, 1):
        at = byte[:, odd::2].reshape(-1)
        tile[..., at] += (code[..., odd::2] << 4 * odd).reshape(*lead, -1)
    tile[..., scale.reshape(-1)] = (e + 127).reshape(*lead, -1)
    return tile.to(torch.uint8)


def unpack(tile, D, is_v):
    """The values of tiles [..., 17 D / 2]: [..., 16, D], 64 bits."""
    byte, scale = _maps(D, is_v)
    code = tile.long()[..., byte] >> 4 * (torch.arange(D) % 2) & 15
    return values(code, tile.long()[..., scale] - 127)


def pool_values(pool, D, is_v):
    """A pool [layers, pages, Hkv, page/16, 17 D / 2] as values [layers, pages, Hkv, page, D]."""
    return unpack(pool, D, is_v).flatten(3, 4)


def pool_of(x, dtype, is_v):
    """A pool that holds what x [layers, pages, Hkv, page, D] is nearest to."""
    code, e = quantise(x.unflatten(3, (-1, 16)), dtype)
    return pack(code, e, is_v)
