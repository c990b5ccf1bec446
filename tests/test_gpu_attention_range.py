"""Block attention over values at the ends of their type's range, whose mean is a value like any other,
against attention from its definition in 64 bits."""
import math

import pytest
import torch

from jacobi_block_refiner_amd import xpress
from tests import mx4_oracle as mx4
from tests.gpu_helpers import log
from tests.serve_oracle import attention, attention_bounds
from tests.test_gpu_attention import Case, _gpu  # noqa: F401 (a fixture)
from tests.test_gpu_mx4 import Case4

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]

CASES = [
    dict(lengths=[1], shared=0, B=1, Hkv=1, G=1, D=64, page=16),
    dict(lengths=[5, 0, 3, 64, 65], shared=0, B=4, Hkv=2, G=3, D=64, page=16),
    dict(lengths=[300, 0, 290, 288, 401], shared=277, B=7, Hkv=1, G=5, D=128, page=64),
    dict(lengths=[700, 650], shared=600, B=16, Hkv=1, G=8, D=256, page=128),
    dict(lengths=[500, 3, 17], shared=450, B=5, Hkv=1, G=2, D=64, page=256),  # rows end in the prefix
    dict(lengths=[1025], shared=0, B=16, Hkv=2, G=7, D=128, page=16),
    dict(lengths=[90, 91, 92, 93], shared=80, B=33, Hkv=1, G=9, D=64, page=16),  # 297 rows a request
    dict(lengths=[1500, 7, 0, 900, 1], shared=0, B=1, Hkv=2, G=8, D=128, page=64),
    dict(lengths=[900, 2, 513], shared=0, B=1, Hkv=1, G=5, D=256, page=32),
    dict(lengths=[4000, 31, 33], shared=0, B=2, Hkv=1, G=8, D=128, page=16),
    dict(lengths=[1000, 1001, 3], shared=0, B=8, Hkv=1, G=4, D=256, page=64),
    dict(lengths=[70] * 300, shared=0, B=1, Hkv=1, G=4, D=256, page=64),  # slim items in 16 bits
    # many query rows a head (D 128): the shared part in wide items
    dict(lengths=[400, 0, 395, 17, 300, 399, 396, 401] * 2, shared=390, B=16, Hkv=2, G=8, D=128, page=16),
]
SIZES = {"huge": 127, "large": 118, "small": -95, "mixed": None}
OF_16_BITS = 90  # log2 of bf16 values whose sums are sure to stay in range


def values(v, size, top):
    """Numbers of the size of 2^`top` (that, at most) in place of numbers of the size of 1, of one sign a
    channel: every sum of them is as large as it can be."""
    sign = 1.0 - 2.0 * (torch.arange(v.shape[-1]) % 2)
    grown = v.double().abs().clamp(0.25, 1.0) * sign * 2.0 ** top
    if size == "mixed":  # every fourth channel as it was, and rows of a few huge values among ordinary ones
        few = (torch.arange(v.shape[-2]) % 13 == 5)[:, None] & (torch.arange(v.shape[-1]) % 4 > 0)
        grown = torch.where(few, grown, v.double())
    return torch.where(v.isnan(), math.nan, grown).float()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("bits,dtype", [(4, torch.bfloat16), (16, torch.bfloat16), (4, torch.float16),
                                        (16, torch.float16)], ids=["4bf16", "16bf16", "4f16", "16f16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_values_at_the_ends_of_the_range(i, bits, dtype, size):
    """Scores of some size, so that weights pass those of the first keys by far."""
    top = SIZES[size] if SIZES[size] is not None else 127
    if dtype == torch.float16:
        top = {127: 15, 118: 13, -95: -10}[top]
    elif bits == 16:
        top = min(top, OF_16_BITS)
    x = (Case4 if bits == 4 else Case)(**CASES[i], dtype=dtype, seed=i, q_scale=3.0)
    log(f"range case {i} {bits} bits {dtype} {size}")
    if bits == 16:
        x.v = values(x.v, size, top).to(dtype)
        c = x.cache()
        x.v = x.v.nan_to_num(0.0)
        x.k = x.k.nan_to_num(0.0)
    else:
        dead = (x.k == 0).all(-1).unflatten(3, (-1, 16))
        v = values(x.v, size, top)
        if size == "huge":  # infinities are held as the largest value
            v[..., ::7] = math.copysign(math.inf, 1.0) * torch.sign(v[..., ::7])
        code, e = mx4.quantise(v.unflatten(3, (-1, 16)), dtype)
        x.v = torch.where(dead.flatten(3, 4)[..., None], 0.0, mx4.values(code, e).flatten(3, 4)).to(dtype)
        code[dead], e[dead] = 15, 128
        x.pools[1] = mx4.pack(code, e, True)
        c = x.cache()
        assert size != "huge" or float(x.v.abs().max()) == (1.5 * 2.0 ** 127 if top == 127 else 49152)
    assert bool(x.v.isfinite().all())
    for shared in {x.shared, 0}:
        x.check(x.run(c, shared=shared), what=f"shared {shared}")


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("D,B,G", [(64, 1, 4), (128, 1, 4), (128, 16, 4), (256, 2, 4), (128, 16, 16)])
def test_a_huge_value_late_in_a_row(D, B, G, bits):
    """One key far along the row, ahead of those before it by less than makes a sum rescale: 2^7 times
    their weight, on a value of 1.5 * 2^127 (in 16 bits 2^89)."""
    page, n, Hq = 64, 900, G
    scale = D ** -0.5
    k = torch.zeros(1, 15, 1, page, D)
    v = torch.ones(1, 15, 1, page, D)
    k[0, 10, 0, 9, 0] = 4.0
    v[0, 10, 0, 9] = 1.5 * 2.0 ** (127 if bits == 4 else OF_16_BITS - 1)
    v[0, 10, 0, 9, ::2] *= -1
    q = torch.zeros(B, Hq * D)
    q[:, ::D] = 7 * math.log(2) / scale / 4
    q = q.bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    meta = dict(table=torch.arange(15, **i32)[None], length=torch.tensor([n], **i32),
                ref=torch.ones(15, **i32))
    if bits == 4:
        c = xpress.Cache(k=mx4.pool_of(k, torch.bfloat16, False).cuda(),
                         v=mx4.pool_of(v, torch.bfloat16, True).cuda(), **meta)
        assert torch.equal(mx4.pool_values(c.v.cpu(), D, True).float(), v)
    else:
        c = xpress.Cache(k=k.bfloat16().cuda(), v=v.bfloat16().cuda(), **meta)
    for shared in (0, 576):
        out = torch.empty(B, Hq * D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(B, Hq, device="cuda")
        xpress.block_attention(c, 0, q.cuda(), B=B, Hq=Hq, N=1, out=out, lse=lse, shared=shared,
                               ws=xpress.attention_workspace(c, 1, B, Hq))
        want, wl, mass, size = attention(k[0], v[0], [range(15)], [n], page, q, [0], B, Hq, scale)
        bound, lse_bound = attention_bounds(want, mass, size, n, D, torch.bfloat16)
        assert bool(((out.cpu().double().view(want.shape) - want).abs() <= bound).all())
        # (2^-18 for logarithms of weights 2^-37 times as large: two roundings of numbers up to 64)
        assert bool(((lse.cpu().double() - wl).abs() <= lse_bound + wl.abs() * 2.0 ** -22 + 2.0 ** -18).all())
