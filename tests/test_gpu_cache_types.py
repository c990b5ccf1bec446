"""The types that a cache follows: its pools', where it holds 16 bits."""
import dataclasses

import pytest
import torch

from jacobi_block_refiner_amd import xpress

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


def test_a_cache_of_16_bits_with_pools_of_the_other_type():
    a = xpress.Cache.empty(1, 4, 2, 16, 64, 2, 3)
    b = dataclasses.replace(a, k=a.k.half(), v=a.v.half())
    ws, lacking = xpress.cache_workspace(b, 2), torch.zeros(1, dtype=torch.int32, device="cuda")
    xpress.cache_extend(b, 3, lacking=lacking, ws=ws)
    new = torch.randn(6, 2 * 64, device="cuda").half()
    xpress.cache_append(b, 0, new, -new, B=3)
    k, v = torch.zeros_like(new), torch.zeros_like(new)
    xpress.cache_read(b, 0, k, v, B=3)
    assert torch.equal(k, new) and torch.equal(v, -new)
    with pytest.raises(TypeError, match="k_new"):
        xpress.cache_append(b, 0, new.bfloat16(), new.bfloat16(), B=3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_a_cache_of_4_bits_keeps_its_type(dtype):
    a = xpress.Cache.empty(1, 4, 2, 16, 64, 2, 3, dtype=dtype, bits=4)
    b = dataclasses.replace(a, k=a.k.clone(), v=a.v.clone())
    assert a.dtype == b.dtype == dtype
    with pytest.raises(TypeError, match="cannot hold"):
        dataclasses.replace(a, dtype=torch.float32)
