"""Token log probabilities without a GPU: argument errors are found on the host (no kernel is launched by
any call here)."""
import ctypes

import pytest
import torch

from jacobi_block_refiner_amd import xpress
from tests.test_serve_abi_cpu import FAKE, ODD2, L, says

ODD4 = ctypes.c_void_p((1 << 20) + 4)


def call(logits=FAKE, dtype=xpress.BF16, ld=1000, token=FAKE, temperature=None, N=4, B=16, V=1000, top=5,
         logprob=FAKE, entropy=FAKE, rank=FAKE, ids=FAKE, values=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return L().xpress_token_logprobs(logits, dtype, ld, token, temperature, N, B, V, top, logprob, entropy,
                                     rank, ids, values, ws, ws_bytes, None)


def test_arguments():
    odd1 = ctypes.c_void_p((1 << 20) + 1)
    for args, text in ((dict(logits=None), b"logits"), (dict(logits=odd1), b"aligned"),
                       (dict(dtype=3), b"type"), (dict(dtype=xpress.F32, logits=ODD2), b"aligned"),
                       (dict(ld=999), b"stride"), (dict(ld=1 << 31), b"stride"),
                       (dict(token=ODD4), b"token"), (dict(token=None), b"token is NULL"),
                       (dict(token=None, logprob=None), b"token is NULL"),
                       (dict(token=None, rank=None), b"token is NULL"),
                       (dict(temperature=ODD2), b"temperature"), (dict(logprob=ODD2), b"logprob"),
                       (dict(entropy=ODD2), b"entropy"), (dict(rank=ODD2), b"rank"),
                       (dict(ids=None), b"top_ids"), (dict(ids=ODD4), b"top_ids"),
                       (dict(values=None), b"top_logprobs"), (dict(values=ODD2), b"top_logprobs"),
                       (dict(N=-1), b"N=-1"), (dict(B=0), b"B=0"), (dict(V=0), b"V=0"),
                       (dict(V=1 << 31, ld=1 << 31), b"V="), (dict(top=-1), b"top=-1"),
                       (dict(top=65), b"top=65"), (dict(N=1 << 20, B=16), b"too large"),
                       (dict(N=1 << 20, B=1, V=151936, ld=151936), b"too large"),
                       (dict(ws=None), b"ws")):
        says(call(**args), text)
    says(call(ws_bytes=1), b"workspace", xpress.ERR_WORKSPACE)
    assert call(N=0) == xpress.OK


def test_the_workspace_grows_with_rows():
    size, last = ctypes.c_size_t(), 0
    for n in range(300):
        assert L().xpress_logprobs_workspace_size(n, 151936, 20, ctypes.byref(size)) == xpress.OK
        assert size.value >= last
        last = size.value
    says(L().xpress_logprobs_workspace_size(1, 0, 20, ctypes.byref(size)), b"V=0")
    says(L().xpress_logprobs_workspace_size(-1, 10, 20, ctypes.byref(size)), b"rows")
    says(L().xpress_logprobs_workspace_size(1, 10, 65, ctypes.byref(size)), b"top")
    says(L().xpress_logprobs_workspace_size(1, 10, 20, None), b"bytes")


def test_the_binding_refuses_host_tensors_and_shapes():
    x, token = torch.zeros(6, 10), torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(TypeError):
        xpress.token_logprobs(x, token, ws=token)
    with pytest.raises(TypeError, match="bfloat16"):
        xpress.token_logprobs(x.to(torch.int8), token, ws=token)
