"""Log probabilities end at 0 and entropies begin there, also in rows whose one id has nearly all."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_logprobs import _gpu, check, run  # noqa: F401 (a fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


def ends(got, top):
    out = {k: v.cpu().double().numpy() for k, v in got.items()}
    assert (out["logprob"] <= 0).all() and (out["entropy"] >= 0).all()
    assert not np.isnan(out["entropy"]).any() and not np.isnan(out["logprob"]).any()
    if top:
        assert (out["top_logprobs"] <= 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,top", [(1, 1), (2, 3), (40, 5), (9000, 0), (40000, 20)])
def test_rows_of_one_likely_id(V, top, dtype):
    """Maxima of many sizes, the others far behind; a few by so little that they still count."""
    rows = 96
    g = torch.Generator().manual_seed(V)
    best = torch.randint(V, (rows,), generator=g)
    x = torch.randn(rows, V, generator=g) - 10
    m = torch.randn(rows, generator=g) * 10
    x -= (m.abs() + torch.rand(rows, generator=g) * 60)[:, None]
    x[torch.arange(rows), best] = m
    x[::7] = -math.inf
    x[torch.arange(0, rows, 7), best[::7]] = m[::7]
    x = x.to(dtype).contiguous()
    token = best[:, None].clone()
    token[::5] = (token[::5] + 1) % V
    temps = torch.tensor([1.0, 0.7, 1.3, 0.01, 3.0, 1e-4, math.inf, 0.0])[torch.arange(rows) % 8]
    for t in (None, temps):
        got = run(x, token, None if t is None else t.tolist(), top)
        check(x, token, None if t is None else t.tolist(), top, got, f"one likely id of {V}")
        ends(got, top)
