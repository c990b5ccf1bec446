"""What greedy tokens are reported with: their log probabilities under a temperature of its own."""
import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import synth, upload
from jacobi_block_refiner_amd.draft_turn import Decoder, Target, main
from tests.test_gpu_logprobs import check

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(120)]


def test_the_command_reports_greedy_samples(capsys):
    main(["--samples", "2", "--turns", "2", "--prompt", "20", "--greedy", "--logprobs"])
    said = capsys.readouterr().out.splitlines()
    assert len(said) == 3
    for line in said[:2]:
        assert float(line.split("log probability ")[1]) < -0.01, line


@pytest.mark.parametrize("report", [1.0, 0.25, None])
def test_greedy_turns_reported_at_a_temperature(report):
    inp = synth.make_inputs(1).rounded_bf16()
    B, samples, prompt, top = inp.wl.B, 2, 30, 3
    target = Target(inp.wl.V, inp.wl.H, most=prompt + 4 * B)
    dec = Decoder(target, upload.weights(inp), samples, most=prompt + 3 * B, temperature=0.0, top=top,
                  report=report)
    dec.prompt(torch.randint(inp.wl.V, (prompt,), generator=torch.Generator().manual_seed(4)).cuda())
    for turn in range(2):
        t = dec.turn()
        assert int(dec.lacking.item()) == 0
        # greedy: every token that stands is the first of its row's largest
        rows = t.logits.view(samples, B, -1).float().cpu().numpy()
        for i in range(samples):
            for s in range(int(t.accepted[i]) + 1):
                assert int(t.out[i, s]) == int(np.argmax(rows[i, s]))
        got = {k: getattr(t, k) for k in ("logprob", "entropy", "rank", "top_ids", "top_logprobs")}
        check(t.logits.cpu(), t.out.cpu(), [0.0 if report is None else report] * samples, top,
              {k: v.reshape(samples * B, *v.shape[2:]) for k, v in got.items()}, f"turn {turn}")
