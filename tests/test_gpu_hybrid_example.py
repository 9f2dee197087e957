"""The hybrid serving example: a token decoded on top of a prefilled prompt answers as the prefill of
the longer prompt does (recurrent against chunked state, absorbed against expanded attention)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import hybrid_serving_step as ex

pytestmark = pytest.mark.gpu


def test_decode_continues_the_prefill():
    lens, extra = (1, 16, 37, 128), 3
    prompts = [[(11 * i + 5 * j) % ex.VOCAB for j in range(n + extra)] for i, n in enumerate(lens)]
    whole = ex.Model(len(lens), max_tokens=140)
    logits, cu = whole.prefill(prompts)
    step = ex.Model(len(lens), max_tokens=140)
    step.prefill([p[:n] for p, n in zip(prompts, lens)])
    for k in range(extra):
        tokens = torch.tensor([p[n + k] for p, n in zip(prompts, lens)], device="cuda")
        got = step.decode(tokens)
        want = logits[torch.tensor([int(cu[i]) + n + k for i, n in enumerate(lens)], device="cuda")]
        # four layers of bf16 activations: each layer rounds about ten times at 2^-9 of its size, a few
        # of them on either side of the comparison: relative error about sqrt(80) 2^-9 < 0.02 a side
        assert (got.float() - want.float()).norm() <= 0.04 * want.float().norm(), k
    assert int(step.status) == 0 and int(whole.status) == 0


def test_the_example_runs(capsys):
    ex.main(steps=3)
    out = capsys.readouterr().out
    assert "step 2" in out and "nan" not in out
