"""examples/hybrid_decode.py: speculative steps, a fork, a release and a compaction against one prompt per sequence."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")


def example():
    spec = importlib.util.spec_from_file_location("hybrid_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("seed", [0, 1])
def test_speculative_steps_give_the_prompt_logits_in_32_bits(seed):
    torch.backends.cuda.matmul.allow_tf32 = False
    sequences, per_step, difference = example().run(torch.float32, seed=seed)
    assert len(sequences) == 5 and per_step >= 1
    # logits are sums of 128 products of about 1; some hundred roundings of 2^-24 each lie between the two ways
    assert difference < 128 * 100 * 2.0 ** -24
