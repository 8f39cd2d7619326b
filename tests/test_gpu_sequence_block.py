"""The example block runs the operators together: it learns to recall (the
same block of plain operations has under a third of the first loss left after
60 steps, so half is asked for), and its token-by-token run gives the whole-sequence one's logits.

Tolerance, fixed before the first run: both runs are fp32 sums of some
hundred terms per layer, the convolution through transforms of 512 points
(1e-5 log2 of that, relative): 1e-4 of the largest logit.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sequence_block.py")
    spec = importlib.util.spec_from_file_location("sequence_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_and_decoding(example):
    block, losses = example.train(steps=60, tokens=64, report=lambda line: None)
    assert all(x == x for x in losses)
    assert sum(losses[-5:]) / 5 < losses[0] / 2
    assert example.decode_error(block) <= 1e-4
