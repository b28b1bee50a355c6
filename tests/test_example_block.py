"""The example that runs the operators together: it learns, and decoding agrees with the pass."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_train_and_decode_a_memory_block():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import test_neural_memory_gb300 as ttm
    ttm.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_memory_block.py")
    spec = importlib.util.spec_from_file_location("train_memory_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, off = example.main(40)
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) / 5 < 0.8 * losses[0], losses
    # y is bf16 and passes a bf16 projection and memory either way: the scan's parity bound
    assert off < 2e-2
