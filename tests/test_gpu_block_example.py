"""The example that uses the operators around the projections together: its
loss falls, and the merged projection serves one token as the trained layer
did (the merged weight is rounded to bf16 once more: 2^-8 relative per weight,
and the outputs of both ways to bf16: within 2e-2 together, the layer tests'
bound)."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "block_step.py")


def test_example_trains_and_serves():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    spec = importlib.util.spec_from_file_location("block_step", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, off = example.main(steps=30, quiet=True)
    import orthogonal_reparameterized_packed_gb300 as poetx
    assert poetx.poetx_device_status() == 0
    assert all(b == b for b in losses)
    assert losses[-1] < 0.5 * losses[0]
    assert off <= 2e-2
