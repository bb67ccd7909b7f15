"""The example that fine-tunes adapters from 8-bit checkpoints and serves them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(cuda_device):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import adapter_finetune
    finally:
        sys.path.pop(0)
    return adapter_finetune


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_adapters_learn_and_serve(example, dtype):
    """The loss falls by a third; a decode step gives the prefill's rows up to the order of
    its sums (three fp32 sums of up to 1024 terms of order 1; in bfloat16, a rounding of
    each layer's result, 2^-8 of values up to about 8)."""
    model = example.Model(dtype=dtype)
    losses, (X, ids) = example.train(model, steps=40)
    assert losses[-1] < losses[0] * 2 / 3, losses
    rows = torch.arange(0, X.shape[0], 100, device="cuda")
    token, _ = model.forward(X[rows].contiguous(), ids[rows].contiguous())
    whole, _ = model.forward(X, ids)
    most = 1e-4 if dtype == torch.float32 else 8 * 2.0 ** -8 * 3
    assert float((token.float() - whole[rows].float()).abs().max()) <= most
