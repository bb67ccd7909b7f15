"""The gated block's backward pass of one to four rows, its sums of a few terms and its long ones, against 64 bits."""
import pytest
import torch

from test_gated_gpu import _gpu, backward_args, binding, check_backward, empty_gradients   # noqa: F401  (_gpu is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("M,N,K", [(4, 77, 2000), (1, 77, 2000), (4, 2000, 77), (2, 1, 1)])
def test_backward_of_few_rows(M, N, K, dtype, act):
    b = binding()
    args = backward_args(M, N, K, dtype, 20)
    dX, dWg, dWu = empty_gradients(M, N, K, dtype)
    b.gated_backward_into(*args, dX=dX, dWg=dWg, dWu=dWu, act=act)
    check_backward(args, act, dX, dWg, dWu)
    assert b.device_status() == 0
