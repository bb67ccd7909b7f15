"""Sums of the layer calls keep fp32 however long they are, in both element types."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


SIZE = 4096   # of the output: whole tiles for every SM, so that the contraction is not split over them


def positive(rows, cols, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.rand(rows, cols, generator=g, device="cuda").to(BF16)


def cancelling_product(op, K):
    """(result, sum of its terms' magnitudes) of a bfloat16 product of which the second half
    of the contraction takes away what the first half gives: zero."""
    b = binding()
    out = torch.empty(SIZE, SIZE, dtype=BF16, device="cuda")
    ids = torch.full((SIZE,), -1, dtype=torch.int32, device="cuda")
    x, w = positive(K // 2, SIZE, 1), positive(K // 2, SIZE, 2)      # x^T w, K-long columns
    if op == "weight gradient":
        q, e = b.act8_store_into(torch.cat((x, x)), *b.act8_empty(K, SIZE))
        b.act8_weight_grad_into(q, e, torch.cat((w, -w)), out)
        x = b.act8_load_into(q, e, torch.empty(K, SIZE, dtype=BF16, device="cuda"))[:K // 2]
    else:
        X, W = torch.cat((x, x)).t().contiguous(), torch.cat((w, -w))
        if op == "forward":
            none = torch.empty(0, K, 1, device="cuda", dtype=BF16)
            b.lora_into(X, W, none, none.new_empty(0, 1, SIZE), ids, out)
        else:
            b.lora_backward_into(X, out, W.t().contiguous(), torch.empty(0, SIZE, 1, device="cuda", dtype=BF16),
                                 torch.empty(0, 1, K, device="cuda", dtype=BF16), ids,
                                 torch.empty(SIZE, 1, device="cuda"), dX=out)
    return out.float(), 2 * (x.float().t() @ w.float())


@pytest.mark.parametrize("K", [8192, 8194, 65536, 200000])
@pytest.mark.parametrize("op", ["forward", "input gradient", "weight gradient"])
def test_a_long_bfloat16_sum_has_no_bias(op, K):
    """The tensor core's sums of at most 8192 k (512 instructions) truncate, each by up to
    2^-23 of the sum so far, which is half the last one on average: 3.1e-5 of the terms'
    magnitudes at most.  What is longer is added up in fp32 to nearest, another 25 * 2^-24."""
    got, mag = cancelling_product(op, K)
    assert float((got.abs() / mag).max()) <= 3.3e-5
