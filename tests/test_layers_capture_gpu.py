"""Every layer call captured once in a graph and replayed on new inputs gives, bit for bit, what
it gives when it is called."""
import pytest
import torch

from _layers import row_ids

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def captured(inputs, outputs, call):
    """The outputs of a replay on fresh inputs against those of a call on them."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (11, 12):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for t in inputs:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        for t in outputs:
            t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outputs]
        for t in outputs:
            t.fill_(55)
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, outputs))
    assert binding().device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 8, 20, 60, 300, 1500])
def test_adapters(M, dtype):
    b, K, N, L, R = binding(), 264, 520, 4, 24
    z = lambda *s: torch.randn(*s, device="cuda").to(dtype)   # noqa: E731
    X, W, A, B, dY = z(M, K), z(K, N), z(L, K, R), z(L, R, N), z(M, N)
    ids, scale = row_ids(M, L, "mixed", 3).cuda(), torch.rand(L, device="cuda") + 0.5
    ranks = torch.tensor([24, 7, 0, 16], dtype=torch.int32, device="cuda")
    Y, H, bias = z(M, N), torch.zeros(M, R, device="cuda"), z(N)
    captured([X, W, A, B, bias], [Y, H], lambda: b.lora_into(X, W, A, B, ids, Y, scale=scale, ranks=ranks, bias=bias, H=H))
    dX, dA, dB = z(M, K), z(L, K, R), z(L, R, N)
    captured([X, W, A, B, dY, H], [dX, dA, dB],
             lambda: b.lora_backward_into(dY, X, W, A, B, ids, H, dX=dX, dA=dA, dB=dB, scale=scale, ranks=ranks))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,N", [(3, 40, 24), (300, 264, 520), (2000, 67, 130)])
def test_checkpoints(M, K, N, dtype):
    b = binding()
    z = lambda *s: torch.randn(*s, device="cuda").to(dtype)   # noqa: E731
    Z, Y, back, dY, dZ, dOut, dW = z(M, K), z(M, K), z(M, K), z(M, K), z(M, K), z(M, N), z(K, N)
    q, e = b.act8_empty(M, K)

    def step():
        b.act8_store_into(Z, q, e, act="gelu", Y=Y)
        b.act8_load_into(q, e, back)
        b.act8_grad_into(q, e, dY, dZ, act="gelu")
        b.act8_weight_grad_into(q, e, dOut, dW)
    captured([Z, dY, dOut], [q, e, Y, back, dZ, dW], step)
    W, A, B = z(K, N), z(2, K, 8), z(2, 8, N)
    H, dX, dA, dB = torch.randn(M, 8, device="cuda"), z(M, K), z(2, K, 8), z(2, 8, N)
    ids = row_ids(M, 2, "runs", 5).cuda()
    captured([dOut, W, A, B, H], [dX, dA, dB],
             lambda: b.lora_backward_into(dOut, (q, e), W, A, B, ids, H, dX=dX, dA=dA, dB=dB))
