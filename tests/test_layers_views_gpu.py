"""Tensors whose rows overlap are refused by every layer call, as input and as output; what
made them contiguous is taken."""
import pytest
import torch

pytestmark = pytest.mark.gpu
M, K, N, L, R = 8, 64, 96, 2, 4


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def overlapping(shape, dtype=torch.float32):
    """An expanded matrix, and one whose rows start one after the other."""
    rows, cols = shape[-2:]
    flat = torch.zeros(cols + rows, dtype=dtype, device="cuda")
    for strides in ((0, 1), (1, 1)):
        view = flat.as_strided((rows, cols), strides)
        yield view if len(shape) == 2 else view.expand(*shape)


def calls():
    """name -> (function, its tensors by name)."""
    from dense_fp32_gemm_02_gb300 import binding as b
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)   # noqa: E731
    q, e = lambda: z(M, K, dtype=torch.int8), lambda: z(M, 2, dtype=torch.int8)   # noqa: E731
    adapters = dict(W=z(K, N), A=z(L, K, R), B=z(L, R, N), ids=z(M, dtype=torch.int32))
    return {
        "lora": (b.lora_into, dict(X=z(M, K), **adapters, Y=z(M, N), H=z(M, R))),
        "lora_backward": (b.lora_backward_into, dict(
            dY=z(M, N), X=z(M, K), **adapters, H=z(M, R), dX=z(M, K), dA=z(L, K, R), dB=z(L, R, N))),
        "act8_store": (b.act8_store_into, dict(Z=z(M, K), q=q(), e=e(), Y=z(M, K))),
        "act8_load": (b.act8_load_into, dict(q=q(), e=e(), X=z(M, K))),
        "act8_grad": (b.act8_grad_into, dict(q=q(), e=e(), dY=z(M, K), dZ=z(M, K))),
        "act8_weight_grad": (b.act8_weight_grad_into, dict(q=q(), e=e(), dY=z(M, N), dW=z(K, N))),
    }


@pytest.mark.parametrize("name", ["lora", "lora_backward", "act8_store", "act8_load", "act8_grad", "act8_weight_grad"])
def test_overlapping_rows_are_refused(name):
    from dense_fp32_gemm_02_gb300 import binding as b
    fn, given = calls()[name]
    fn(**given)
    launches = b.kernel_launch_count()
    for what, t in given.items():
        if t.dim() == 1:
            continue
        for view in overlapping(t.shape, t.dtype):
            with pytest.raises(ValueError, match=f"{what}: rows must not overlap"):
                fn(**{**given, what: view})
    assert b.kernel_launch_count() == launches
    torch.cuda.synchronize()
    assert b.device_status() == b.SGEMM_OK


def test_an_expanded_gradient_made_contiguous():
    from dense_fp32_gemm_02_gb300 import binding as b
    fn, given = calls()["lora_backward"]
    dY = torch.randn(1, N, device="cuda").expand(M, N)
    given["W"].normal_()
    fn(**{**given, "dY": dY.contiguous()})
    ref = (dY[:1].double() @ given["W"].double().t()).expand(M, K)
    # a sum of N products in fp32, each within 2^-23 of its magnitude
    mag = (dY[:1].double().abs() @ given["W"].double().abs().t()).expand(M, K)
    assert bool(((given["dX"].double() - ref).abs() <= (N + 16) * 2.0 ** -23 * mag).all())
    assert b.device_status() == b.SGEMM_OK
