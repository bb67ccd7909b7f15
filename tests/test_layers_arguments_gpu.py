"""Which arguments of the layer calls may be left out, and what the others' absence raises."""
import pytest
import torch

pytestmark = pytest.mark.gpu
M, K, N, L, R = 70, 64, 96, 2, 4


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def tensors():
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    return dict(X=r(M, K), dY=r(M, N), W=r(K, N), A=r(L, K, R), B=r(L, R, N), H=r(M, R), Y=r(M, N), dX=r(M, K),
                dA=r(L, K, R), dB=r(L, R, N), Z=r(M, K), dZ=r(M, K), dW=r(K, N),
                ids=torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32),
                q=torch.zeros(M, K, dtype=torch.int8, device="cuda"), e=torch.zeros(M, 2, dtype=torch.int8, device="cuda"))


def test_the_input_gradient_alone_needs_neither_x_nor_h():
    b, t = binding(), tensors()
    whole = b.lora_backward_into(t["dY"], t["X"], t["W"], t["A"], t["B"], t["ids"], t["H"], dX=t["dX"], dA=t["dA"],
                                 dB=t["dB"])[0].clone()
    for X in (t["X"], (t["q"], t["e"]), None):
        t["dX"].fill_(float("nan"))
        dX, dA, dB = b.lora_backward_into(t["dY"], X, t["W"], t["A"], t["B"], t["ids"], None, dX=t["dX"])
        assert torch.equal(dX, whole) and dA is None and dB is None


def test_the_stacks_gradients_need_x_and_h():
    b, t = binding(), tensors()
    given = dict(dX=t["dX"], dA=t["dA"], dB=t["dB"])
    with pytest.raises(TypeError, match="H must be"):
        b.lora_backward_into(t["dY"], t["X"], t["W"], t["A"], t["B"], t["ids"], None, **given)
    with pytest.raises(TypeError, match="X must be"):
        b.lora_backward_into(t["dY"], None, t["W"], t["A"], t["B"], t["ids"], t["H"], **given)


CALLS = {"lora_into": ("X", "W", "A", "B", "ids", "Y"), "lora_backward_into": ("dY", "X", "W", "A", "B", "ids", "H"),
         "act8_store_into": ("Z", "q", "e"), "act8_load_into": ("q", "e", "X"), "act8_grad_into": ("q", "e", "dY", "dZ"),
         "act8_weight_grad_into": ("q", "e", "dY", "dW")}


@pytest.mark.parametrize("bad", [None, 3.0, [1.0]], ids=str)
@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS.items() for n in names])
def test_what_is_missing_or_no_tensor_raises_a_type_error(call, name, bad):
    b, t = binding(), tensors()
    more = dict(dX=t["dX"], dA=t["dA"], dB=t["dB"]) if call == "lora_backward_into" else {}
    args = [bad if n == name else t[n] for n in CALLS[call]]
    with pytest.raises(TypeError, match=f"{name} must be"):
        getattr(b, call)(*args, **more)


def test_no_adapters_need_no_ids():
    b, t = binding(), tensors()
    none = torch.empty(0, K, 1, device="cuda")
    b.lora_into(t["X"], t["W"], none, none.new_empty(0, 1, N), None, t["Y"])
    ref = t["X"].double() @ t["W"].double()
    mag = t["X"].double().abs() @ t["W"].double().abs()
    assert bool(((t["Y"].double() - ref).abs() <= (K + 16) * 2.0 ** -23 * mag).all())


def test_the_device_of_an_empty_checkpoint():
    b = binding()
    for device in (None, 0, "cuda:0", torch.device("cuda", 0)):
        assert all(t.device == torch.device("cuda", 0) for t in b.act8_empty(3, 40, device))
    assert all(t.device.type == "cpu" for t in b.act8_empty(3, 40, "cpu"))


@pytest.mark.parametrize("rows", [1, 5, 40, 300, 1500])
@pytest.mark.parametrize("cols", [96, 0])
def test_h_of_an_empty_stack_is_zero(rows, cols):
    """Every row is one without an adapter; what lies beside H's columns is left alone."""
    b = binding()
    X, W = torch.randn(rows, K, device="cuda"), torch.randn(K, cols, device="cuda")
    Y = torch.empty(rows, cols, device="cuda")
    H = torch.full((rows, R + 3), 7.0, device="cuda")
    b.lora_into(X, W, X.new_empty(0, K, R), X.new_empty(0, R, cols), None, Y, H=H[:, :R])
    assert bool((H[:, :R] == 0).all()) and bool((H[:, R:] == 7).all())
    plain = torch.empty_like(Y)
    b.lora_into(X, W, X.new_empty(0, K, R), X.new_empty(0, R, cols), None, plain)
    assert torch.equal(Y, plain) and b.device_status() == b.SGEMM_OK
