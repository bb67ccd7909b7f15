"""Refusals of the adapter layer's and the checkpoints' entry points, on the CPU: every
case returns or raises before any CUDA call."""
import ctypes

import pytest
import torch

from dense_fp32_gemm_02_gb300 import build as sgbuild

OK, INVALID, TOO_LARGE = 0, 1, 6


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(sgbuild.build())


P = 0x100000   # 16-byte aligned addresses that nothing dereferences
i, ll, f, p = ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_void_p

ARGS = {
    "sgemm_lora": dict(
        type=(i, 0), M=(i, 4), N=(i, 8), K=(i, 6), L=(i, 2), R=(i, 3), X=(p, P), ldx=(i, 6),
        W=(p, 2 * P), ldw=(i, 8), A=(p, 3 * P), lda=(i, 3), stride_a=(ll, 18), B=(p, 4 * P),
        ldb=(i, 8), stride_b=(ll, 24), ids=(p, 5 * P), ranks=(p, None), scales=(p, None),
        bias=(p, None), H=(p, None), ldh=(i, 0), Y=(p, 6 * P), ldy=(i, 8), stream=(p, None)),
    "sgemm_lora_backward": dict(
        type=(i, 0), M=(i, 4), N=(i, 8), K=(i, 6), L=(i, 2), R=(i, 3), dY=(p, P), lddy=(i, 8),
        X=(p, 2 * P), ldx=(i, 6), q=(p, None), ldq=(i, 0), e=(p, None), lde=(i, 0), W=(p, 3 * P),
        ldw=(i, 8), A=(p, 4 * P), lda=(i, 3), stride_a=(ll, 18), B=(p, 5 * P), ldb=(i, 8),
        stride_b=(ll, 24), ids=(p, 6 * P), ranks=(p, None), scales=(p, None), H=(p, 7 * P),
        ldh=(i, 3), dX=(p, 8 * P), lddx=(i, 6), dA=(p, 9 * P), ldda=(i, 3), stride_da=(ll, 18),
        dB=(p, 10 * P), lddb=(i, 8), stride_db=(ll, 24), stream=(p, None)),
    "sgemm_act8_store": dict(
        type=(i, 0), M=(i, 4), K=(i, 40), Z=(p, P), ldz=(i, 40), act=(i, 0), q=(p, 2 * P),
        ldq=(i, 40), e=(p, 3 * P), lde=(i, 2), Y=(p, None), ldy=(i, 0), stream=(p, None)),
    "sgemm_act8_load": dict(
        type=(i, 0), M=(i, 4), K=(i, 40), q=(p, 2 * P), ldq=(i, 40), e=(p, 3 * P), lde=(i, 2),
        X=(p, P), ldx=(i, 40), stream=(p, None)),
    "sgemm_act8_grad": dict(
        type=(i, 0), M=(i, 4), K=(i, 40), q=(p, 2 * P), ldq=(i, 40), e=(p, 3 * P), lde=(i, 2),
        act=(i, 2), dY=(p, P), lddy=(i, 40), dZ=(p, 4 * P), lddz=(i, 40), stream=(p, None)),
    "sgemm_act8_weight_grad": dict(
        type=(i, 0), M=(i, 4), N=(i, 8), K=(i, 40), q=(p, 2 * P), ldq=(i, 40), e=(p, 3 * P),
        lde=(i, 2), dY=(p, P), lddy=(i, 8), beta=(f, 0.0), dW=(p, 4 * P), lddw=(i, 8),
        stream=(p, None)),
}


def call(lib, entry, **change):
    spec = dict(ARGS[entry])
    fn = getattr(lib, entry)
    fn.argtypes, fn.restype = [t for t, _ in spec.values()], ctypes.c_int
    return fn(*[change.pop(k, v) for k, (_, v) in spec.items()])


REFUSED = [
    ("sgemm_lora", dict(type=2)), ("sgemm_lora", dict(M=-1)), ("sgemm_lora", dict(K=-1)),
    ("sgemm_lora", dict(R=0)), ("sgemm_lora", dict(R=129)), ("sgemm_lora", dict(L=-1)),
    ("sgemm_lora", dict(L=1025)), ("sgemm_lora", dict(X=None)), ("sgemm_lora", dict(X=P + 2)),
    ("sgemm_lora", dict(type=1, X=P + 1)), ("sgemm_lora", dict(ldx=5)), ("sgemm_lora", dict(W=None)),
    ("sgemm_lora", dict(ldw=7)), ("sgemm_lora", dict(A=None)), ("sgemm_lora", dict(lda=2)),
    ("sgemm_lora", dict(stride_a=17)), ("sgemm_lora", dict(stride_b=-24)), ("sgemm_lora", dict(B=None)),
    ("sgemm_lora", dict(ids=None)), ("sgemm_lora", dict(ids=P + 2)), ("sgemm_lora", dict(ranks=P + 1)),
    ("sgemm_lora", dict(scales=P + 2)), ("sgemm_lora", dict(bias=P + 2)), ("sgemm_lora", dict(Y=None)),
    ("sgemm_lora", dict(ldy=7)), ("sgemm_lora", dict(H=P, ldh=2)), ("sgemm_lora", dict(H=P + 2, ldh=3)),
    ("sgemm_lora_backward", dict(type=-1)), ("sgemm_lora_backward", dict(dY=None)),
    ("sgemm_lora_backward", dict(lddy=7)), ("sgemm_lora_backward", dict(dA=None)),
    ("sgemm_lora_backward", dict(dB=None)), ("sgemm_lora_backward", dict(H=None)),
    ("sgemm_lora_backward", dict(ldh=2)), ("sgemm_lora_backward", dict(X=None)),
    ("sgemm_lora_backward", dict(X=None, q=P, ldq=6)), ("sgemm_lora_backward", dict(X=None, q=P, ldq=5, e=P, lde=1)),
    ("sgemm_lora_backward", dict(ldx=5)), ("sgemm_lora_backward", dict(W=None)),
    ("sgemm_lora_backward", dict(lddx=5)), ("sgemm_lora_backward", dict(stride_da=17)),
    ("sgemm_lora_backward", dict(stride_db=23)), ("sgemm_lora_backward", dict(ids=None)),
    ("sgemm_act8_store", dict(type=3)), ("sgemm_act8_store", dict(K=-1)), ("sgemm_act8_store", dict(act=3)),
    ("sgemm_act8_store", dict(Z=None)), ("sgemm_act8_store", dict(Z=P + 2)), ("sgemm_act8_store", dict(ldz=39)),
    ("sgemm_act8_store", dict(q=None)), ("sgemm_act8_store", dict(ldq=39)), ("sgemm_act8_store", dict(lde=1)),
    ("sgemm_act8_store", dict(Y=P, ldy=39)), ("sgemm_act8_store", dict(Y=P + 1, ldy=40)),
    ("sgemm_act8_load", dict(X=None)), ("sgemm_act8_load", dict(e=None)), ("sgemm_act8_load", dict(ldx=39)),
    ("sgemm_act8_grad", dict(act=-1)), ("sgemm_act8_grad", dict(dY=None)), ("sgemm_act8_grad", dict(lddz=39)),
    ("sgemm_act8_weight_grad", dict(q=None)), ("sgemm_act8_weight_grad", dict(dY=None)),
    ("sgemm_act8_weight_grad", dict(dW=None)), ("sgemm_act8_weight_grad", dict(lddw=7)),
    ("sgemm_act8_weight_grad", dict(lde=1)), ("sgemm_act8_weight_grad", dict(N=-1)),
]


@pytest.mark.parametrize("entry,change", REFUSED)
def test_invalid_arguments_are_refused(lib, entry, change):
    assert call(lib, entry, **change) == INVALID


@pytest.mark.parametrize("entry", sorted(ARGS))
def test_sizes_past_the_limit_are_refused(lib, entry):
    for size in ("M", "K") + (("N",) if "N" in ARGS[entry] else ()):
        assert call(lib, entry, **{size: 2 ** 31 - 1}) == TOO_LARGE


@pytest.mark.parametrize("entry,change", [
    ("sgemm_lora", dict(M=0)), ("sgemm_lora", dict(N=0)), ("sgemm_lora_backward", dict(dX=None, dA=None, dB=None)),
    ("sgemm_lora_backward", dict(M=0, dA=None, dB=None)), ("sgemm_act8_store", dict(M=0, Z=None)),
    ("sgemm_act8_load", dict(K=0)), ("sgemm_act8_grad", dict(M=0)), ("sgemm_act8_weight_grad", dict(N=0)),
    ("sgemm_act8_weight_grad", dict(K=0, q=None))])
def test_nothing_to_compute_is_a_success(lib, entry, change):
    assert call(lib, entry, **change) == OK


# ------------------------------------------------------------------ the binding
def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_the_binding_refuses_host_tensors_and_other_types():
    from dense_fp32_gemm_02_gb300 import binding as b
    ids = t(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="X must be a CUDA float32 or bfloat16"):
        b.lora_into(t(4, 6), t(6, 8), t(2, 6, 3), t(2, 3, 8), ids, t(4, 8))
    with pytest.raises(TypeError, match="dY must be a CUDA"):
        b.lora_backward_into(t(4, 8), t(4, 6), t(6, 8), t(2, 6, 3), t(2, 3, 8), ids, t(4, 3))
    q, e = t(4, 40, dtype=torch.int8), t(4, 2, dtype=torch.int8)
    with pytest.raises(TypeError, match="Z must be a CUDA"):
        b.act8_store_into(t(4, 40, dtype=torch.float16), q, e)
    with pytest.raises(TypeError, match="X must be a CUDA"):
        b.act8_load_into(q, e, t(4, 40))
    with pytest.raises(TypeError, match="dY must be a CUDA"):
        b.act8_grad_into(q, e, t(4, 40), t(4, 40))
    with pytest.raises(TypeError, match="dY must be a CUDA"):
        b.act8_weight_grad_into(q, e, t(4, 8), t(40, 8))


def test_views_and_shapes():
    from dense_fp32_gemm_02_gb300 import binding as b
    assert b._matrix("Y", None, 3, 4) == (None, 0) and b._stack("dA", None, 2, 3, 4) == (None, 0, 0)
    x = t(5, 9)[:, :4]
    assert b._matrix("X", x, 5, 4) == (x.data_ptr(), 9)
    with pytest.raises(ValueError, match=r"X must be \(4, 4\)"):
        b._matrix("X", x, 4, 4)
    with pytest.raises(ValueError, match="contiguous"):
        b._matrix("X", t(4, 5).t(), 5, 4)
    s = t(3, 5, 9)[:, :, :4]
    assert b._stack("A", s, 3, 5, 4) == (s.data_ptr(), 9, 45)
    assert b._stack("A", s[:1], 1, 5, 4)[2] == 0
    with pytest.raises(ValueError, match="A must be"):
        b._stack("A", s, 2, 5, 4)
    with pytest.raises(ValueError, match="rank must be 1 to 128"):
        b._adapters(t(2, 6, 129), t(2, 129, 8), None, 4, None, None, "cpu")
    with pytest.raises(ValueError, match="at most 1024"):
        b._adapters(t(1025, 1, 1), t(1025, 1, 1), None, 4, None, None, "cpu")
