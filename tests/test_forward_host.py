"""Refusals of the norm's, the 8-bit product's and the gated block's entry points, on the CPU: every
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
i, f, p = ctypes.c_int, ctypes.c_float, ctypes.c_void_p

ARGS = {
    "sgemm_rmsnorm": dict(
        type=(i, 0), M=(i, 4), K=(i, 40), X=(p, P), ldx=(i, 40), R=(p, 2 * P), ldr=(i, 40), w=(p, 3 * P), eps=(f, 1e-6),
        S=(p, 4 * P), lds=(i, 40), Y=(p, 5 * P), ldy=(i, 40), q=(p, 6 * P), ldq=(i, 40), scale=(p, 7 * P), stream=(p, None)),
    "sgemm_rmsnorm_backward": dict(
        type=(i, 0), M=(i, 4), K=(i, 40), dY=(p, P), lddy=(i, 40), V=(p, 2 * P), ldv=(i, 40), w=(p, 3 * P), eps=(f, 1e-6),
        dS=(p, 4 * P), ldds=(i, 40), dX=(p, 5 * P), lddx=(i, 40), dw=(p, 6 * P), stream=(p, None)),
    "sgemm_linear8": dict(
        type=(i, 0), M=(i, 4), N=(i, 8), K=(i, 40), X=(p, None), ldx=(i, 0), q=(p, P), ldq=(i, 40), scale=(p, 2 * P),
        W=(p, 3 * P), ldw=(i, 8), wscale=(p, 4 * P), bias=(p, None), Y=(p, 5 * P), ldy=(i, 8), stream=(p, None)),
    "sgemm_gated": dict(
        type=(i, 0), M=(i, 4), N=(i, 8), K=(i, 6), X=(p, P), ldx=(i, 6), Wg=(p, 2 * P), ldwg=(i, 8), Wu=(p, 3 * P), ldwu=(i, 8),
        act=(i, 3), G=(p, 4 * P), ldg=(i, 8), U=(p, 5 * P), ldu=(i, 8), H=(p, 6 * P), ldh=(i, 8), stream=(p, None)),
    "sgemm_gated_backward": dict(
        type=(i, 0), M=(i, 4), N=(i, 8), K=(i, 6), act=(i, 3), dH=(p, P), lddh=(i, 8), X=(p, 2 * P), ldx=(i, 6), G=(p, 3 * P),
        ldg=(i, 8), U=(p, 4 * P), ldu=(i, 8), Wg=(p, 5 * P), ldwg=(i, 8), Wu=(p, 6 * P), ldwu=(i, 8), dX=(p, 7 * P), lddx=(i, 6),
        dWg=(p, 8 * P), lddwg=(i, 8), dWu=(p, 9 * P), lddwu=(i, 8), stream=(p, None)),
}
MATRICES = {   # matrix -> its pitch, columns and element (of float32)
    "sgemm_rmsnorm": {"X": ("ldx", 40, 4), "R": ("ldr", 40, 4), "S": ("lds", 40, 4), "Y": ("ldy", 40, 4), "q": ("ldq", 40, 1)},
    "sgemm_rmsnorm_backward": {"dY": ("lddy", 40, 4), "V": ("ldv", 40, 4), "dS": ("ldds", 40, 4), "dX": ("lddx", 40, 4)},
    "sgemm_linear8": {"q": ("ldq", 40, 1), "W": ("ldw", 8, 1), "Y": ("ldy", 8, 4)},
    "sgemm_gated": {"X": ("ldx", 6, 4), "Wg": ("ldwg", 8, 4), "Wu": ("ldwu", 8, 4), "G": ("ldg", 8, 4), "U": ("ldu", 8, 4),
                    "H": ("ldh", 8, 4)},
    "sgemm_gated_backward": {"dH": ("lddh", 8, 4), "X": ("ldx", 6, 4), "G": ("ldg", 8, 4), "U": ("ldu", 8, 4),
                             "Wg": ("ldwg", 8, 4), "Wu": ("ldwu", 8, 4), "dX": ("lddx", 6, 4), "dWg": ("lddwg", 8, 4),
                             "dWu": ("lddwu", 8, 4)},
}
MAY_BE_MISSING = {("sgemm_rmsnorm", "R"), ("sgemm_rmsnorm", "S"), ("sgemm_rmsnorm", "Y"), ("sgemm_rmsnorm_backward", "dS"),
                  ("sgemm_gated_backward", "dX")}


def call(lib, entry, **change):
    spec = dict(ARGS[entry])
    assert set(change) <= set(spec)
    fn = getattr(lib, entry)
    fn.argtypes, fn.restype = [t for t, _ in spec.values()], ctypes.c_int
    return fn(*[change.pop(k, v) for k, (_, v) in spec.items()])


@pytest.mark.parametrize("entry,name", [(e, m) for e, ms in MATRICES.items() for m in ms])
def test_bad_matrices_are_refused(lib, entry, name):
    pitch, columns, element = MATRICES[entry][name]
    assert call(lib, entry, **{pitch: columns - 1}) == INVALID
    if element > 1:
        assert call(lib, entry, **{name: P + 2}) == INVALID
        assert call(lib, entry, type=1, **{name: P + 1}) == INVALID
    if (entry, name) not in MAY_BE_MISSING:
        assert call(lib, entry, **{name: None}) == INVALID


REFUSED = [(e, dict(type=t)) for e in ARGS for t in (-1, 2)] + [(e, {s: -1}) for e in ARGS for s in ("M", "K")] + [
    ("sgemm_rmsnorm", dict(eps=-1e-9)), ("sgemm_rmsnorm", dict(eps=float("nan"))), ("sgemm_rmsnorm", dict(eps=float("inf"))),
    ("sgemm_rmsnorm", dict(w=None)), ("sgemm_rmsnorm", dict(w=P + 2)), ("sgemm_rmsnorm", dict(scale=None)),
    ("sgemm_rmsnorm", dict(scale=P + 2)), ("sgemm_rmsnorm", dict(S=None, Y=None, q=None, scale=None)),
    ("sgemm_rmsnorm", dict(S=5 * P)), ("sgemm_rmsnorm_backward", dict(eps=-1.0)), ("sgemm_rmsnorm_backward", dict(w=None)),
    ("sgemm_rmsnorm_backward", dict(dw=P + 2)), ("sgemm_rmsnorm_backward", dict(M=0, dw=P + 2)),
    ("sgemm_linear8", dict(scale=None)), ("sgemm_linear8", dict(scale=P + 2)), ("sgemm_linear8", dict(wscale=None)),
    ("sgemm_linear8", dict(wscale=P + 1)), ("sgemm_linear8", dict(bias=P + 2)), ("sgemm_linear8", dict(X=P + 2, ldx=40)),
    ("sgemm_linear8", dict(X=P, ldx=39)), ("sgemm_linear8", dict(N=-1)), ("sgemm_gated", dict(N=-1)),
    ("sgemm_gated", dict(act=4)), ("sgemm_gated", dict(act=-1)), ("sgemm_gated_backward", dict(act=4)),
    ("sgemm_gated_backward", dict(act=-1)), ("sgemm_gated_backward", dict(N=-1)),
]


@pytest.mark.parametrize("entry,change", REFUSED)
def test_invalid_arguments_are_refused(lib, entry, change):
    assert call(lib, entry, **change) == INVALID


@pytest.mark.parametrize("entry", sorted(ARGS))
def test_sizes_past_the_limit_are_refused(lib, entry):
    for size in ("M", "K") + (("N",) if "N" in ARGS[entry] else ()):
        assert call(lib, entry, **{size: 2 ** 31 - 1}) == TOO_LARGE


def test_a_sum_that_int32_may_not_hold_is_refused(lib):
    assert call(lib, "sgemm_linear8", K=131072, ldq=131072) == TOO_LARGE


def test_silu_is_the_gated_blocks_alone(lib):
    """The other entry points refuse it as any number past their activations."""
    lib.sgemm_ex.restype = ctypes.c_int
    ll = ctypes.c_longlong
    lib.sgemm_ex.argtypes = [i, i, i, f, p, i, ll, p, i, ll, f, p, i, ll, i, p, ll, i, p]
    assert lib.sgemm_ex(4, 4, 4, 1.0, P, 4, 0, 2 * P, 4, 0, 0.0, 3 * P, 4, 0, 1, None, 0, 3, None) == INVALID


@pytest.mark.parametrize("entry,change", [
    ("sgemm_rmsnorm", dict(M=0)), ("sgemm_rmsnorm", dict(K=0, S=None, Y=None, q=None, scale=None)),
    ("sgemm_rmsnorm_backward", dict(K=0)), ("sgemm_linear8", dict(M=0)), ("sgemm_linear8", dict(N=0)),
    ("sgemm_gated", dict(M=0)), ("sgemm_gated", dict(N=0)), ("sgemm_gated_backward", dict(dX=None, dWg=None, dWu=None)),
    ("sgemm_gated_backward", dict(K=0)), ("sgemm_gated_backward", dict(M=0, dWg=None, dWu=None))])
def test_nothing_to_compute_is_a_success(lib, entry, change):
    assert call(lib, entry, **change) == OK


# ------------------------------------------------------------------ the binding
def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_the_binding_refuses_host_tensors_and_other_types():
    from dense_fp32_gemm_02_gb300 import binding as b
    with pytest.raises(TypeError, match="X must be a CUDA float32 or bfloat16"):
        b.rmsnorm_into(t(4, 8), t(8), Y=t(4, 8))
    with pytest.raises(TypeError, match="dY must be a CUDA"):
        b.rmsnorm_backward_into(t(4, 8), t(4, 8), t(8), t(4, 8))
    with pytest.raises(TypeError, match="Y must be a CUDA"):
        b.linear8_into((t(4, 8, dtype=torch.int8), t(4)), t(8, 6, dtype=torch.int8), t(6), t(4, 6))
    with pytest.raises(TypeError, match="X must be a CUDA"):
        b.gated_into(t(4, 8, dtype=torch.float16), t(8, 6), t(8, 6), t(4, 6))
    with pytest.raises(TypeError, match="dH must be a CUDA"):
        b.gated_backward_into(t(4, 6), t(4, 8), t(8, 6), t(8, 6), t(4, 6), t(4, 6))


def test_activations_and_eps():
    from dense_fp32_gemm_02_gb300 import binding as b
    assert b._gate_number("silu") == 3 and b._gate_number("gelu") == 2 and "silu" not in b.ACTIVATIONS
    with pytest.raises(ValueError, match="act must be one of"):
        b._gate_number("swish")
    assert b._eps(0) == 0.0
    for bad in (-1e-6, float("nan"), float("inf"), 1e39):
        with pytest.raises(ValueError, match="eps must be"):
            b._eps(bad)


def test_the_package_offers_them():
    import dense_fp32_gemm_02_gb300 as package
    for name in ("rmsnorm_into", "rmsnorm_backward_into", "linear8_into", "gated_into", "gated_backward_into"):
        assert name in package.__all__ and callable(getattr(package, name)) and getattr(package, name).__doc__
