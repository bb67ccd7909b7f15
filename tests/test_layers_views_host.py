"""What a tensor's strides may be, on the CPU: the layer calls' matrices and stacks whose rows
overlap, or whose strides or sizes an int does not hold, are refused before any library call."""
import pytest
import torch

from dense_fp32_gemm_02_gb300 import binding as b


def t(*shape):
    return torch.zeros(*shape)


class View:
    """A view that needs no memory: what _matrix() and _stack() ask of a tensor."""
    def __init__(self, shape, strides):
        self.shape, self._strides = torch.Size(shape), strides

    def stride(self):
        return self._strides

    def data_ptr(self):
        return 0x100000


@pytest.mark.parametrize("view", [t(64).expand(8, 64), t(1, 64).expand(8, 64), t(120).unfold(0, 64, 8),
                                  t(71).as_strided((8, 64), (1, 1)), t(1, 1).expand(8, 1), t(64 * 7 + 63).as_strided((8, 64), (63, 1))])
def test_overlapping_rows_are_refused(view):
    with pytest.raises(ValueError, match="X: .*overlap"):
        b._matrix("X", view, *view.shape)
    with pytest.raises(ValueError, match="A: .*overlap"):
        b._stack("A", view.unsqueeze(0), 1, *view.shape)
    with pytest.raises(ValueError, match="A: .*overlap"):
        b._stack("A", view.unsqueeze(0).expand(3, *view.shape), 3, *view.shape)


def test_the_gradient_of_a_sum_over_rows_is_such_a_view():
    seen = []

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return x * 2

        @staticmethod
        def backward(ctx, dY):
            seen.append(dY)
            return dY * 2

    Layer.apply(t(8, 64).requires_grad_()).sum(0).backward(torch.arange(64.0))
    assert seen[0].stride() == (0, 1)
    with pytest.raises(ValueError, match="dY: .*overlap"):
        b._matrix("dY", seen[0], 8, 64)
    dY = seen[0].contiguous()
    assert b._matrix("dY", dY, 8, 64) == (dY.data_ptr(), 64)


@pytest.mark.parametrize("rows,cols,strides,pitch", [
    (1, 64, (0, 1), 64), (1, 64, (7, 1), 64), (8, 0, (1, 1), 1), (0, 64, (64, 1), 64), (0, 0, (1, 1), 1),
    (8, 1, (1, 1), 1), (8, 1, (5, 0), 5), (8, 64, (64, 1), 64), (8, 64, (2 ** 31 - 1, 1), 2 ** 31 - 1)])
def test_views_that_hold_their_rows_apart(rows, cols, strides, pitch):
    assert b._matrix("X", View((rows, cols), strides), rows, cols) == (0x100000, pitch)
    assert b._stack("A", View((2, rows, cols), (2 ** 40, *strides)), 2, rows, cols) == (0x100000, pitch, 2 ** 40)


@pytest.mark.parametrize("stride", [2 ** 31, 2 ** 32 + 64, 2 ** 33])
def test_rows_too_far_apart_are_refused(stride):
    with pytest.raises(ValueError, match="X: .*apart"):
        b._matrix("X", View((8, 64), (stride, 1)), 8, 64)
    with pytest.raises(ValueError, match="A: .*apart"):
        b._stack("A", View((2, 8, 64), (8 * stride, stride, 1)), 2, 8, 64)


@pytest.mark.parametrize("rows,cols", [(2 ** 31, 1), (2 ** 32 + 3, 1), (1, 2 ** 31), (1, 2 ** 32 + 8), (2 ** 32, 0)])
def test_sizes_past_an_int_are_too_large(rows, cols):
    with pytest.raises(b.SgemmError) as e:
        b._matrix("X", View((rows, cols), (max(cols, 1), 1)), rows, cols)
    assert e.value.status == b.SGEMM_ERR_TOO_LARGE
    with pytest.raises(b.SgemmError) as e:
        b._stack("A", View((2, rows, cols), (rows * cols, max(cols, 1), 1)), 2, rows, cols)
    assert e.value.status == b.SGEMM_ERR_TOO_LARGE
