"""Row pitches that the GEMM entry points do not take, on the CPU: rows that overlap, and strides
and sizes that an int does not hold, are refused before any library call."""
import pytest
import torch

from dense_fp32_gemm_02_gb300 import binding as b


@pytest.mark.parametrize("view", [torch.zeros(64).expand(8, 64), torch.zeros(120).unfold(0, 64, 8),
                                  torch.zeros(1, 1).expand(8, 1)])
def test_overlapping_rows_are_refused(view):
    with pytest.raises(ValueError, match="overlap"):
        b._ld(view, view.shape[1])


class View:
    """A 2-D view that needs no memory."""
    def __init__(self, shape, strides):
        self.shape, self._strides = torch.Size(shape), strides

    def dim(self):
        return 2

    def numel(self):
        return self.shape.numel()

    def size(self, i):
        return self.shape[i]

    def stride(self, i):
        return self._strides[i]


def test_strides_past_an_int_are_refused():
    assert b._ld(View((2, 64), (2 ** 31 - 1, 1)), 64) == 2 ** 31 - 1
    for stride in (2 ** 31, 2 ** 32 + 64):
        with pytest.raises(ValueError, match="apart"):
            b._ld(View((2, 64), (stride, 1)), 64)


@pytest.mark.parametrize("M,N,K", [(2 ** 31, 1, 1), (1, 2 ** 32 + 5, 1), (1, 1, 2 ** 33)])
def test_sizes_past_an_int_are_too_large(M, N, K):
    A, B, C = View((M, K), (K, 1)), View((K, N), (N, 1)), View((M, N), (N, 1))
    with pytest.raises(b.SgemmError) as e:
        b._shapes(A, B, C)
    assert e.value.status == b.SGEMM_ERR_TOO_LARGE
