"""The norm's entry point of rows without columns, on the CPU: it looks at the scales alone."""
from test_forward_host import INVALID, OK, P, call, lib   # noqa: F401  (lib is a fixture)


def test_scales_of_rows_without_columns(lib):   # noqa: F811
    nothing = dict(K=0, S=None, Y=None, q=None)
    assert call(lib, "sgemm_rmsnorm", **nothing, scale=None) == OK
    assert call(lib, "sgemm_rmsnorm", **nothing, scale=P + 2) == INVALID
    assert call(lib, "sgemm_rmsnorm", **nothing, M=0, scale=P + 2) == OK
