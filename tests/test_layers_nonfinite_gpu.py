"""Infinities and NaNs through the layer calls: where they must show and where they must not."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def same(got, want):
    """Equal, a NaN for a NaN."""
    got, want = got.cpu().double(), want.double()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(7), want.nan_to_num(7))


@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [64, 67])     # rows read 16 bytes at a time, and of any alignment
def test_activations_of_infinities(K, dtype, act):
    """0.5 z (1 + erf(z / sqrt 2)) is +inf at +inf and, 0 times infinity, NaN at -inf; relu(-inf)
    is 0; a NaN stays one; the largest finite values are not past anything."""
    b = binding()
    top = torch.finfo(dtype).max
    special = [INF, -INF, NAN, top, -top, 1.0]
    want = {"none": special, "relu": [INF, 0, NAN, top, 0, 1.0], "gelu": [INF, NAN, NAN, top, 0, None]}[act]
    z = torch.randn(6, K, generator=torch.Generator().manual_seed(1)).to(dtype)
    plain = torch.empty(6, K, dtype=dtype, device="cuda")
    b.act8_store_into(z.cuda(), *b.act8_empty(6, K), act=act, Y=plain)
    z[:, 5] = torch.tensor(special, dtype=dtype)
    y = torch.empty_like(plain)
    q, e = b.act8_store_into(z.cuda(), *b.act8_empty(6, K), act=act, Y=y)
    for i, w in enumerate(want):
        if w is not None:
            assert same(y[i, 5:6], torch.tensor([w], dtype=dtype)), (special[i], float(y[i, 5]))
    others = [c for c in range(K) if c != 5]
    assert torch.equal(y[:, others], plain[:, others])
    # the first three blocks are kept as NaN and no others are
    assert (e[:, 0] == -128).tolist() == [True] * 3 + [False] * 3 and bool((e[:, 1:] != -128).all())
    in_place = z.cuda()
    b.act8_store_into(in_place, q, e, act=act, Y=in_place)
    assert same(in_place, y.cpu())
