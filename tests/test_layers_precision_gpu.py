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


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("M", [3, 40, 300, 1500])
def test_the_rank_side_keeps_fp32(M, dtype):
    """X A is 2^20 + 2^10 + 1 and 2^20 + 2^10 (21 bits, with a gap in them after the first 8 and
    after the next), and B takes one from the other: exactly 1 in fp32."""
    b, K, N = binding(), 72, 264
    X, A, B = torch.zeros(M, K), torch.zeros(1, K, 2), torch.zeros(1, 2, N)
    X[:, 0], X[:, 1], X[:, 2] = 1024, 32, 1
    A[0, 0], A[0, 1], A[0, 2, 0] = 1024, 32, 1
    B[0, 0], B[0, 1] = 1, -1
    X, A, B = (t.to(dtype).cuda() for t in (X, A, B))
    Y = torch.empty(M, N, dtype=dtype, device="cuda")
    b.lora_into(X, torch.zeros(K, N, dtype=dtype, device="cuda"), A, B,
                torch.zeros(M, dtype=torch.int32, device="cuda"), Y)
    assert bool((Y == 1).all())


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("M", [2, 700])
def test_the_rank_sides_gradients_keep_fp32(M, dtype):
    """The same of the gradients: G in dX and in dA, H in dB."""
    b, K, N = binding(), 72, 264
    X, dY, H = torch.zeros(M, K), torch.zeros(M, N), torch.zeros(M, 2)
    A, B = torch.zeros(1, K, 2), torch.zeros(1, 2, N)
    X[0], X[1] = 1, -1
    dY[:2, 0], dY[:2, 1], dY[0, 2] = 1024, 32, 1
    dY[0, 5], dY[1, 5] = 1, -1
    B[0, :, 0], B[0, :, 1], B[0, 0, 2] = 1024, 32, 1
    H[0, 0], H[1, 0] = 2 ** 20 + 2 ** 10 + 1, 2 ** 20 + 2 ** 10
    A[0, :, 0], A[0, :, 1] = 1, -1
    X, dY, A, B = (t.to(dtype).cuda() for t in (X, dY, A, B))
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[:2] = 0
    dX, dA, dB = b.lora_backward_into(dY, X, torch.zeros(K, N, dtype=dtype, device="cuda"), A, B, ids, H.cuda(),
                                      dX=torch.empty_like(X), dA=torch.empty_like(A), dB=torch.empty_like(B))
    assert bool((dX[0] == 1).all()) and bool((dX[1] == 0).all())
    assert bool((dA[0, :, 0] == 1).all()) and bool((dA[0, :, 1] == 0).all())
    assert bool((dB[0, 0, 5] == 1).all()) and bool((dB[0, 1] == 0).all())


@pytest.mark.parametrize("K", [128, 131])     # rows read 16 bytes at a time, and of any alignment
def test_gelu_keeps_the_relative_accuracy_of_small_values(K):
    """float32 at z from -8 to 0, where Phi falls to 6e-16.  Relative: exp(-z^2/2) is off by the
    roundings of its exponent, 2^-23 z^2/2 (6e-8 z^2), and by 2e-7 of its own; the tail over it by
    6e-7; products and sums by 2^-24 each: under 2e-6 + 6e-8 z^2.  The slope below -3 is a difference
    of which the smaller part is a ninth at most: a quarter more."""
    b = binding()
    z = -(torch.arange(64 * K, device="cuda") % 128).view(64, K).float() / 16      # kept exactly
    z[:, ::32] = -127 / 16
    y = torch.empty_like(z)
    q, e = b.act8_store_into(z, *b.act8_empty(64, K), act="gelu", Y=y)
    assert torch.equal(b.act8_load_into(q, e, torch.empty_like(z)), z)
    slope = b.act8_grad_into(q, e, torch.ones_like(z), torch.empty_like(z), act="gelu").double()
    z = z.double()
    cdf, bell = 0.5 * torch.erfc(-z / 2 ** 0.5), torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    limit = 2e-6 + 6e-8 * z * z
    assert bool(((y.double() - z * cdf).abs() <= limit * (z * cdf).abs()).all())
    ref = cdf + z * bell
    low = z < -3
    assert bool(((slope - ref).abs() <= 1.25 * limit * ref.abs())[low].all())
    assert float((slope - ref).abs().max()) <= 4e-7


@pytest.mark.parametrize("R", [16, 128])
def test_adapters_beside_a_long_contraction(R):
    """The rank side's slabs come after those of a contraction that is added up in chunks.  A
    result is within half a bfloat16 spacing (2^-8) of a sum that is off by at most 3.3e-5 of its
    terms' magnitudes (the contraction) and 2^-23 of each of the R terms beside it."""
    b, M, LONG, SHORT, L = binding(), 4096, 8320, 2560, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(R)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)   # noqa: E731
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    some = slice(0, SHORT, 20)

    def check(got, x, w, v1, v2):     # got = x w + (x v1) v2 of the row's adapter
        ref, mag = x.double() @ w[:, some].double(), x.double().abs() @ w[:, some].double().abs()
        for a in range(L):
            mine = (ids == a).double().unsqueeze(1)
            s = mine * (x.double() @ v1[a].double())
            ref += s @ v2[a][:, some].double()
            mag += (mine * (x.double().abs() @ v1[a].double().abs())) @ v2[a][:, some].double().abs() * R * 2.0 ** -8
        err = (got[:, some].double() - ref).abs()
        limit = 3.3e-5 * mag
        assert bool((err <= 2.0 ** -8 * (ref.abs() + limit) + limit).all())

    X, W, A, B = r(M, LONG), r(LONG, SHORT), r(L, LONG, R), r(L, R, SHORT)
    Y = b.lora_into(X, W, A, B, ids, torch.empty(M, SHORT, dtype=BF16, device="cuda"))
    check(Y, X, W, A, B)
    dX = torch.empty(M, SHORT, dtype=BF16, device="cuda")
    A, B, W = A.transpose(1, 2).contiguous(), B.transpose(1, 2).contiguous(), W.t().contiguous()
    b.lora_backward_into(X, dX, W, B, A, ids, torch.zeros(M, R, device="cuda"), dX=dX)
    check(dX, X, W.t(), A.transpose(1, 2), B.transpose(1, 2))
    assert b.device_status() == b.SGEMM_OK
