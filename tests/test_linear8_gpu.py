"""The product of int8 matrices with scales against exact sums."""
import pytest
import torch

from _forward import linear8_reference, rounded, rows8_reference
from _layers import device_matrix

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def bytes_of(rows, cols, seed, low=-128):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randint(low, 128, (rows, cols), generator=g, dtype=torch.int32).to(torch.int8)


def floats(n, seed, dtype=torch.float32):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.rand(n, generator=g) * 0.01 + 1e-4).to(dtype)


def check(Y, q, scale, W, wscale, bias, what):
    ref, mag = linear8_reference(q.cuda(), scale.cuda(), W.cuda(), wscale.cuda(), None if bias is None else bias.cuda())
    # the exact sum to fp32, the scales' product, theirs, the bias: four roundings
    rounded(Y, ref.cpu(), 4 * 2.0 ** -24 * mag.cpu(), what)


SHAPES = [(1, 1, 1), (1, 520, 33), (1, 4096, 4096), (2, 511, 100), (3, 64, 1025), (4, 1000, 1000), (5, 16, 8), (8, 2048, 515),
          (9, 64, 64), (12, 1031, 77), (64, 520, 1024), (70, 130, 2049), (130, 600, 1030), (256, 256, 64), (257, 300, 3001),
          (513, 1111, 520), (1000, 64, 5000), (300, 4000, 128)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_rows_in_8_bits(M, N, K, dtype):
    b = binding()
    q, W, scale, wscale = bytes_of(M, K, 1), bytes_of(K, N, 2), floats(M, 3), floats(N, 4)
    for bias in (None, floats(N, 5, dtype) * 100):
        Y = torch.full((M, N), 77, dtype=dtype, device="cuda")
        assert b.linear8_into((q.cuda(), scale.cuda()), W.cuda(), wscale.cuda(), Y, bias=None if bias is None else bias.cuda()) is Y
        check(Y, q, scale, W, wscale, bias, "Y")
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 520, 33), (4, 1000, 1000), (8, 300, 2048), (40, 130, 515), (300, 600, 1024)])
def test_rows_of_the_type(M, N, K, dtype):
    """Rows that the call brings to 8 bits are those of the definition."""
    b = binding()
    g = torch.Generator()
    g.manual_seed(6)
    X = (torch.randn(M, K, generator=g) * 3).to(dtype)
    X[M // 2] = 0
    W, wscale = bytes_of(K, N, 7, -127), floats(N, 8)
    q, scale = rows8_reference(X)
    Y = torch.empty(M, N, dtype=dtype, device="cuda")
    b.linear8_into(X.cuda(), W.cuda(), wscale.cuda(), Y)
    ref, mag = linear8_reference(q, scale, W, wscale, None)
    rounded(Y, ref, 5 * 2.0 ** -24 * mag, "Y")      # (the rows' scale is rounded too)
    assert bool((Y[M // 2] == 0).all())
    X[0, K // 3] = float("nan")
    b.linear8_into(X.cuda(), W.cuda(), wscale.cuda(), Y)
    assert bool(torch.isnan(Y[0]).all()) and (M == 1 or bool(torch.isfinite(Y[1:]).all()))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("N,K", [(1, 1), (63, 3), (65, 5), (128, 256), (129, 257), (2432, 511), (2433, 513), (70, 2049), (64, 16385),
                                 (9, 65536), (7, 65537), (20000, 40)])
def test_few_rows(M, N, K, dtype):
    """Rows given in 8 bits and rows of the type, from aligned and from odd places, with the same sums."""
    b = binding()
    g = torch.Generator()
    g.manual_seed(M * 100003 + N * 101 + K)
    X = (torch.randn(M, K, generator=g) * 5).to(dtype)
    W, wscale, bias = bytes_of(K, N, 41), floats(N, 42), floats(N, 43, dtype)
    q, scale = rows8_reference(X)
    scale = scale.float()
    flat = torch.full((K * N + 64,), 99, dtype=torch.int8, device="cuda")
    for offset in (0, 1, 4, 8):
        view = flat[offset:offset + K * N].view(K, N)
        view.copy_(W)
        Y, Z = (torch.full((M, N + 1), 3.0, dtype=dtype, device="cuda")[:, :N] for _ in range(2))
        b.linear8_into((q.cuda(), scale.cuda()), view, wscale.cuda(), Y, bias=bias.cuda())
        check(Y, q, scale, W, wscale, bias, "Y")
        b.linear8_into(device_matrix(X, offset, offset // 4), view, wscale.cuda(), Z, bias=bias.cuda())
        ref, mag = linear8_reference(q, rows8_reference(X)[1], W, wscale, bias)
        rounded(Z, ref, 5 * 2.0 ** -24 * mag, "rows of the type")
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M", [1, 2, 4])
def test_few_rows_out_of_range(M, dtype):
    """Rows of the smallest and the largest values, of ties, of zeros, with an infinity and a NaN: as in many rows."""
    b = binding()
    K, N = 1000, 200
    x = torch.arange(K).float() % 255 - 127.0
    rows = [x * 0.5, x * 2.0 ** -133, x * 2.0 ** -120, x * 2.0 ** 120, x * 2.0 ** 115, x * 0.0, x + 0.0, x * 1.5, x.clone()]
    rows[6][17], rows[7][999], rows[8][0] = float("inf"), float("-inf"), float("nan")
    W, wscale = bytes_of(K, N, 44), floats(N, 45)
    many = torch.stack(rows + [x * 0.75] * 8).to(dtype).cuda()
    all_rows = b.linear8_into(many, W.cuda(), wscale.cuda(), torch.empty(len(many), N, dtype=dtype, device="cuda"))
    for r in range(len(rows)):
        Y = b.linear8_into(many[r:r + M].contiguous(), W.cuda(), wscale.cuda(), torch.empty(M, N, dtype=dtype, device="cuda"))
        assert torch.equal(torch.nan_to_num(Y, 3.0), torch.nan_to_num(all_rows[r:r + M], 3.0)), r


@pytest.mark.parametrize("fill", [63, 64, 65, 127, -128])
def test_many_rows_with_magnitudes_at_the_bound(fill):
    """Rows whose 2048 magnitudes add up to just under, to and past 2^17, in one row of many: sums that fp32 holds
    exactly every 2048 terms, or every 1024 only."""
    b = binding()
    M, N, K = 2600, 4096, 4500
    q, W = bytes_of(M, K, 31, -20) // 7, bytes_of(K, N, 32)
    q[1234, 2048:4096] = fill
    W[:, ::2] = 127
    W[:, 1::4] = -128
    one, ones, Y = torch.ones(M, device="cuda"), torch.ones(N, device="cuda"), torch.empty(M, N, device="cuda")
    b.linear8_into((q.cuda(), one), W.cuda(), ones, Y)
    assert torch.equal(Y, (q.cuda().double() @ W.cuda().double()).float())


@pytest.mark.parametrize("M", [1, 8, 40, 300, 700])
@pytest.mark.parametrize("K", [1024, 5000, 131071])
def test_the_largest_sums_are_exact(M, K):
    """All values at their limits: sums up to 2^31, to the last integer."""
    b = binding()
    N = 70
    q, W = torch.full((M, K), -128, dtype=torch.int8), torch.full((K, N), -128, dtype=torch.int8)
    W[:, 1::3] = 127
    W[::2, 2::3] = 127
    q[::2, ::5] = 127
    W[K - 1, :] = bytes_of(1, N, 3)[0]
    Y = torch.empty(M, N, device="cuda")
    one, ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    b.linear8_into((q.cuda(), one), W.cuda(), ones, Y)
    sums = (q.double().cuda() @ W.double().cuda()).cpu()
    assert torch.equal(Y.cpu(), sums.float())
    # the lowest bits too: the sum less what fp32 keeps of it, by a bias in the other direction
    b.linear8_into((q.cuda(), one), W.cuda(), ones, Y, bias=(-sums[0]).float().cuda())
    assert torch.equal(Y.cpu(), (sums.float().double() - sums[0].float().double()).float())
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K,pad,offset", [(1, 64, 100, 3, 1), (5, 130, 64, 16, 16), (8, 513, 70, 1, 5), (40, 200, 90, 8, 8),
                                              (300, 257, 130, 5, 3)])
def test_views(M, N, K, pad, offset, dtype):
    b = binding()
    q, W, scale, wscale, bias = bytes_of(M, K, 11), bytes_of(K, N, 12), floats(M, 13), floats(N, 14), floats(N + 1, 15, dtype)

    def placed(x, p):
        flat = torch.full((x.shape[0] * (x.shape[1] + p) + offset + 8,), 99, dtype=torch.int8, device="cuda")
        view = flat[offset:offset + x.shape[0] * (x.shape[1] + p)].view(x.shape[0], x.shape[1] + p)[:, :x.shape[1]]
        view.copy_(x)
        return view
    flat = torch.full((M, N + pad + 2), 5.0, dtype=dtype, device="cuda")
    Y = flat[:, 1:1 + N]
    b.linear8_into((placed(q, pad), scale.cuda()), placed(W, pad + 1), wscale.cuda(), Y, bias=bias.cuda()[1:])
    check(Y, q, scale, W, wscale, bias[1:], "Y")
    assert bool((flat[:, 0] == 5).all()) and bool((flat[:, 1 + N:] == 5).all())
    X = (torch.arange(M * K).reshape(M, K) % 23 - 11).to(dtype)
    Z = torch.empty_like(Y)
    b.linear8_into(device_matrix(X, pad, offset), W.cuda(), wscale.cuda(), Z)
    q2, s2 = rows8_reference(X)
    ref, mag = linear8_reference(q2, s2, W, wscale, None)
    rounded(Z, ref, 5 * 2.0 ** -24 * mag, "rows of the type")


def test_scales_of_infinity_zero_and_nan():
    b = binding()
    for M in (4, 40):
        q, W = bytes_of(M, 50, 16), bytes_of(50, 60, 17)
        scale, wscale = floats(M, 18), floats(60, 19)
        scale[1], scale[2], wscale[3] = float("nan"), 0.0, float("inf")
        Y = torch.empty(M, 60, device="cuda")
        b.linear8_into((q.cuda(), scale.cuda()), W.cuda(), wscale.cuda(), Y)
        ref = (q.double() @ W.double()).float() * (scale.unsqueeze(1) * wscale)
        assert torch.equal(torch.isnan(Y.cpu()), torch.isnan(ref)) and torch.equal(torch.isinf(Y.cpu()), torch.isinf(ref))
        fine = torch.isfinite(ref)
        assert torch.equal(Y.cpu()[fine], ref[fine])


def test_nothing_to_add_up():
    b = binding()
    for M in (3, 40):
        Y, bias = torch.full((M, 20), 7.0, device="cuda"), floats(20, 20).cuda()
        q, W = torch.empty(M, 0, dtype=torch.int8, device="cuda"), torch.empty(0, 20, dtype=torch.int8, device="cuda")
        scale, wscale = floats(M, 21).cuda(), floats(20, 22).cuda()
        b.linear8_into((q, scale), W, wscale, Y, bias=bias)
        assert torch.equal(Y, bias.expand(M, 20))
        b.linear8_into(torch.empty(M, 0, device="cuda"), W, wscale, Y)
        assert bool((Y == 0).all())
    b.linear8_into((torch.empty(0, 9, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")),
                   torch.empty(9, 20, dtype=torch.int8, device="cuda"), wscale, torch.empty(0, 20, device="cuda"))
    assert b.device_status() == 0


@pytest.mark.parametrize("M", [1, 8, 64, 700])
def test_bitwise_the_same_from_call_to_call(M):
    b = binding()
    q, W, scale, wscale = bytes_of(M, 3001, 23).cuda(), bytes_of(3001, 1024, 24).cuda(), floats(M, 25).cuda(), floats(1024, 26).cuda()
    first = b.linear8_into((q, scale), W, wscale, torch.empty(M, 1024, device="cuda"))
    for _ in range(5):
        assert torch.equal(b.linear8_into((q, scale), W, wscale, torch.empty(M, 1024, device="cuda")), first)
