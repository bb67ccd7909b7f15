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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("where", ["X", "checkpoint", "dY", "H"])
@pytest.mark.parametrize("R", [5, 24, 64, 100])
def test_the_stacks_gradients_are_zero_past_the_rank(R, where, dtype):
    """... whatever the rows hold: an infinity or a NaN in a row of adapter 1 shows in its
    gradients, in the columns (rows) within its rank, and nowhere else."""
    b, M, K, N, L = binding(), 700, 136, 200, 3
    g = torch.Generator().manual_seed(R)
    X, dY = torch.randn(M, K, generator=g).to(dtype), torch.randn(M, N, generator=g).to(dtype)
    W, A, B = (torch.randn(*s, generator=g).to(dtype) for s in ((K, N), (L, K, R), (L, R, N)))
    H = torch.randn(M, R, generator=g)
    ids, ranks = torch.arange(M, dtype=torch.int32) % L, torch.tensor([R, R // 2, 0], dtype=torch.int32)
    row = 1                                  # of adapter 1
    if where in ("X", "checkpoint"):
        X[row, 40] = INF
    elif where == "dY":
        dY[row, 17] = INF
    else:
        H[row, 0], H[:, R // 2:] = NAN, NAN   # (past its rank an adapter's H is not read)
        H[0::3, R // 2:] = 1.0
    x = X.cuda()
    if where == "checkpoint":
        x = b.act8_store_into(x, *b.act8_empty(M, K))
    dA, dB = (torch.full(t.shape, 7.0, dtype=dtype, device="cuda") for t in (A, B))
    b.lora_backward_into(dY.cuda(), x, W.cuda(), A.cuda(), B.cuda(), ids.cuda(), H.cuda(), dA=dA, dB=dB,
                         ranks=ranks.cuda())
    for a in range(L):
        assert bool((dA[a, :, int(ranks[a]):] == 0).all()) and bool((dB[a, int(ranks[a]):] == 0).all())
    assert bool(torch.isfinite(dA[0]).all()) and bool(torch.isfinite(dB[0]).all())
    assert bool((dA[0] != 0).any()) and bool((dB[0] != 0).any())
    within_a, within_b = dA[1, :, :R // 2], dB[1, :R // 2]
    if where == "X":
        assert not torch.isfinite(within_a[40]).any() and bool(torch.isfinite(within_a[41:]).all())
    elif where == "checkpoint":               # the block of 32 columns
        assert not torch.isfinite(within_a[32:64]).any() and bool(torch.isfinite(within_a[64:]).all())
    elif where == "dY":
        assert not torch.isfinite(within_a).any() and not torch.isfinite(within_b[:, 17]).any()
        assert bool(torch.isfinite(within_b[:, 18:]).all())
    else:
        assert not torch.isfinite(within_b[0]).any() and bool(torch.isfinite(within_b[1:]).all())
    assert b.device_status() == b.SGEMM_OK


def product(x, w):
    """x w in 64 bits, every product and sum by IEEE 754's rules (infinity times zero among them)."""
    return torch.stack([(row.double().unsqueeze(1) * w.double()).sum(0) for row in x])


def same_kinds(got, ref):
    got = got.cpu().double()
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(kind(got), kind(ref)), (kind.__name__, int((kind(got) != kind(ref)).sum()))


def few_bits(rows, cols, seed):
    """Values that bfloat16 holds, zeros among them: float32 of these has nothing but zeros
    past its first bits."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-4, 5, (rows, cols), generator=g) / 2


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 40, 65, 300, 1500])
def test_infinities_of_x_and_w_are_those_of_the_formula(M, dtype):
    """However many rows there are: infinity times a number is infinity of its sign, times
    zero, or with infinity of the other sign in the sum, NaN."""
    b, K, N = binding(), 72, 136
    X, W = few_bits(M, K, 1), few_bits(K, N, 2)
    X[0, 3], W[5, 2], W[7, 4], W[8, 4], W[9, 6] = INF, INF, -INF, INF, NAN
    if M > 2:
        X[1, 4], X[2, 5], X[2, 6] = -INF, INF, -INF       # (X[2, 5] meets W[5, 2])
    W[3, 10:20] = torch.linspace(0.1, 2.3, 10)            # of all bits
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    A, B = torch.zeros(1, K, 4, dtype=dtype, device="cuda"), torch.zeros(1, 4, N, dtype=dtype, device="cuda")
    X, W = X.to(dtype), W.to(dtype)
    Y = b.lora_into(X.cuda(), W.cuda(), A, B, ids, torch.empty(M, N, dtype=dtype, device="cuda"))
    same_kinds(Y, product(X, W))
    dX = torch.empty(M, N, dtype=dtype, device="cuda")
    b.lora_backward_into(X.cuda(), dX, W.t().contiguous().cuda(), torch.zeros(1, N, 4, dtype=dtype, device="cuda"),
                         torch.zeros(1, 4, K, dtype=dtype, device="cuda"), ids, torch.zeros(M, 4, device="cuda"), dX=dX)
    same_kinds(dX, product(X, W))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [3, 16, 70, 1500])
def test_infinities_of_the_rank_side_are_those_of_the_formula(M, dtype):
    """An infinity in X reaches H and, through it, Y; one in dY reaches the gradients."""
    b, K, N, R = binding(), 72, 136, 4
    X, A, B, dY = few_bits(M, K, 1), few_bits(K, R, 2), few_bits(R, N, 3), few_bits(M, N, 4)
    W = torch.zeros(K, N)
    X[1, 3], dY[2, 7] = INF, -INF
    W[3] = torch.where((product(product(X[1:2], A), B)[0]) > 0, 1.0, -1.0)   # (no inf - inf by W)
    X, A, B, dY, W = (t.to(dtype) for t in (X, A, B, dY, W))
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    H = torch.empty(M, R, device="cuda")
    Y = b.lora_into(X.cuda(), W.cuda(), A[None].cuda(), B[None].cuda(), ids,
                    torch.empty(M, N, dtype=dtype, device="cuda"), H=H)
    h = product(X, A)
    same_kinds(H, h)
    same_kinds(Y, product(X, W) + product(h, B))
    dX, dA, dB = (torch.empty(*s, dtype=dtype, device="cuda") for s in ((M, K), (1, K, R), (1, R, N)))
    H = few_bits(M, R, 5)
    x = X.nan_to_num(0, 0, 0)
    b.lora_backward_into(dY.cuda(), x.cuda(), torch.zeros_like(W).cuda(), A[None].cuda(), B[None].cuda(), ids, H.cuda(),
                         dX=dX, dA=dA, dB=dB)
    G = product(dY, B.t())
    ref = product(dY, torch.zeros(N, K)) + product(G, A.t())
    same_kinds(dX, ref)
    same_kinds(dA[0], product(x.t(), G))
    same_kinds(dB[0], product(H.t(), dY))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 70, 700])
def test_infinities_of_a_weight_gradient_are_those_of_the_formula(M, dtype):
    b, K, N = binding(), 72, 136
    x, dY = few_bits(M, K, 1), few_bits(M, N, 2)
    dY[0, 3], dY[M // 2, 5], dY[M - 1, 7] = INF, -INF, NAN
    dY = dY.to(dtype)
    q, e = b.act8_store_into(x.cuda(), *b.act8_empty(M, K))
    dW = b.act8_weight_grad_into(q, e, dY.cuda(), torch.empty(K, N, dtype=dtype, device="cuda"))
    same_kinds(dW, product(x.t(), dY))
