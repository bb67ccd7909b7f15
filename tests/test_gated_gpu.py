"""The gated block, forward and backward, against 64 bits."""
import pytest
import torch

from _forward import (act_reference, gated_backward_reference, gated_reference, norm_close, rounded)
from _layers import device_matrix

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_device):
    yield


def binding():
    from dense_fp32_gemm_02_gb300 import binding
    return binding


def normal(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(dtype)


def weights(K, N, dtype, seed):
    return normal(K, N, dtype, seed, max(1, K) ** -0.5), normal(K, N, dtype, seed + 1, max(1, K) ** -0.5)


def check_forward(X, Wg, Wu, act, H, G=None, U=None):
    h, g, u, sh, sg, su = (t.cpu() for t in gated_reference(X, Wg, Wu, act))
    rounded(H, h, sh, "H")
    norm_close(H, h, "H")
    if G is not None:
        rounded(G, g, sg, "G")
        rounded(U, u, su, "U")
        norm_close(G, g, "G")
        norm_close(U, u, "U")


SHAPES = [(1, 1, 1), (1, 300, 200), (1, 2048, 1024), (2, 64, 515), (3, 1000, 64), (4, 77, 2000), (5, 128, 128), (8, 1031, 1000),
          (8, 4096, 2048), (9, 64, 64), (16, 200, 300), (17, 1000, 77), (33, 130, 1000), (64, 512, 512), (65, 96, 70), (100, 1111, 520),
          (256, 128, 64), (257, 129, 65), (300, 700, 1030), (1025, 200, 333), (700, 1536, 640)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(M, N, K, dtype):
    b = binding()
    X, (Wg, Wu) = normal(M, K, dtype, 1), weights(K, N, dtype, 2)
    for act in ("silu", "gelu"):
        H, G, U = (torch.full((M, N), 77, dtype=dtype, device="cuda") for _ in range(3))
        assert b.gated_into(X, Wg, Wu, H, act=act, G=G, U=U) is H
        check_forward(X, Wg, Wu, act, H, G, U)
        alone = torch.empty_like(H)
        b.gated_into(X, Wg, Wu, alone, act=act)
        assert torch.equal(alone, H)
    assert b.device_status() == 0


@pytest.mark.parametrize("pad", [0, 4, 3])
@pytest.mark.parametrize("M,N,K", [(17, 4, 1), (17, 128, 64), (31, 132, 63), (48, 260, 65), (64, 516, 257), (65, 128, 1000), (100, 96, 515),
                                   (128, 1000, 130), (129, 64, 260), (192, 388, 300), (193, 130, 70), (40, 64, 4100)])
def test_forward_between_few_and_many_rows(M, N, K, pad):
    """Float32 weights at pitches that the TMA reads and at others, over tiles and ranges that end inside one another."""
    b = binding()
    X, (Wg, Wu) = normal(M, K, torch.float32, 71), weights(K, N, torch.float32, 72)
    pg, pu = device_matrix(Wg.cpu(), pad, 4), device_matrix(Wu.cpu(), 0 if pad != 4 else 8, 0)
    flat = [torch.full((M + 2, N), 5.0, device="cuda") for _ in range(3)]
    H, G, U = (f[1:1 + M] for f in flat)
    b.gated_into(device_matrix(X.cpu(), 1, 1), pg, pu, H, G=G, U=U)
    check_forward(X, Wg, Wu, "silu", H, G, U)
    assert all(bool((f[0] == 5).all()) and bool((f[-1] == 5).all()) for f in flat)
    assert torch.equal(b.gated_into(X, pg, pu, torch.empty_like(H)), H)
    assert b.device_status() == 0


@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("M,N,K", [(1, 8, 1), (1, 128, 8200), (2, 136, 63), (7, 64, 65), (15, 200, 513), (16, 65, 1000), (17, 1031, 64),
                                   (32, 256, 2048), (33, 8, 300), (48, 129, 129), (63, 264, 70), (64, 1000, 520), (3, 72, 65536),
                                   (3, 72, 65537), (64, 40, 8193)])
def test_forward_of_few_bfloat16_rows(M, N, K, pad):
    """Tiles, ranges and rows that end inside one another, the projections kept or not; what lies around the outputs is
    left alone."""
    b = binding()
    X, (Wg, Wu) = normal(M, K, torch.bfloat16, 75), weights(K, N, torch.bfloat16, 76)
    pg, pu = device_matrix(Wg.cpu(), pad, pad), device_matrix(Wu.cpu(), 0, 0)
    flat = [torch.full((M + 2, N + 2), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    H, G, U = (f[1:1 + M, 1:1 + N] for f in flat)
    b.gated_into(device_matrix(X.cpu(), pad, 0), pg, pu, H, G=G, U=U, act="gelu")
    check_forward(X, Wg, Wu, "gelu", H, G, U)
    for f in flat:
        f[1:1 + M, 1:1 + N] = 5
    assert all(bool((f == 5).all()) for f in flat)
    alone = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    b.gated_into(X, pg, pu, alone, act="silu")
    check_forward(X, Wg, Wu, "silu", alone)
    assert b.device_status() == 0


@pytest.mark.parametrize("pad", [0, 3])
def test_values_of_every_size_between_few_and_many_rows(pad):
    """Float32 that needs all of its three parts, from 2^-100 to 2^60, each against the sum's own magnitudes; infinities reach
    their own rows and columns alone."""
    b = binding()
    M, N, K = 50, 200, 300
    g = torch.Generator()
    g.manual_seed(73)
    size = lambda *s: torch.exp2(torch.randint(-100, 61, s, generator=g).float())   # noqa: E731
    X, Wg = torch.randn(M, K, generator=g) * size(M, 1), torch.randn(K, N, generator=g) * size(1, N)
    Wu = torch.randn(K, N, generator=g)
    X[3, 5], Wg[7, 11], Wu[9, 13] = float("inf"), float("-inf"), float("nan")
    H, G, U = (torch.empty(M, N, device="cuda") for _ in range(3))
    b.gated_into(X.cuda(), device_matrix(Wg, pad), device_matrix(Wu, pad), H, act="relu", G=G, U=U)
    for got, W in ((G, Wg), (U, Wu)):
        ref, mag = X.double() @ W.double(), X.double().abs() @ W.double().abs()
        fine = torch.isfinite(ref) & (ref.abs() < 1e38)
        assert bool(torch.isfinite(got.cpu()[fine]).all())
        # the six pairs leave 2^-23.4 of a product, sums and their chunks (16 truncating additions of 2^-23, 3 chunks) the rest
        over = (got.cpu().double() - ref).abs()[fine] > (24 * 2.0 ** -23) * mag[fine] + 1e-37
        assert not bool(over.any())
        odd = ~torch.isfinite(ref)
        assert not bool(torch.isfinite(got.cpu()[odd]).any())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M", [2, 40, 300])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_other_activations(M, act, dtype):
    b = binding()
    X, (Wg, Wu) = normal(M, 100, dtype, 3), weights(100, 72, dtype, 4)
    H = torch.empty(M, 72, dtype=dtype, device="cuda")
    b.gated_into(X, Wg, Wu, H, act=act)
    check_forward(X, Wg, Wu, act, H)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K,pad,offset", [(1, 64, 100, 3, 1), (6, 130, 64, 8, 8), (8, 200, 70, 1, 5), (20, 96, 100, 8, 0),
                                              (70, 200, 90, 8, 8), (300, 257, 130, 5, 3)])
def test_views(M, N, K, pad, offset, dtype):
    """Any pitch and alignment, each matrix its own; what lies beside the outputs is left alone."""
    b = binding()
    X, (Wg, Wu) = normal(M, K, dtype, 5), weights(K, N, dtype, 6)
    flat = [torch.full((M, N + pad + 2), 5.0, dtype=dtype, device="cuda") for _ in range(3)]
    H, G, U = (f[:, 1:1 + N] for f in flat)
    pg, pu = device_matrix(Wg.cpu(), pad, offset), device_matrix(Wu.cpu(), 0, 0)
    b.gated_into(device_matrix(X.cpu(), pad, offset), pg, pu, H, G=G, U=U)
    check_forward(X, Wg, Wu, "silu", H, G, U)
    both = torch.cat((Wg, Wu), 1)      # the halves of one matrix
    again = torch.empty(M, N, dtype=dtype, device="cuda")
    b.gated_into(X, both[:, :N], both[:, N:], again)
    check_forward(X, Wg, Wu, "silu", again)
    assert all(bool((f[:, 0] == 5).all()) and bool((f[:, 1 + N:] == 5).all()) for f in flat)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
def test_far_values_of_the_activation(act, dtype):
    """G from -120 to 120: the exponentials' whole range; relative to the value where the tail is small."""
    b = binding()
    z = torch.linspace(-120, 120, 1001)
    X = torch.ones(20, 1, dtype=dtype, device="cuda")
    Wg, Wu = z.to(dtype).cuda().unsqueeze(0), torch.ones(1, 1001, dtype=dtype, device="cuda")
    H = torch.empty(20, 1001, dtype=dtype, device="cuda")
    for rows in (1, 20):
        b.gated_into(X[:rows], Wg, Wu, H[:rows], act=act)
        check_forward(X[:rows], Wg, Wu, act, H[:rows])
    if act == "silu":
        g = Wg[0].double().cpu()
        ref = act_reference(g, act)[0]
        near = (g > -85) & (g != 0)     # (beyond, the value is below the least normal number)
        rel = ((H[0].double().cpu() - ref) / ref).abs()[near]
        assert float(rel.max()) <= (2.0 ** -8 if dtype == torch.bfloat16 else 0) + 140 * 2.0 ** -23


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M", [3, 30, 300])
def test_infinities_and_nans(M, dtype):
    b = binding()
    X, (Wg, Wu) = normal(M, 70, dtype, 7), weights(70, 90, dtype, 8)
    X[0, 3], X[1, 5] = float("inf"), float("nan")
    Wg[7, 11], Wu[9, 13] = float("-inf"), float("nan")
    H, G, U = (torch.empty(M, 90, dtype=dtype, device="cuda") for _ in range(3))
    for act in ("silu", "gelu", "relu"):
        b.gated_into(X, Wg, Wu, H, act=act, G=G, U=U)
        g, u = X.double() @ Wg.double(), X.double() @ Wu.double()
        h = act_reference(g, act)[0] * u
        for got, ref, what in ((G, g, "G"), (U, u, "U"), (H, h, "H")):
            assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
            assert torch.equal(torch.isinf(got), torch.isinf(ref)), what
            inf = torch.isinf(ref)
            assert torch.equal(got[inf].double(), ref[inf]), what


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_long_contractions(dtype):
    """Sums that are added up in chunks, in one range and in several."""
    b = binding()
    for M, N, K in ((20000, 16, 9001), (300, 200, 20000), (70, 64, 40000)):
        X, (Wg, Wu) = normal(M, K, dtype, 9), weights(K, N, dtype, 10)
        H, G, U = (torch.empty(M, N, dtype=dtype, device="cuda") for _ in range(3))
        b.gated_into(X, Wg, Wu, H, G=G, U=U)
        check_forward(X, Wg, Wu, "silu", H, G, U)


# ------------------------------------------------------------------ backward
def check_backward(args, act, dX=None, dWg=None, dWu=None):
    x, g, u, sx, sg, su = (t.cpu() for t in gated_backward_reference(*args, act))
    for got, ref, slack, what in ((dX, x, sx, "dX"), (dWg, g, sg, "dWg"), (dWu, u, su, "dWu")):
        if got is not None:
            rounded(got, ref, slack, what)
            norm_close(got, ref, what)


def backward_args(M, N, K, dtype, seed):
    X, (Wg, Wu) = normal(M, K, dtype, seed), weights(K, N, dtype, seed + 1)
    return normal(M, N, dtype, seed + 3), X, Wg, Wu, normal(M, N, dtype, seed + 4, 1.5), normal(M, N, dtype, seed + 5, 1.5)


def empty_gradients(M, N, K, dtype):
    return (torch.full((M, K), 77, dtype=dtype, device="cuda"), torch.full((K, N), 77, dtype=dtype, device="cuda"),
            torch.full((K, N), 77, dtype=dtype, device="cuda"))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[0] != 4] + [(2000, 64, 40), (40, 300, 2000)])
def test_backward(M, N, K, dtype):
    b = binding()
    args = backward_args(M, N, K, dtype, 20)
    for act in ("silu", "gelu"):
        dX, dWg, dWu = empty_gradients(M, N, K, dtype)
        out = b.gated_backward_into(*args, dX=dX, dWg=dWg, dWu=dWu, act=act)
        assert out[0] is dX and out[1] is dWg and out[2] is dWu
        check_backward(args, act, dX, dWg, dWu)
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("act", ["none", "relu"])
def test_backward_of_other_activations(act, dtype):
    b = binding()
    args = backward_args(70, 90, 64, dtype, 30)
    args[4][0, :5] = 0.0
    dX, dWg, dWu = empty_gradients(70, 90, 64, dtype)
    b.gated_backward_into(*args, dX=dX, dWg=dWg, dWu=dWu, act=act)
    check_backward(args, act, dX, dWg, dWu)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_gradients_alone(dtype):
    """Each gradient without the others is the same; what it does not need may be missing."""
    b = binding()
    dH, X, Wg, Wu, G, U = backward_args(150, 90, 70, dtype, 40)
    dX, dWg, dWu = b.gated_backward_into(dH, X, Wg, Wu, G, U, *empty_gradients(150, 90, 70, dtype))
    alone = b.gated_backward_into(dH, None, Wg, Wu, G, U, dX=torch.empty_like(dX))
    assert torch.equal(alone[0], dX) and alone[1] is None and alone[2] is None
    alone = b.gated_backward_into(dH, X, Wg, Wu, G, U, dWg=torch.empty_like(dWg), dWu=torch.empty_like(dWu))
    assert alone[0] is None and torch.equal(alone[1], dWg) and torch.equal(alone[2], dWu)
    launches = b.kernel_launch_count()
    assert b.gated_backward_into(dH, X, Wg, Wu, G, U) == (None, None, None)
    assert b.kernel_launch_count() == launches
    with pytest.raises(ValueError, match="given together"):
        b.gated_backward_into(dH, X, Wg, Wu, G, U, dWg=torch.empty_like(dWg))
    with pytest.raises(TypeError, match="X must be"):
        b.gated_backward_into(dH, None, Wg, Wu, G, U, dWg=dWg, dWu=dWu)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K,pad,offset", [(1, 64, 100, 3, 1), (70, 200, 90, 8, 8), (300, 257, 130, 5, 3)])
def test_backward_views(M, N, K, pad, offset, dtype):
    b = binding()
    args = backward_args(M, N, K, dtype, 50)
    placed = [device_matrix(t.cpu(), pad + (i % 2) * 8, offset) for i, t in enumerate(args)]
    flat = [torch.full((r, c + pad + 2), 5.0, dtype=dtype, device="cuda") for r, c in ((M, K), (K, N), (K, N))]
    dX, dWg, dWu = (f[:, 1:-pad - 1] for f in flat)
    b.gated_backward_into(*placed, dX=dX, dWg=dWg, dWu=dWu)
    check_backward(args, "silu", dX, dWg, dWu)
    assert all(bool((f[:, 0] == 5).all()) and bool((f[:, -pad - 1:] == 5).all()) for f in flat)
    both = torch.empty(K, 2 * N, dtype=dtype, device="cuda")       # the gradients as halves of one matrix
    b.gated_backward_into(*args, dWg=both[:, :N], dWu=both[:, N:])
    check_backward(args, "silu", None, both[:, :N], both[:, N:])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_backward_of_long_sums(dtype):
    b = binding()
    for M, N, K in ((20000, 64, 40), (200, 10000, 64), (9000, 300, 264)):
        args = backward_args(M, N, K, dtype, 60)
        dX, dWg, dWu = empty_gradients(M, N, K, dtype)
        b.gated_backward_into(*args, dX=dX, dWg=dWg, dWu=dWu)
        check_backward(args, "silu", dX, dWg, dWu)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_against_differences(act):
    """The gradients against central differences of the forward pass in 64 bits."""
    b = binding()
    M, N, K = 3, 8, 6
    X, (Wg, Wu), dH = normal(M, K, torch.float32, 70), weights(K, N, torch.float32, 71), normal(M, N, torch.float32, 73)
    H, G, U = (torch.empty(M, N, device="cuda") for _ in range(3))
    b.gated_into(X, Wg, Wu, H, act=act, G=G, U=U)
    dX, dWg, dWu = empty_gradients(M, N, K, torch.float32)
    b.gated_backward_into(dH, X, Wg, Wu, G, U, dX=dX, dWg=dWg, dWu=dWu, act=act)
    at = [t.double().cpu() for t in (X, Wg, Wu)]
    dh, step = dH.double().cpu(), 1e-5

    def loss(x, wg, wu):
        return float((act_reference(x @ wg, act)[0] * (x @ wu) * dh).sum())
    for which, got in enumerate((dX, dWg, dWu)):
        for i in range(got.shape[0]):
            for j in range(got.shape[1]):
                lo, hi = [t.clone() for t in at], [t.clone() for t in at]
                lo[which][i, j] -= step
                hi[which][i, j] += step
                # the difference's own error: step^2 times the third derivative, and 1e-16 / step
                assert abs((loss(*hi) - loss(*lo)) / (2 * step) - float(got[i, j])) < 2e-5


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_nothing_to_add_up(dtype):
    b = binding()
    e = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")   # noqa: E731
    H, G, U = (torch.full((5, 30), 7, dtype=dtype, device="cuda") for _ in range(3))
    b.gated_into(e(5, 0), e(0, 30), e(0, 30), H, G=G, U=U)
    assert all(bool((t == 0).all()) for t in (H, G, U))
    b.gated_into(e(0, 9), e(9, 30), e(9, 30), e(0, 30))
    b.gated_into(e(4, 9), e(9, 0), e(9, 0), e(4, 0))
    dX, dWg, dWu = empty_gradients(0, 30, 9, dtype)
    b.gated_backward_into(e(0, 30), e(0, 9), e(9, 30), e(9, 30), e(0, 30), e(0, 30), dX=dX, dWg=dWg, dWu=dWu)
    assert bool((dWg == 0).all()) and bool((dWu == 0).all())
    dX = torch.full((4, 9), 7, dtype=dtype, device="cuda")
    b.gated_backward_into(e(4, 0), e(4, 9), e(9, 0), e(9, 0), e(4, 0), e(4, 0), dX=dX)
    assert bool((dX == 0).all())
    b.gated_backward_into(e(4, 30), e(4, 0), e(0, 30), e(0, 30), e(4, 30), e(4, 30), dX=e(4, 0), dWg=e(0, 30), dWu=e(0, 30))
    assert b.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_bitwise_the_same_from_call_to_call(dtype):
    b = binding()
    for M in (1, 8, 60, 700):
        args = backward_args(M, 520, 264, dtype, 80)
        dH, X, Wg, Wu, G, U = args
        h = b.gated_into(X, Wg, Wu, torch.empty_like(dH))
        d = b.gated_backward_into(*args, *empty_gradients(M, 520, 264, dtype))
        for _ in range(3):
            assert torch.equal(b.gated_into(X, Wg, Wu, torch.empty_like(dH)), h)
            again = b.gated_backward_into(*args, *empty_gradients(M, 520, 264, dtype))
            assert all(torch.equal(x, y) for x, y in zip(d, again))
